"""Thin ctypes binding of libmxq (include/mxq.h).

Argument marshalling only: every step of the computation runs in the HIP
kernels of libmxq.so.  PyTorch supplies device memory and the current stream.
Loading fails loudly when the library has not been built; there is no
fallback path.
"""
from __future__ import annotations

import ctypes as C
import os

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libmxq.so")

OK, ERR_NULL, ERR_SHAPE, ERR_ALIGN, ERR_UNSUPPORTED, ERR_DEVICE, ERR_WORKSPACE = range(7)
GRID_E2M1, GRID_E1M2, GRID_E2M1_MAX4, GRID_E2M1_MAX3 = 0, 1, 2, 3
RTNE, SR = 0, 1
FMT_FP4, FMT_E2M3 = 0, 1
LAYOUT_ROWS, LAYOUT_MFMA = 0, 1
AXIS_ROW, AXIS_COL = 0, 1
OUT_F32, OUT_BF16 = 0, 1
SIGNS_MASK, SIGNS_PER_BLOCK = 0, 1
NORM_LAYER, NORM_RMS = 0, 1
TOP_MAX = 64

SYMBOLS = ("mxq_quantize", "mxq_quantize_batch", "mxq_dequantize", "mxq_wgrad_gemm", "mxq_gemm_abt", "mxq_bias_stats",
           "mxq_bias_stats_workspace_size", "mxq_bias_stats_noalloc", "mxq_bucket_ratio", "mxq_round_to_grid", "mxq_rht_sign_mask", "mxq_rotate",
           "mxq_norm_forward", "mxq_norm_backward", "mxq_norm_backward_workspace_size", "mxq_token_logprobs",
           "mxq_token_logprobs_backward", "mxq_vocab_workspace_size", "mxq_distill_forward",
           "mxq_distill_backward", "mxq_distill", "mxq_linear_ce_forward", "mxq_linear_ce_forward_workspace_size",
           "mxq_linear_ce_backward", "mxq_linear_ce_backward_workspace_size",
           "mxq_grad_norm", "mxq_grad_norm_workspace_size", "mxq_grad_clip", "mxq_status_string", "mxq_abi_version")


class QConfig(C.Structure):
    _fields_ = [("grid", C.c_int32), ("round", C.c_int32), ("hadamard_n", C.c_int32),
                ("sign_mask", C.c_uint32), ("sr_seed", C.c_uint64), ("sr_stream", C.c_uint32),
                ("sr_bits", C.c_uint32), ("sign_mode", C.c_uint32), ("reserved", C.c_uint32),
                ("sign_seed", C.c_uint64)]


class QTensor(C.Structure):
    _fields_ = [("codes", C.c_void_p), ("scales", C.c_void_p), ("fmt", C.c_int32),
                ("grid", C.c_int32), ("layout", C.c_int32)]


class Grad(C.Structure):
    _fields_ = [("g", C.c_void_p), ("out", C.c_void_p), ("n", C.c_int64), ("dtype", C.c_int32), ("out_dtype", C.c_int32)]


class QuantizeJob(C.Structure):
    _fields_ = [("cfg", C.POINTER(QConfig)), ("x", C.c_void_p), ("rows", C.c_int64),
                ("cols", C.c_int64), ("ld_x", C.c_int64), ("row_out", C.POINTER(QTensor)),
                ("col_out", C.POINTER(QTensor))]


class Stats(C.Structure):
    _fields_ = [("sum_abs_y", C.c_double), ("sum_signed_err", C.c_double),
                ("sum_y2", C.c_double), ("sum_err2", C.c_double), ("sum_err_norm", C.c_double),
                ("sum_err_norm_sat", C.c_double), ("level_err_norm", C.c_double * 8),
                ("n", C.c_uint64), ("n_saturated", C.c_uint64),
                ("n_nonfinite_blocks", C.c_uint64), ("level_count", C.c_uint64 * 8)]


class MxqError(RuntimeError):
    def __init__(self, fn: str, status: int):
        super().__init__(f"{fn} failed: {status_string(status)} (status {status})")
        self.status = status


_lib = None


def lib() -> C.CDLL:
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"libmxq.so is not built ({LIB_PATH}); run "
                              "`python -m fp4_microscaling_quantization_amd.build` first")
        L = C.CDLL(LIB_PATH)
        P, i32, i64 = C.c_void_p, C.c_int32, C.c_int64
        L.mxq_quantize.argtypes = [C.POINTER(QConfig), P, i64, i64, i64, C.POINTER(QTensor),
                                   C.POINTER(QTensor), P]
        L.mxq_quantize_batch.argtypes = [C.POINTER(QuantizeJob), i32, P]
        L.mxq_dequantize.argtypes = [C.POINTER(QTensor), i64, i64, i32, P, i64, P]
        L.mxq_wgrad_gemm.argtypes = [C.POINTER(QTensor), C.POINTER(QTensor), i64, i64, i64, P,
                                     i64, P]
        L.mxq_gemm_abt.argtypes = L.mxq_wgrad_gemm.argtypes
        L.mxq_rht_sign_mask.argtypes = [C.c_uint64, C.c_uint32]
        L.mxq_rotate.argtypes = [C.POINTER(QConfig), P, i64, i64, i64, i32, i32, P, i64, P]
        L.mxq_rht_sign_mask.restype = C.c_uint32
        L.mxq_bias_stats.argtypes = [C.POINTER(QConfig), P, i64, i64, i64, i32, C.POINTER(QTensor),
                                     P, P, C.c_size_t, P]
        L.mxq_bias_stats_noalloc.argtypes = [C.POINTER(QConfig), P, i64, i64, i64, i32,
                                             C.POINTER(QTensor), P, P]
        L.mxq_bias_stats_workspace_size.argtypes = [i64, i64, i32]
        L.mxq_bias_stats_workspace_size.restype = C.c_size_t
        L.mxq_round_to_grid.argtypes = [i32, i32, i32, P, P, i64, P, P]
        L.mxq_bucket_ratio.argtypes = [C.POINTER(Stats), i32]
        L.mxq_bucket_ratio.restype = C.c_double
        sz, f32 = C.c_size_t, C.c_float
        L.mxq_norm_forward.argtypes = [i32, P, i32, i64, i64, i64, P, P, f32, P, i32, i64, P, P, P]
        L.mxq_norm_backward.argtypes = [i32, P, i32, i64, P, i32, i64, i64, i64, P, P, P, P, i32,
                                        i64, P, P, P, sz, P]
        L.mxq_norm_backward_workspace_size.argtypes = [i64, i64]
        L.mxq_norm_backward_workspace_size.restype = sz
        logits = [P, i32, i64, i64, i64, f32]
        teacher = [P, P, i32, i32, P]
        L.mxq_token_logprobs.argtypes = logits + [P, P, P, P, i32, P, P, P, sz, P]
        L.mxq_token_logprobs_backward.argtypes = logits + [P, P, P, P, P, P, i32, i64, P]
        L.mxq_vocab_workspace_size.argtypes = [i64, i64, i32]
        L.mxq_vocab_workspace_size.restype = sz
        L.mxq_distill_forward.argtypes = logits + teacher + [P, P, P, sz, P]
        L.mxq_distill_backward.argtypes = logits + teacher + [P, P, i32, i64, P]
        L.mxq_distill.argtypes = logits + teacher + [P, P, i32, i64, P, sz, P]
        head = [P, i64, P, i64, i64, i64, i64, f32, P, P]
        L.mxq_linear_ce_forward.argtypes = head + [P, P, P, sz, P]
        L.mxq_linear_ce_backward.argtypes = head + [P, P, i64, P, i64, P, sz, P]
        for name in ("mxq_linear_ce_forward_workspace_size", "mxq_linear_ce_backward_workspace_size"):
            getattr(L, name).argtypes = [i64, i64, i64]
            getattr(L, name).restype = sz
        L.mxq_grad_norm.argtypes = [C.POINTER(Grad), i64, P, P, P, sz, P]
        L.mxq_grad_norm_workspace_size.argtypes = [C.POINTER(Grad), i64]
        L.mxq_grad_norm_workspace_size.restype = sz
        L.mxq_grad_clip.argtypes = [C.POINTER(Grad), i64, P, f32, f32, P]
        L.mxq_status_string.argtypes = [i32]
        L.mxq_status_string.restype = C.c_char_p
        L.mxq_abi_version.restype = i32
        for name in ("mxq_quantize", "mxq_quantize_batch", "mxq_dequantize", "mxq_wgrad_gemm", "mxq_gemm_abt",
                     "mxq_bias_stats", "mxq_bias_stats_noalloc", "mxq_round_to_grid", "mxq_rotate",
                     "mxq_norm_forward", "mxq_norm_backward", "mxq_token_logprobs",
                     "mxq_token_logprobs_backward", "mxq_distill_forward", "mxq_distill_backward",
                     "mxq_distill", "mxq_linear_ce_forward", "mxq_linear_ce_backward",
                     "mxq_grad_norm", "mxq_grad_clip"):
            getattr(L, name).restype = i32
        _lib = L
    return _lib


def status_string(status: int) -> str:
    return lib().mxq_status_string(status).decode()


def _check(fn: str, status: int):
    if status != OK:
        raise MxqError(fn, status)


def _ptr(t) -> int | None:
    return None if t is None else t.data_ptr()


def _stream(stream=None):
    import torch
    s = torch.cuda.current_stream() if stream is None else stream
    return C.c_void_p(s.cuda_stream)


def qconfig(grid=GRID_E2M1, round=RTNE, hadamard_n=0, sign_mask=0, sr_seed=0, sr_stream=0,
            sr_bits=16, sign_mode=SIGNS_MASK, sign_seed=0) -> QConfig:
    return QConfig(grid, round, hadamard_n, sign_mask & 0xFFFFFFFF, sr_seed, sr_stream, sr_bits,
                   sign_mode, 0, sign_seed)


def block_bytes(fmt: int) -> int:
    return 16 if fmt == FMT_FP4 else 24


def qtensor_sizes(lines: int, k: int, fmt: int, layout: int = LAYOUT_ROWS):
    """(code bytes, scale bytes) of a [lines x k] block-quantized tensor."""
    nb = k // 32
    if layout == LAYOUT_ROWS:
        return lines * nb * block_bytes(fmt), lines * nb
    ntiles = (lines + 15) // 16
    nsteps = k // 128
    return nsteps * ntiles * 64 * block_bytes(fmt), ((nsteps + 3) // 4) * ntiles * 256


def empty_qtensor(lines: int, k: int, fmt: int, device, layout: int = LAYOUT_ROWS, fill=None):
    """Device buffers (codes, scales): 2-D [lines, ...] for the row layout,
    1-D byte arrays for the MFMA layout."""
    import torch
    nb = k // 32
    if layout == LAYOUT_ROWS:
        codes = torch.empty((lines, nb * block_bytes(fmt)), dtype=torch.uint8, device=device)
        scales = torch.empty((lines, nb), dtype=torch.uint8, device=device)
    else:
        cb, sb = qtensor_sizes(lines, k, fmt, layout)
        codes = torch.empty(cb, dtype=torch.uint8, device=device)
        scales = torch.empty(sb, dtype=torch.uint8, device=device)
    if fill is not None:
        codes.fill_(fill)
        scales.fill_(fill)
    return codes, scales


def qtensor(codes, scales, fmt: int, grid: int, layout: int = LAYOUT_ROWS) -> QTensor:
    return QTensor(codes.data_ptr(), scales.data_ptr(), fmt, grid, layout)


# ---- entry points ---------------------------------------------------------

def quantize_into(cfg: QConfig, x, row=None, col=None, rows=None, cols=None, ld=None,
                  stream=None):
    """mxq_quantize on caller-owned buffers.
    row/col: (codes, scales, fmt) or (codes, scales, fmt, layout), or None."""
    rows = x.shape[0] if rows is None else rows
    cols = x.shape[1] if cols is None else cols
    ld = x.stride(0) if ld is None else ld

    def desc(o):
        if not o:
            return None
        lay = o[3] if len(o) > 3 else LAYOUT_ROWS
        return QTensor(o[0].data_ptr(), o[1].data_ptr(), o[2], cfg.grid, lay)
    rt, ct = desc(row), desc(col)
    st = lib().mxq_quantize(C.byref(cfg), _ptr(x), rows, cols, ld,
                            C.byref(rt) if rt else None, C.byref(ct) if ct else None,
                            _stream(stream))
    _check("mxq_quantize", st)


def prepare_quantize(cfg: QConfig, x, row=None, col=None, stream=None):
    """The call quantize_into(cfg, x, row, col) marshalled once: returns a
    function of no arguments that launches it again on the same buffers (for
    timing loops, where per-call argument conversion would leave the GPU
    waiting on the host).  The function holds every tensor it was given, so
    their memory cannot be freed and handed to another tensor while it can
    still launch."""
    rows, cols, ld = x.shape[0], x.shape[1], x.stride(0)

    def desc(o):
        if not o:
            return None
        lay = o[3] if len(o) > 3 else LAYOUT_ROWS
        return QTensor(o[0].data_ptr(), o[1].data_ptr(), o[2], cfg.grid, lay)
    rt, ct = desc(row), desc(col)
    cfg_ = QConfig.from_buffer_copy(cfg)
    args = (C.byref(cfg_), _ptr(x), rows, cols, ld, C.byref(rt) if rt else None,
            C.byref(ct) if ct else None, _stream(stream))
    fn = lib().mxq_quantize
    keep = (cfg_, rt, ct, x, row, col)

    def call():
        _check("mxq_quantize", fn(*args))
    call._keep = keep
    return call


def _addr(t) -> int:
    """Device address of t; an empty view keeps the address of its storage
    (torch reports 0 for tensors without elements)."""
    p = t.data_ptr()
    if p == 0 and t.numel() == 0:
        p = t.untyped_storage().data_ptr() + t.storage_offset() * t.element_size()
    return p


def _batch_args(jobs):
    """ctypes array of QuantizeJob for [(cfg, x, row, col), ...] (row / col as
    in quantize_into) and the objects it points into."""
    arr = (QuantizeJob * len(jobs))()
    keep = [arr]
    for i, (cfg, x, row, col) in enumerate(jobs):
        cfg_ = QConfig.from_buffer_copy(cfg)

        def desc(o):
            if not o:
                return None
            lay = o[3] if len(o) > 3 else LAYOUT_ROWS
            return QTensor(o[0].data_ptr(), o[1].data_ptr(), o[2], cfg_.grid, lay)
        rt, ct = desc(row), desc(col)
        keep += [cfg_, rt, ct, x, row, col]
        arr[i] = QuantizeJob(C.pointer(cfg_), _addr(x), x.shape[0], x.shape[1], x.stride(0),
                             C.pointer(rt) if rt else None, C.pointer(ct) if ct else None)
    return arr, keep


def quantize_batch(jobs, stream=None):
    """mxq_quantize_batch: jobs = [(cfg, x, row, col), ...] with row / col
    (codes, scales, fmt[, layout]) or None, as quantize_into."""
    arr, keep = _batch_args(jobs)
    st = lib().mxq_quantize_batch(arr, len(jobs), _stream(stream))
    del keep
    _check("mxq_quantize_batch", st)


def prepare_quantize_batch(jobs, stream=None):
    """quantize_batch(jobs) marshalled once (see prepare_quantize; the function
    holds every job's tensors)."""
    arr, keep = _batch_args(jobs)
    args = (arr, len(jobs), _stream(stream))
    fn = lib().mxq_quantize_batch

    def call():
        _check("mxq_quantize_batch", fn(*args))
    call._keep = keep
    return call


def quantize(x, grid=GRID_E2M1, round=RTNE, hadamard_n=0, sign_mask=0, sr_seed=0, sr_stream=0,
             sr_bits=16, row=True, col=False, row_fmt=FMT_FP4, col_fmt=FMT_FP4,
             row_layout=LAYOUT_ROWS, col_layout=LAYOUT_ROWS, fill=None, stream=None,
             sign_mode=SIGNS_MASK, sign_seed=0):
    """Quantize a 2-D bf16 CUDA tensor; returns {'row': (codes, scales), 'col': (...)}."""
    cfg = qconfig(grid, round, hadamard_n, sign_mask, sr_seed, sr_stream, sr_bits, sign_mode,
                  sign_seed)
    rows, cols = x.shape
    out = {}
    r = c = None
    if row:
        rc, rs = empty_qtensor(rows, cols, row_fmt, x.device, row_layout, fill)
        r = (rc, rs, row_fmt, row_layout)
        out["row"] = (rc, rs)
    if col:
        cc, cs = empty_qtensor(cols, rows, col_fmt, x.device, col_layout, fill)
        c = (cc, cs, col_fmt, col_layout)
        out["col"] = (cc, cs)
    quantize_into(cfg, x, r, c, stream=stream)
    return out


def dequantize(codes, scales, fmt: int, grid: int, out_dtype=OUT_F32, layout=LAYOUT_ROWS,
               lines=None, k=None, stream=None):
    import torch
    if layout == LAYOUT_ROWS:
        lines = scales.shape[0] if lines is None else lines
        k = scales.shape[1] * 32 if k is None else k
    dt = torch.float32 if out_dtype == OUT_F32 else torch.bfloat16
    out = torch.empty((lines, k), dtype=dt, device=codes.device)
    q = qtensor(codes, scales, fmt, grid, layout)
    _check("mxq_dequantize", lib().mxq_dequantize(C.byref(q), lines, k, out_dtype, _ptr(out), k,
                                                  _stream(stream)))
    return out


def wgrad_gemm(a_codes, a_scales, a_fmt, a_grid, b_codes, b_scales, b_fmt, b_grid, out=None,
               layout=LAYOUT_ROWS, m=None, n=None, k=None, stream=None):
    """C [m x n] fp32 = A [m x k] B [n x k]^T on block-quantized operands (both
    in `layout`; m, n, k are required for the MFMA layout)."""
    import torch
    if layout == LAYOUT_ROWS:
        m = a_scales.shape[0] if m is None else m
        n = b_scales.shape[0] if n is None else n
        k = a_scales.shape[1] * 32 if k is None else k
        assert b_scales.shape[1] * 32 == k
    c = torch.empty((m, n), dtype=torch.float32, device=a_codes.device) if out is None else out
    qa = qtensor(a_codes, a_scales, a_fmt, a_grid, layout)
    qb = qtensor(b_codes, b_scales, b_fmt, b_grid, layout)
    _check("mxq_wgrad_gemm", lib().mxq_wgrad_gemm(C.byref(qa), C.byref(qb), m, n, k, _ptr(c),
                                                  c.stride(0), _stream(stream)))
    return c


def prepare_wgrad_gemm(a_codes, a_scales, a_fmt, a_grid, b_codes, b_scales, b_fmt, b_grid, out,
                       layout, m, n, k, stream=None, entry="mxq_wgrad_gemm"):
    """wgrad_gemm(...) marshalled once into a function of no arguments
    (entry="mxq_gemm_abt" for the same product under its general name) that
    holds every tensor it was given."""
    qa = qtensor(a_codes, a_scales, a_fmt, a_grid, layout)
    qb = qtensor(b_codes, b_scales, b_fmt, b_grid, layout)
    args = (C.byref(qa), C.byref(qb), m, n, k, _ptr(out), out.stride(0), _stream(stream))
    fn = getattr(lib(), entry)

    def call():
        _check(entry, fn(*args))
    call._keep = (qa, qb, a_codes, a_scales, b_codes, b_scales, out)
    return call


def gemm_abt(a_codes, a_scales, a_fmt, a_grid, b_codes, b_scales, b_fmt, b_grid, out=None,
             layout=LAYOUT_ROWS, m=None, n=None, k=None, stream=None):
    """C [m x n] fp32 = A [m x k] B [n x k]^T through mxq_gemm_abt: Fprop
    (X row-wise, W row-wise), Dgrad (dY row-wise, W column-wise) or Wgrad
    (dY column-wise, X column-wise)."""
    import torch
    if layout == LAYOUT_ROWS:
        m = a_scales.shape[0] if m is None else m
        n = b_scales.shape[0] if n is None else n
        k = a_scales.shape[1] * 32 if k is None else k
    c = torch.empty((m, n), dtype=torch.float32, device=a_codes.device) if out is None else out
    qa = qtensor(a_codes, a_scales, a_fmt, a_grid, layout)
    qb = qtensor(b_codes, b_scales, b_fmt, b_grid, layout)
    _check("mxq_gemm_abt", lib().mxq_gemm_abt(C.byref(qa), C.byref(qb), m, n, k, _ptr(c),
                                              c.stride(0), _stream(stream)))
    return c


def rotate(x, axis: int, hadamard_n: int, sign_mask: int = 0, out_dtype=OUT_F32, out=None,
           stream=None, sign_mode=SIGNS_MASK, sign_seed=0):
    """The block rotation alone, in x's orientation (fp32 or bf16 out)."""
    import torch
    dt = torch.float32 if out_dtype == OUT_F32 else torch.bfloat16
    o = torch.empty(x.shape, dtype=dt, device=x.device) if out is None else out
    cfg = qconfig(hadamard_n=hadamard_n, sign_mask=sign_mask, sign_mode=sign_mode,
                  sign_seed=sign_seed)
    _check("mxq_rotate", lib().mxq_rotate(C.byref(cfg), _ptr(x), x.shape[0], x.shape[1],
                                          x.stride(0), axis, out_dtype, _ptr(o), o.stride(0),
                                          _stream(stream)))
    return o


def prepare_rotate(x, axis: int, hadamard_n: int, sign_mask: int, out_dtype, out, stream=None):
    """rotate(...) marshalled once into a function of no arguments that holds
    x and out."""
    cfg = qconfig(hadamard_n=hadamard_n, sign_mask=sign_mask)
    args = (C.byref(cfg), _ptr(x), x.shape[0], x.shape[1], x.stride(0), axis, out_dtype, _ptr(out),
            out.stride(0), _stream(stream))
    fn = lib().mxq_rotate

    def call():
        _check("mxq_rotate", fn(*args))
    call._keep = (cfg, x, out)
    return call


def rht_sign_mask(seed: int, n: int) -> int:
    """Sign mask of the randomized Hadamard rotation drawn from `seed` (host)."""
    return int(lib().mxq_rht_sign_mask(seed, n))


def bias_stats(x, axis: int, codes, scales, fmt: int, grid=GRID_E2M1, round=RTNE, hadamard_n=0,
               sign_mask=0, sr_seed=0, sr_stream=0, sr_bits=16, stream=None,
               sign_mode=SIGNS_MASK, sign_seed=0) -> dict:
    import torch
    cfg = qconfig(grid, round, hadamard_n, sign_mask, sr_seed, sr_stream, sr_bits, sign_mode,
                  sign_seed)
    rows, cols = x.shape
    wsb = lib().mxq_bias_stats_workspace_size(rows, cols, axis)
    ws = torch.empty(max(wsb, 8), dtype=torch.uint8, device=x.device)
    out = torch.zeros(C.sizeof(Stats), dtype=torch.uint8, device=x.device)
    q = qtensor(codes, scales, fmt, grid)
    _check("mxq_bias_stats", lib().mxq_bias_stats(C.byref(cfg), _ptr(x), rows, cols, x.stride(0),
                                                  axis, C.byref(q), _ptr(out), _ptr(ws), wsb,
                                                  _stream(stream)))
    return _stats_dict(out)


def prepare_bias_stats(x, axis: int, codes, scales, fmt: int, out, ws, grid=GRID_E2M1,
                       round=RTNE, hadamard_n=0, sign_mask=0, sr_seed=0, sr_stream=0,
                       sr_bits=16, stream=None, sign_mode=SIGNS_MASK, sign_seed=0):
    """bias_stats(...) marshalled once into a function of no arguments that
    holds every tensor it was given: `out` is a device byte tensor of
    sizeof(mxq_stats), `ws` one of at least mxq_bias_stats_workspace_size
    bytes.  The call leaves the statistics in `out` (no host copy)."""
    cfg = qconfig(grid, round, hadamard_n, sign_mask, sr_seed, sr_stream, sr_bits, sign_mode,
                  sign_seed)
    rows, cols = x.shape
    q = qtensor(codes, scales, fmt, grid)
    args = (C.byref(cfg), _ptr(x), rows, cols, x.stride(0), axis, C.byref(q), _ptr(out),
            _ptr(ws), ws.numel(), _stream(stream))
    fn = lib().mxq_bias_stats

    def call():
        _check("mxq_bias_stats", fn(*args))
    call._keep = (cfg, q, x, codes, scales, out, ws)
    return call


def _stats_dict(out) -> dict:
    """The mxq_stats a call wrote into the device byte tensor `out`."""
    st = Stats.from_buffer_copy(bytes(out.cpu().numpy().tobytes()))
    d = {k: getattr(st, k) for k, _ in Stats._fields_}
    d["level_err_norm"] = list(st.level_err_norm)
    d["level_count"] = list(st.level_count)
    return d


def bias_stats_noalloc(x, axis: int, codes, scales, fmt: int, out=None, grid=GRID_E2M1, round=RTNE,
                       hadamard_n=0, sign_mask=0, sr_seed=0, sr_stream=0, sr_bits=16, stream=None,
                       sign_mode=SIGNS_MASK, sign_seed=0, raw=False):
    """mxq_bias_stats_noalloc into `out` (a device byte tensor of sizeof(mxq_stats),
    allocated here when not given); returns the stats dict, or `out` itself
    when raw=True (no host copy)."""
    import torch
    cfg = qconfig(grid, round, hadamard_n, sign_mask, sr_seed, sr_stream, sr_bits, sign_mode,
                  sign_seed)
    rows, cols = x.shape
    if out is None:
        out = torch.zeros(C.sizeof(Stats), dtype=torch.uint8, device=x.device)
    q = qtensor(codes, scales, fmt, grid)
    _check("mxq_bias_stats_noalloc",
           lib().mxq_bias_stats_noalloc(C.byref(cfg), _ptr(x), rows, cols, x.stride(0), axis,
                                        C.byref(q), _ptr(out), _stream(stream)))
    return out if raw else _stats_dict(out)


def bucket_ratio(level_count, grid: int) -> float:
    """mxq_bucket_ratio on a histogram of magnitude codes (8 counts)."""
    st = Stats()
    for m, c in enumerate(level_count[:8]):
        st.level_count[m] = int(c)
    return float(lib().mxq_bucket_ratio(C.byref(st), grid))


def round_to_grid(a, grid: int, round=RTNE, rand=None, sr_bits=16, out=None, stream=None):
    """Nibble of each fp32 value of `a` (already divided by its block scale)."""
    import torch
    n = a.numel()
    codes = torch.empty(n, dtype=torch.uint8, device=a.device) if out is None else out
    _check("mxq_round_to_grid", lib().mxq_round_to_grid(grid, round, sr_bits, _ptr(a), _ptr(rand),
                                                        n, _ptr(codes), _stream(stream)))
    return codes


# ---- the operators around the products --------------------------------------
# These take tensors of their own types and strides, so the binding checks what
# the C entry points cannot see: a wrong element type, a stride along the row,
# a vector of another length or a tensor elsewhere raises a ValueError.

_DTYPES = None


def _dtype(t) -> int:
    """MXQ_OUT_* of a tensor or torch dtype."""
    global _DTYPES
    if _DTYPES is None:
        import torch
        _DTYPES = {torch.float32: OUT_F32, torch.bfloat16: OUT_BF16}
    code = _DTYPES.get(getattr(t, "dtype", t))
    if code is None:
        raise ValueError(f"float32 or bfloat16 expected, not {getattr(t, 'dtype', t)}")
    return code


def _matrix(name, t, like=None):
    """(address, dtype code, leading dimension) of a 2-D tensor whose rows are contiguous."""
    code = _dtype(t)
    if t.dim() != 2 or (like is not None and t.shape != like.shape):
        raise ValueError(f"{name}: shape {tuple(t.shape)}" + (f", not {tuple(like.shape)}" if like is not None else " is not 2-D"))
    rows, cols = t.shape
    ld, inner = t.stride()
    if (cols > 1 and inner != 1) or (rows > 1 and ld < cols):
        raise ValueError(f"{name}: rows must be contiguous and apart (strides {t.stride()})")
    if like is not None and t.device != like.device:
        raise ValueError(f"{name}: on {t.device}, not {like.device}")
    return t.data_ptr(), code, ld if rows > 1 else max(ld, cols)


def _vector(name, t, shape, like, dtype=None):
    """Address of a packed fp32 (or `dtype`) tensor of this shape, None for None."""
    if t is None:
        return None
    if dtype is None:
        import torch
        dtype = torch.float32
    if t.dtype != dtype or t.shape != shape or not t.is_contiguous() or t.device != like.device:
        raise ValueError(f"{name}: packed {dtype} of shape {shape} on {like.device} expected, "
                         f"not {t.dtype} {tuple(t.shape)} strides {t.stride()} on {t.device}")
    return t.data_ptr()


_torch = None


def _enter(x, stream):
    """(torch, handle of the call's stream) for a call on x's device."""
    global _torch
    if _torch is None:
        import torch
        _torch = torch
    index = x.get_device()
    if index < 0:
        raise ValueError("GPU tensors expected")
    if index != _torch.cuda.current_device():
        raise ValueError(f"the tensors are on cuda:{index}, the current device is cuda:{_torch.cuda.current_device()}")
    return _torch, _torch._C._cuda_getCurrentRawStream(index) if stream is None else stream.cuda_stream


def _new(x, shape, dtype, stream):
    """A packed tensor on x's device, allocated on the stream that uses it, so
    that its memory is not handed on early."""
    if stream is None:
        return x.new_empty(shape, dtype=dtype)
    with _torch.cuda.stream(stream):
        return x.new_empty(shape, dtype=dtype)


def norm_forward(x, gamma=None, beta=None, *, eps, kind=NORM_LAYER, out_dtype=None, out=None, stream=None):
    """mxq_norm_forward: (y, mean, rstd); mean is None for NORM_RMS.  y has x's
    dtype unless out_dtype says otherwise, or is `out` (x itself serves)."""
    torch, handle = _enter(x, stream)
    f32 = torch.float32
    rows, cols = x.shape
    y = _new(x, (rows, cols), out_dtype or x.dtype, stream) if out is None else out
    xp, xt, ldx = _matrix("x", x)
    yp, yt, ldy = _matrix("out", y, x)
    mean = _new(x, (rows,), f32, stream) if kind == NORM_LAYER else None
    rstd = _new(x, (rows,), f32, stream)
    _check("mxq_norm_forward", lib().mxq_norm_forward(
        kind, xp, xt, ldx, rows, cols, _vector("gamma", gamma, (cols,), x),
        _vector("beta", beta, (cols,), x), eps, yp, yt, ldy, _ptr(mean), _ptr(rstd), handle))
    return y, mean, rstd


def norm_backward(dy, x, gamma, mean, rstd, *, kind=NORM_LAYER, weight=True, bias=True, out_dtype=None,
                  out=None, stream=None):
    """mxq_norm_backward: (dx, dgamma, dbeta); dgamma without `weight` and dbeta
    without `bias` are None.  dx has x's dtype unless out_dtype says otherwise,
    or is `out` (dy or x itself serves)."""
    torch, handle = _enter(x, stream)
    f32 = torch.float32
    rows, cols = x.shape
    dx = _new(x, (rows, cols), out_dtype or x.dtype, stream) if out is None else out
    xp, xt, ldx = _matrix("x", x)
    dp, dt, ldd = _matrix("dy", dy, x)
    op, ot, ldo = _matrix("out", dx, x)
    dgamma = _new(x, (cols,), f32, stream) if weight else None
    dbeta = _new(x, (cols,), f32, stream) if bias else None
    size = lib().mxq_norm_backward_workspace_size(rows, cols) if weight or bias else 0
    ws = _new(x, (size,), torch.uint8, stream) if size else None
    _check("mxq_norm_backward", lib().mxq_norm_backward(
        kind, dp, dt, ldd, xp, xt, ldx, rows, cols, _vector("gamma", gamma, (cols,), x),
        _vector("mean", mean if kind == NORM_LAYER else None, (rows,), x),
        _vector("rstd", rstd, (rows,), x), op, ot, ldo, _ptr(dgamma), _ptr(dbeta), _ptr(ws), size,
        handle))
    return dx, dgamma, dbeta


def token_logprobs(logits, tokens=None, *, top_k=0, temperature=1, entropy=True, stream=None):
    """mxq_token_logprobs: [logprob, entropy, stats], and top_ids, top_logprobs
    after them where top_k > 0; logprob is None without tokens (int32), entropy
    where it is not asked for."""
    torch, handle = _enter(logits, stream)
    f32, i32 = torch.float32, torch.int32
    rows, vocab = logits.shape
    zp, zt, ld = _matrix("logits", logits)
    out = [_new(logits, (rows,), f32, stream) if tokens is not None else None,
           _new(logits, (rows,), f32, stream) if entropy else None, _new(logits, (rows, 2), f32, stream)]
    ids = lps = None
    if top_k > 0:
        ids, lps = _new(logits, (rows, top_k), i32, stream), _new(logits, (rows, top_k), f32, stream)
    size = lib().mxq_vocab_workspace_size(rows, vocab, top_k)
    ws = _new(logits, (size,), torch.uint8, stream) if size else None
    _check("mxq_token_logprobs", lib().mxq_token_logprobs(
        zp, zt, ld, rows, vocab, temperature, _vector("tokens", tokens, (rows,), logits, i32),
        _ptr(out[0]), _ptr(out[1]), _ptr(out[2]), top_k, _ptr(ids), _ptr(lps), _ptr(ws), size, handle))
    return out + [ids, lps] if top_k > 0 else out


def token_logprobs_backward(logits, tokens, stats, entropy=None, d_logprob=None, d_entropy=None, *,
                            temperature=1, out_dtype=None, out=None, stream=None):
    """mxq_token_logprobs_backward: the gradient of the logits, in their dtype
    unless out_dtype says otherwise, or in `out` (the logits themselves serve)."""
    torch, handle = _enter(logits, stream)
    rows, vocab = logits.shape
    o = _new(logits, (rows, vocab), out_dtype or logits.dtype, stream) if out is None else out
    zp, zt, ld = _matrix("logits", logits)
    op, ot, ldo = _matrix("out", o, logits)
    _check("mxq_token_logprobs_backward", lib().mxq_token_logprobs_backward(
        zp, zt, ld, rows, vocab, temperature,
        _vector("tokens", tokens, (rows,), logits, torch.int32),
        _vector("stats", stats, (rows, 2), logits), _vector("entropy", entropy, (rows,), logits),
        _vector("d_logprob", d_logprob, (rows,), logits),
        _vector("d_entropy", d_entropy, (rows,), logits), op, ot, ldo, handle))
    return o


def _teacher_args(logits, ids, logprobs, weight, renormalize):
    rows, top_k = logits.shape[0], ids.shape[-1]
    return (_vector("teacher_ids", ids, (rows, top_k), logits, _torch.int32),
            _vector("teacher_logprobs", logprobs, (rows, top_k), logits), top_k,
            1 if renormalize else 0, _vector("weight", weight, (rows,), logits))


def distill_forward(logits, teacher_ids, teacher_logprobs, weight=None, *, temperature=1,
                    renormalize=True, stream=None):
    """mxq_distill_forward: (loss, stats)."""
    torch, handle = _enter(logits, stream)
    rows, vocab = logits.shape
    zp, zt, ld = _matrix("logits", logits)
    loss, stats = _new(logits, (rows,), torch.float32, stream), _new(logits, (rows, 2), torch.float32, stream)
    size = lib().mxq_vocab_workspace_size(rows, vocab, 0)
    ws = _new(logits, (size,), torch.uint8, stream) if size else None
    _check("mxq_distill_forward", lib().mxq_distill_forward(
        zp, zt, ld, rows, vocab, temperature,
        *_teacher_args(logits, teacher_ids, teacher_logprobs, weight, renormalize),
        _ptr(loss), _ptr(stats), _ptr(ws), size, handle))
    return loss, stats


def distill_backward(logits, teacher_ids, teacher_logprobs, stats, weight=None, *, temperature=1,
                     renormalize=True, out_dtype=None, out=None, stream=None):
    """mxq_distill_backward: the gradient of the logits, in their dtype unless
    out_dtype says otherwise, or in `out` (the logits themselves serve)."""
    torch, handle = _enter(logits, stream)
    rows, vocab = logits.shape
    o = _new(logits, (rows, vocab), out_dtype or logits.dtype, stream) if out is None else out
    zp, zt, ld = _matrix("logits", logits)
    op, ot, ldo = _matrix("out", o, logits)
    _check("mxq_distill_backward", lib().mxq_distill_backward(
        zp, zt, ld, rows, vocab, temperature,
        *_teacher_args(logits, teacher_ids, teacher_logprobs, weight, renormalize),
        _vector("stats", stats, (rows, 2), logits), op, ot, ldo, handle))
    return o


def distill(logits, teacher_ids, teacher_logprobs, weight=None, *, temperature=1, renormalize=True,
            out_dtype=None, out=None, stream=None):
    """mxq_distill: (loss, gradient of the logits) in one pass; the gradient as
    in distill_backward."""
    torch, handle = _enter(logits, stream)
    rows, vocab = logits.shape
    o = _new(logits, (rows, vocab), out_dtype or logits.dtype, stream) if out is None else out
    zp, zt, ld = _matrix("logits", logits)
    op, ot, ldo = _matrix("out", o, logits)
    loss = _new(logits, (rows,), torch.float32, stream)
    size = lib().mxq_vocab_workspace_size(rows, vocab, 0)
    ws = _new(logits, (size,), torch.uint8, stream) if size else None
    _check("mxq_distill", lib().mxq_distill(
        zp, zt, ld, rows, vocab, temperature,
        *_teacher_args(logits, teacher_ids, teacher_logprobs, weight, renormalize),
        _ptr(loss), op, ot, ldo, _ptr(ws), size, handle))
    return loss, o


# ---- the ends of a training step ---------------------------------------------

def _bf16(name, t, shape, like):
    """(address, leading dimension) of a 2-D bf16 tensor of this shape whose rows are contiguous."""
    p, code, ld = _matrix(name, t)
    if code != OUT_BF16 or tuple(t.shape) != tuple(shape) or t.device != like.device:
        raise ValueError(f"{name}: bfloat16 of shape {tuple(shape)} on {like.device} expected, "
                         f"not {t.dtype} {tuple(t.shape)} on {t.device}")
    return p, ld


def _rows_of(t):
    """(address, bytes between rows, bytes of a row, rows) of a matrix whose rows are contiguous, or a packed vector."""
    size = t.element_size()
    if t.dim() == 2 and t.shape[0] > 1 and not t.is_contiguous():
        return t.data_ptr(), t.stride(0) * size, t.shape[1] * size, t.shape[0]
    return t.data_ptr(), t.numel() * size, t.numel() * size, 1


def _share(a, b) -> bool:
    """Whether two such tensors have a byte in common; interleaved columns of one buffer have none."""
    if a.numel() == 0 or b.numel() == 0:
        return False
    (p, ld_p, wide_p, rows_p), (q, ld_q, wide_q, rows_q) = sorted((_rows_of(a), _rows_of(b)), key=lambda r: r[3])
    if p + (rows_p - 1) * ld_p + wide_p <= q or q + (rows_q - 1) * ld_q + wide_q <= p:
        return False
    if ld_p == ld_q:
        between, (first, second) = abs(q - p) % ld_p, (wide_p, wide_q) if p <= q else (wide_q, wide_p)
        return between < first or between + second > ld_p
    for at in range(p, p + rows_p * ld_p, ld_p):
        # the first of the other's rows that ends behind this one's start
        row = max(0, (at - q - wide_q) // ld_q + 1)
        if row < rows_q and q + row * ld_q < at + wide_p:
            return True
    return False


def _refuse_shared(**tensors):
    """Refuses an output (dx, dw) that shares memory with another tensor of the call."""
    for name in ("dx", "dw"):
        for other, t in tensors.items():
            if other != name and tensors[name] is not None and t is not None and _share(tensors[name], t):
                raise ValueError(f"{name}: in the same memory as {other}")


def linear_ce_forward(x, w, targets, weight=None, *, temperature=1, stream=None):
    """mxq_linear_ce_forward: (loss, stats) of the output layer with weight w
    [vocab, hidden] on the hidden states x [rows, hidden]."""
    torch, handle = _enter(x, stream)
    (rows, hidden), vocab = x.shape, w.shape[0]
    xp, ldx = _bf16("x", x, (rows, hidden), x)
    wp, ldw = _bf16("w", w, (vocab, hidden), x)
    loss, stats = _new(x, (rows,), torch.float32, stream), _new(x, (rows, 2), torch.float32, stream)
    size = lib().mxq_linear_ce_forward_workspace_size(rows, hidden, vocab)
    ws = _new(x, (size,), torch.uint8, stream) if size else None
    _check("mxq_linear_ce_forward", lib().mxq_linear_ce_forward(
        xp, ldx, wp, ldw, rows, hidden, vocab, temperature,
        _vector("targets", targets, (rows,), x, torch.int32), _vector("weight", weight, (rows,), x),
        _ptr(loss), _ptr(stats), _ptr(ws), size, handle))
    return loss, stats


def linear_ce_backward(x, w, targets, stats, weight=None, *, temperature=1, dx=True, dw=True, stream=None):
    """mxq_linear_ce_backward: (dx, dw), new tensors for True, None for False; a
    tensor takes the gradient itself, and shares memory with no other one."""
    torch, handle = _enter(x, stream)
    (rows, hidden), vocab = x.shape, w.shape[0]
    xp, ldx = _bf16("x", x, (rows, hidden), x)
    wp, ldw = _bf16("w", w, (vocab, hidden), x)

    def gradient(name, given, shape):
        if given is False or given is None:
            return None, None, 0
        t = _new(x, shape, torch.bfloat16, stream) if given is True else given
        return (t, *_bf16(name, t, shape, x))
    own = any(torch.is_tensor(t) for t in (dx, dw))
    dx, dxp, lddx = gradient("dx", dx, (rows, hidden))
    dw, dwp, lddw = gradient("dw", dw, (vocab, hidden))
    if own:
        _refuse_shared(dx=dx, dw=dw, x=x, w=w, targets=targets, stats=stats, weight=weight)
    size = lib().mxq_linear_ce_backward_workspace_size(rows, hidden, vocab)
    ws = _new(x, (size,), torch.uint8, stream) if size else None
    _check("mxq_linear_ce_backward", lib().mxq_linear_ce_backward(
        xp, ldx, wp, ldw, rows, hidden, vocab, temperature,
        _vector("targets", targets, (rows,), x, torch.int32), _vector("weight", weight, (rows,), x),
        _vector("stats", stats, (rows, 2), x), dxp, lddx, dwp, lddw, _ptr(ws), size, handle))
    return dx, dw


def _dense(t) -> bool:
    """Whether t's elements lie side by side, each once, in whatever order of its dimensions."""
    if t.is_contiguous():
        return True
    at = 1
    for stride, size in sorted((stride, size) for stride, size in zip(t.stride(), t.shape) if size != 1):
        if stride != at:
            return False
        at *= size
    return True


def _same_order(a, b) -> bool:
    """Whether two dense tensors of one shape have their elements in the same order: strides count where
    there is a step to take."""
    return a.numel() == 0 or all(s == t for s, t, size in zip(a.stride(), b.stride(), a.shape) if size > 1)


def _refuse_overlaps(spans):
    """Refuses an output that shares memory with another tensor of the list, or with a part of its own gradient.
    spans: (first byte, end, whether it is written, place in the list)."""
    def name(write, i):
        return f"{'output' if write else 'gradient'} {i}"
    read = written = (0, 0, False, 0)    # of the spans so far, those that end last
    for span in sorted(spans):
        at, end, write, i = span
        other = read if write and read[1] > written[1] else written
        if at < other[1]:
            one, two = (name(write, i), name(*other[2:]))[::1 if write else -1]
            raise ValueError(f"{one}: in the same memory as {two}")
        if write:
            written = max(written, span, key=lambda s: s[1])
        elif end > read[1]:
            read = span


def _grad_list(grads, out=None, write=True):
    """The mxq_grad array of a list of tensors (written in place, or to the list `out`), and what it points into."""
    grads = list(grads)
    out = grads if out is None else list(out)
    if not grads:
        raise ValueError("no gradients: the device is theirs")
    if len(out) != len(grads):
        raise ValueError(f"{len(out)} outputs for {len(grads)} gradients")
    device, spans = grads[0].device, []
    arr = (Grad * len(grads))()

    def seen(name, i, t):
        if t.device != device or not _dense(t):
            raise ValueError(f"{name} {i}: a dense tensor on {device} expected, not strides {t.stride()} on {t.device}")
        return t.data_ptr(), _dtype(t)
    for i, (g, o) in enumerate(zip(grads, out)):
        at, code = to, to_code = seen("gradient", i, g)
        n = g.numel()
        if o is not g:
            to, to_code = seen("output", i, o)
            if o.shape != g.shape or (o.stride() != g.stride() and not _same_order(o, g)):
                raise ValueError(f"output {i}: shape {tuple(o.shape)} strides {o.stride()}, not {tuple(g.shape)} {g.stride()}")
        arr[i] = Grad(at, to, n, code, to_code)
        if write and n:
            spans.append((to, to + n * (4 if to_code == OUT_F32 else 2), True, i))
            if at != to:
                spans.append((at, at + n * (4 if code == OUT_F32 else 2), False, i))
    _refuse_overlaps(spans)
    return arr, (grads, out)


def prepare_grad_norm(grads):
    """grad_norm(grads) marshalled once: a function that launches it on the current
    stream (or `stream`) again and returns the same (norm, sum_sq) tensors.  It
    holds the gradients and a workspace, made on the stream that is current here;
    calls of it that overlap race."""
    return _prepared_norm(*_grad_list(grads, write=False))


def _prepared_norm(arr, keep):
    first = keep[0][0]
    torch, _ = _enter(first, None)
    size = lib().mxq_grad_norm_workspace_size(arr, len(arr))
    ws = first.new_empty(max(size, 8), dtype=torch.uint8)
    norm, sum_sq = first.new_empty((), dtype=torch.float32), first.new_empty((), dtype=torch.float64)
    ptrs = _ptr(norm), _ptr(sum_sq), _ptr(ws), size
    fn = lib().mxq_grad_norm

    def call(stream=None):
        _check("mxq_grad_norm", fn(arr, len(arr), *ptrs, _enter(first, stream)[1]))
        return norm, sum_sq
    call._keep = (arr, keep, ws)
    return call


def prepare_clip_grad_norm(grads, max_norm, *, eps, out=None):
    """clip_grad_norm(grads, max_norm) marshalled once: a function that launches it
    on the current stream (or `stream`) again and returns the same norm tensor.  It
    holds the gradients, the outputs and a workspace, made on the stream that is
    current here; calls of it that overlap race."""
    arr, keep = _grad_list(grads, out)
    first = keep[0][0]
    measure = _prepared_norm(arr, keep)
    fn = lib().mxq_grad_clip

    def call(stream=None):
        norm, sum_sq = measure(stream)
        _check("mxq_grad_clip", fn(arr, len(arr), _ptr(sum_sq), max_norm, eps, _enter(first, stream)[1]))
        return norm
    call._keep = (arr, keep, measure)
    return call


def grad_norm(grads, stream=None):
    """mxq_grad_norm: (norm, sum_sq) over a list of tensors, fp32 and fp64 scalars."""
    arr, keep = _grad_list(grads, write=False)
    return _norm(arr, keep[0][0], stream)


def _norm(arr, first, stream):
    torch, handle = _enter(first, stream)
    size = lib().mxq_grad_norm_workspace_size(arr, len(arr))
    ws = _new(first, (max(size, 8),), torch.uint8, stream)
    norm, sum_sq = _new(first, (), torch.float32, stream), _new(first, (), torch.float64, stream)
    _check("mxq_grad_norm", lib().mxq_grad_norm(arr, len(arr), _ptr(norm), _ptr(sum_sq), _ptr(ws), size, handle))
    return norm, sum_sq


def grad_clip(grads, sum_sq, max_norm, *, eps, out=None, stream=None):
    """mxq_grad_clip: the gradients scaled to max_norm by a sum of squares (fp64), in
    place or into `out`, a list of tensors of the same shapes, which may share memory
    with no other of them."""
    arr, keep = _grad_list(grads, out)
    _clip(arr, keep[0][0], sum_sq, max_norm, eps, stream)


def _clip(arr, first, sum_sq, max_norm, eps, stream):
    torch, handle = _enter(first, stream)
    _check("mxq_grad_clip", lib().mxq_grad_clip(
        arr, len(arr), _vector("sum_sq", sum_sq, (), first, torch.float64), max_norm, eps, handle))


def clip_grad_norm(grads, max_norm, *, eps, out=None, stream=None):
    """grad_norm, then grad_clip by it; returns the norm."""
    arr, keep = _grad_list(grads, out)
    norm, sum_sq = _norm(arr, keep[0][0], stream)
    _clip(arr, keep[0][0], sum_sq, max_norm, eps, stream)
    return norm
