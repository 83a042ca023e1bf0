"""Launches over more rows (or chunks of rows) than they have workgroups, where a workgroup takes several
in turn and uses its LDS again: with more rows than the library launches workgroups, and for every form of
the kernels with the library built for five workgroups, which has to give the bits of the other.  Rows
that are ignored, foreign ids, non-finite and masked rows come in every order."""
import os

import pytest
import torch

import row_refs as ref
from gpuhelp import dev, say
from test_gpu_norm import EPS, placed, rand, untouched
from test_gpu_vocab import check_logprobs, special, teacher_of, tokens_of

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
INF = float("inf")
GRID = 1 << 20      # workgroups of the library's largest launch over rows
BASE = 19           # different rows; no workgroup's rows are all alike
SAME = BASE * 8     # rows apart that are alike and at the same offset from a 16-byte boundary


def rows_of(vocab, dtype):
    """BASE rows, their tokens, teachers and weights."""
    z = torch.cat([special(vocab, dtype), rand((BASE - 16, vocab), 8, dtype, 2.0)])
    tokens = tokens_of(z, 1)
    tokens[0], tokens[5], tokens[6] = -1, vocab, vocab - 1
    ids, lps = teacher_of(z, 12, 3)
    ids[0], lps[5], ids[6, 3] = -1, -INF, vocab
    w = rand((BASE,), 4)
    w[2] = w[7] = w[17] = 0.0
    return z, tokens, ids, lps, w


def repeat(t, rows):
    return t[torch.arange(rows, device=t.device) % BASE]


def bits(t):
    return t.contiguous().view({2: torch.int16, 4: torch.int32}[t.element_size()])


def same_rows(what, *outs):
    for n, out in enumerate(outs):
        b = bits(out)
        assert torch.equal(b[SAME:], b[:-SAME]), (what, n)


@pytest.mark.parametrize("vocab", [5, 9])
@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
def test_more_rows_than_workgroups(mxq_lib, vocab, dtype):
    m, rows = mxq_lib, GRID + 5
    z, tokens, ids, lps, w = rows_of(vocab, dtype)
    big = [repeat(x.to(dev()), rows) for x in (z, tokens, ids, lps, w)]
    z, tokens, ids, lps, w = (repeat(x, SAME) for x in (z, tokens, ids, lps, w))
    say("many rows, logprobs", vocab, dtype)
    for k in (0, 7):
        out = m.token_logprobs(big[0], big[1], top_k=k)
        check_logprobs((vocab, k), [x[:SAME] for x in out], z, 1.0, tokens, k)
        same_rows(("logprobs", k), *out)
    stats, ent = out[2], out[1]
    gl, gh = (repeat(rand((BASE,), n, scale=s), SAME) for n, s in ((1, 1.0), (2, 0.1)))
    say("many rows, logprobs backward", vocab, dtype)
    back = m.token_logprobs_backward(big[0], big[1], stats, ent, *(repeat(x[:BASE].to(dev()), rows) for x in (gl, gh)))
    want, bound = ref.logprobs_backward(ref.Distribution(z, 1.0, stats[:SAME]), tokens, ent[:SAME], gl, gh)
    ref.check("dlogits", back[:SAME], want, ref.store(dtype, want, bound))
    same_rows("logprobs backward", back)
    say("many rows, distill", vocab, dtype)
    rl, rz, e_l, e_z = ref.distill(ref.Distribution(z, 1.0), ids, lps, w, True)
    loss, stats = m.distill_forward(big[0], *big[2:])
    ref.check("loss", loss[:SAME], rl, e_l.nan_to_num() + 1e-37)
    back = m.distill_backward(big[0], big[2], big[3], stats, big[4])
    loss2, both = m.distill(big[0], *big[2:], out=big[0])
    for what, got in (("backward", back), ("gradient of the pass", both)):
        ref.check(what, got[:SAME], rz, ref.store(dtype, rz, e_z.nan_to_num()))
    ref.check("loss of the pass", loss2[:SAME], rl, e_l.nan_to_num() + 1e-37)
    same_rows("distill", loss, stats, back, loss2, both)


@pytest.mark.parametrize("rows,cols", [(GRID + 5, 3), (GRID + 5, 5), (2 * GRID + 3, 8)])
@pytest.mark.parametrize("kind", ["layer", "rms"])
def test_norm_of_more_rows_than_workgroups(mxq_lib, kind, rows, cols):
    m, layer = mxq_lib, kind == "layer"
    say("many rows, norm", kind, rows, cols)
    x, dy = rand((BASE, cols), 1, BF16, 1.7, 0.6), rand((BASE, cols), 2, F32, 0.1)
    gamma = rand((cols,), 3, scale=0.3, offset=1.0)
    xd, dd = repeat(x.to(dev()), rows), repeat(dy.to(dev()), rows)
    code = m.NORM_LAYER if layer else m.NORM_RMS
    x, dy = repeat(x, SAME), repeat(dy, SAME)
    y, mean, rstd = m.norm_forward(xd, gamma.to(dev()), eps=EPS, kind=code, out_dtype=F32)
    ry, rmean, rrstd, d_y, d_mean, d_rstd = ref.norm(x, gamma, None, EPS, layer)
    ref.check("rstd", rstd[:SAME], rrstd, d_rstd)
    ref.check("y", y[:SAME], ry, d_y)
    same_rows("norm", y, rstd, *([mean] if layer else []))
    dx, _, _ = m.norm_backward(dd, xd, gamma.to(dev()), mean, rstd, kind=code, weight=False, bias=False, out_dtype=F32)
    rdx, _, _, e_dx, _, _ = ref.norm_backward(dy, x, gamma, mean[:SAME] if layer else None, rstd[:SAME], layer)
    ref.check("dx", dx[:SAME], rdx, e_dx)
    same_rows("norm backward", dx)


def with_loops(mxq, monkeypatch, f):
    """f() with the library whose launches have five workgroups."""
    from fp4_microscaling_quantization_amd import build
    assert os.path.exists(build.LOOP_LIB), "libmxq_loop.so is not built"
    with monkeypatch.context() as p:
        p.setattr(mxq, "LIB_PATH", build.LOOP_LIB)
        p.setattr(mxq, "_lib", None)
        out = f()
        torch.cuda.synchronize()
        return out


# the forms: shorter than a vector, a wave a row, 256, 512 and 1024 threads, rows longer than they hold, parts
SHAPES = [(23, 6), (2051, 5), (2051, 515), (2051, 4000), (23, 4099), (23, 30000), (23, 40000), (540, 50257), (23, 50257),
          (210, 65545), (210, 100000), (110, 131075), (23, 200003)]


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
def test_every_form(mxq_lib, monkeypatch, shape, dtype):
    m = mxq_lib
    rows, vocab = shape
    z, tokens, ids, lps, w = (repeat(x.to(dev()), rows) for x in rows_of(vocab, dtype))
    gl, gh = (repeat(rand((BASE,), n).to(dev()), rows) for n in (1, 2))
    zd, zb = placed(z, 3, 1)

    def run():
        outs = []
        for k in (0, 20, 64):
            outs += m.token_logprobs(zd, tokens, top_k=k, temperature=2.0)
        ent, stats = outs[-4], outs[-3]
        for ot in (F32, BF16):
            outs.append(m.token_logprobs_backward(zd, tokens, stats, ent, gl, gh, temperature=2.0, out_dtype=ot))
        outs += m.distill_forward(zd, ids, lps, w, temperature=2.0)
        for ot in (F32, BF16):
            outs.append(m.distill_backward(zd, ids, lps, stats, w, temperature=2.0, out_dtype=ot))
            outs += m.distill(zd, ids, lps, w, temperature=2.0, out_dtype=ot)
        for f in (lambda o: m.token_logprobs_backward(o, tokens, stats, ent, gl, gh, temperature=2.0, out=o),
                  lambda o: m.distill(o, ids, lps, w, temperature=2.0, out=o)[1]):
            over, ob = placed(z, 3, 1)
            outs.append(f(over))
            assert untouched(over, ob)
        return outs
    say("loops, one", shape, dtype)
    want = run()
    say("loops, five workgroups", shape, dtype)
    got = with_loops(m, monkeypatch, run)
    assert len(got) == len(want)
    for n, (a, b) in enumerate(zip(got, want)):
        assert torch.equal(bits(a), bits(b)), (shape, n)
    assert untouched(zd, zb)


@pytest.mark.parametrize("shape", [(23, 3), (4099, 6), (4099, 515), (4098, 2041), (23, 1024), (23, 4099), (23, 9001), (23, 16392),
                                   (23, 40001), (23, 70001)], ids=str)
@pytest.mark.parametrize("kind", ["layer", "rms"])
def test_every_form_of_the_norm(mxq_lib, monkeypatch, kind, shape):
    m = mxq_lib
    rows, cols = shape
    code = m.NORM_LAYER if kind == "layer" else m.NORM_RMS
    x, dy = repeat(rand((BASE, cols), 1, F32, 1.7, 0.6), rows), repeat(rand((BASE, cols), 2, F32, 0.1), rows)
    x[4, cols // 2], x[9, 0] = float("nan"), INF
    gamma = rand((cols,), 3, scale=0.3, offset=1.0).to(dev())

    def run():
        outs = []
        for xt, ot in ((F32, BF16), (BF16, F32), (BF16, BF16)):
            xd, dd = placed(x.to(xt), 3, 1)[0], placed(dy.to(ot), 1, 3)[0]
            y, mean, rstd = m.norm_forward(xd, gamma, eps=EPS, kind=code, out_dtype=ot)
            dx, dg, db = m.norm_backward(dd, xd, gamma, mean, rstd, kind=code, out_dtype=ot)
            over, _, _ = m.norm_forward(xd, gamma, eps=EPS, kind=code, out=xd)
            outs += [t for t in (y, mean, rstd, dx, dg, db, over) if t is not None]
        return outs
    say("loops of the norm, one", kind, shape)
    want = run()
    say("loops of the norm, five workgroups", kind, shape)
    for n, (a, b) in enumerate(zip(with_loops(m, monkeypatch, run), want)):
        assert torch.equal(bits(a), bits(b)), (shape, n)
