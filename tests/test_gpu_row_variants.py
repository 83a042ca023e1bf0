"""The row operators where many rows or long ones choose another kernel: a wave
a row, two rows a wave, workgroups of 512 and 1024 threads, rows read in several
stretches.  Sixteen rows are compared with 64 bits; every other row repeats one
of them at the same alignment and has to have the same bits."""
import pytest
import torch

import row_refs as ref
from gpuhelp import dev, say
from test_gpu_norm import EPS, placed, rand, untouched
from test_gpu_vocab import check_logprobs, special, teacher_of, tokens_of

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
INF = float("inf")
BASE = 16

# many short rows, then rows of one stretch and of several
SHAPES = [(2050, 9), (2051, 515), (2048, 1000), (2049, 2045), (2051, 4089), (2048, 4093), (2049, 8185),
          (170, 40000), (600, 50257), (200, 65545), (100, 131072), (52, 131075), (520, 131075)]


def repeat(t, rows):
    return t[torch.arange(rows) % BASE]


def stored(t):
    """64-bit values that are to be fp32: beyond its range they are infinite."""
    return torch.where(t.abs() > torch.finfo(F32).max, t * INF, t)


def same_rows(what, *outs):
    for n, out in enumerate(outs):
        bits = out.contiguous().view({2: torch.int16, 4: torch.int32}[out.element_size()])
        want = bits[:BASE][torch.arange(len(bits), device=bits.device) % BASE]
        assert torch.equal(bits, want), (what, n, (bits != want).nonzero()[:4].tolist())


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
def test_logprobs(mxq_lib, shape, dtype):
    rows, vocab = shape
    z = special(vocab, dtype)
    tokens = tokens_of(z, 1)
    tokens[0], tokens[5], tokens[6] = -1, vocab, vocab - 1
    for t, k, pad, shift in ((1.0, 0, 0, 0), (2.0, 20, 3, 1), (0.7, 64, 8, 8)):
        say("logprobs", shape, dtype, (t, k, pad, shift))
        zd, zb = placed(repeat(z, rows), pad, shift)
        out = mxq_lib.token_logprobs(zd, repeat(tokens, rows).to(dev()), top_k=k, temperature=t)
        d = ref.Distribution(z, t)
        d.logq = stored(d.logq)        # the lowest value over 0.7
        check_logprobs((shape, t, k), [x[:BASE] for x in out], z, t, tokens, k, d)
        same_rows((shape, t, k), *out)
        assert untouched(zd, zb)


@pytest.mark.parametrize("vocab", [500, 4000, 8000])
@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
def test_top_clustered(mxq_lib, vocab, dtype):
    """The largest logits in one lane's places, in one stretch, and all equal."""
    rows = 2048
    for step in (1, 4, 8, 64, 256, 512, 1024):
        say("clustered", vocab, step, dtype)
        z = rand((BASE, vocab), step, F32, 0.5)
        at = torch.arange(vocab) // step % max(2, vocab // step // 64) == 1
        z[:, at] = 20.0 + 4 * rand((BASE, int(at.sum())), 9)
        z[3::4] = z[3::4].round()
        z = z.to(dtype)
        out = mxq_lib.token_logprobs(repeat(z, rows).to(dev()), top_k=64)
        assert torch.equal(out[3][:BASE].cpu().long(), ref.Distribution(z, 1.0).top(64)), (vocab, step)
        same_rows((vocab, step), out[3], out[4])


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
def test_logprobs_backward(mxq_lib, shape, dtype):
    m = mxq_lib
    rows, vocab = shape
    z = special(vocab, dtype)
    tokens = tokens_of(z, 1)
    tokens[0], tokens[5], tokens[6] = -1, vocab, vocab - 1
    gl, gh = rand((BASE,), 1), rand((BASE,), 2, scale=0.1)
    _, ent, stats = m.token_logprobs(z.to(dev()), tokens.to(dev()))
    d = ref.Distribution(z, 1.0, stats)
    want, bound = ref.logprobs_backward(d, tokens, ent, gl, gh)
    args = [repeat(x.cpu(), rows).to(dev()) for x in (tokens, stats, ent, gl, gh)]
    for ot, pad, shift in ((BF16, 0, 0), (F32, 3, 1), (dtype, 8, 8)):
        say("logprobs backward", shape, dtype, ot, (pad, shift))
        zd, zb = placed(repeat(z, rows), pad, shift)
        inplace = pad == 8
        out, ob = (zd, zb) if inplace else placed(torch.zeros((rows, vocab), dtype=ot), pad + 1, shift)
        m.token_logprobs_backward(zd, *args, out=out)
        ref.check("dlogits", out[:BASE], want, ref.store(ot, want, bound))
        same_rows(shape, out)
        assert untouched(out, ob)


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
def test_distill(mxq_lib, shape, dtype):
    """Loss, its gradient and the pass that gives both; the last one also over the logits."""
    m = mxq_lib
    rows, vocab = shape
    z = special(vocab, dtype)
    for n, (t, renorm, ot, pad, shift) in enumerate([(1.0, True, BF16, 0, 0), (2.0, False, F32, 3, 1), (1.0, True, dtype, 8, 8)]):
        say("distill", shape, dtype, (t, renorm, ot, pad, shift))
        ids, lps = teacher_of(z, (12, 33, 64)[n], 3 + n, ragged=n > 0)
        ids[0], lps[5], ids[6, 3] = -1, -INF, vocab
        w = rand((BASE,), 4)
        w[2] = 0.0
        d = ref.Distribution(z, t)
        rl, rz, e_l, e_z = ref.distill(d, ids, lps, w, renorm)
        bound = ref.store(ot, rz, e_z.nan_to_num())
        zd, zb = placed(repeat(z, rows), pad, shift)
        i, p, wd = (repeat(x, rows).to(dev()) for x in (ids, lps, w))
        loss, stats = m.distill_forward(zd, i, p, wd, temperature=t, renormalize=renorm)
        ref.check("loss", loss[:BASE], rl, e_l.nan_to_num() + 1e-37)
        same_rows(shape, loss, stats)
        back = m.distill_backward(zd, i, p, stats, wd, temperature=t, renormalize=renorm, out_dtype=ot)
        ref.check("backward", back[:BASE], rz, bound)
        same_rows(shape, back)
        inplace = pad == 8
        out, ob = (zd, zb) if inplace else placed(torch.zeros((rows, vocab), dtype=ot), pad + 1, shift)
        loss, _ = m.distill(zd, i, p, wd, temperature=t, renormalize=renorm, out=out)
        ref.check("loss of the pass", loss[:BASE], rl, e_l.nan_to_num() + 1e-37)
        ref.check("gradient of the pass", out[:BASE], rz, bound)
        same_rows(shape, loss, out)
        assert untouched(out, ob)


@pytest.mark.parametrize("cols", [8, 9, 64, 1023, 2041, 2048, 2057, 4096])
@pytest.mark.parametrize("rows", [4096, 4099])
@pytest.mark.parametrize("kind", ["layer", "rms"])
def test_norm_forward(mxq_lib, kind, rows, cols):
    m = mxq_lib
    layer = kind == "layer"
    gamma = rand((cols,), 2, scale=0.3, offset=1.0)
    beta = rand((cols,), 3) if layer else None
    for n, (xt, yt) in enumerate([(BF16, BF16), (F32, BF16), (BF16, F32), (F32, F32)]):
        pad, shift = ((0, 0), (5, 1), (8, 8), (0, 0))[n]
        say("norm forward", kind, (rows, cols), xt, yt, (pad, shift))
        x = rand((BASE, cols), 10 * n + 1, xt, 1.7, 0.6)
        x[3] = 2.5
        xd, xb = placed(repeat(x, rows), pad, shift)
        out, ob = placed(torch.zeros((rows, cols), dtype=yt), pad + 1, shift)
        y, mean, rstd = m.norm_forward(xd, gamma.to(dev()), None if beta is None else beta.to(dev()), eps=EPS,
                                       kind=m.NORM_LAYER if layer else m.NORM_RMS, out=out)
        ry, rmean, rrstd, d_y, d_mean, d_rstd = ref.norm(x, gamma, beta, EPS, layer)
        if layer:
            ref.check("mean", mean[:BASE], rmean, d_mean)
            same_rows("mean", mean)
        ref.check("rstd", rstd[:BASE], rrstd, d_rstd)
        ref.check("y", y[:BASE], ry, ref.store(yt, ry, d_y))
        same_rows("norm", y, rstd)
        assert untouched(out, ob) and untouched(xd, xb)


@pytest.mark.parametrize("shape", [(2048, 64), (4099, 96), (2100, 1030), (600, 3001), (1030, 4099), (300, 8192),
                                   (300, 9001), (261, 14336)], ids=str)
@pytest.mark.parametrize("kind", ["layer", "rms"])
@pytest.mark.parametrize("bias", [True, False], ids=["bias", "no bias"])
def test_norm_backward(mxq_lib, shape, kind, bias):
    m = mxq_lib
    layer = kind == "layer"
    rows, cols = shape
    for n, (dt, xt, ot) in enumerate([(BF16, BF16, BF16), (F32, BF16, F32), (F32, F32, BF16), (BF16, F32, F32)]):
        pad, shift = ((0, 0), (5, 1), (8, 8), (0, 0))[n]
        say("norm backward", kind, shape, dt, xt, ot, (pad, shift), bias)
        x = rand(shape, 10 * n + 1, xt, 1.7, 0.6)
        dy = rand(shape, 10 * n + 2, dt, 0.1)
        gamma = rand((cols,), 4, scale=0.3, offset=1.0)
        _, mean, rstd, *_ = ref.norm(x, None, None, EPS, layer)
        mean, rstd = mean.float(), rstd.float()
        xd, _ = placed(x, pad, shift)
        dd, db = placed(dy, pad + 2, shift)
        out, ob = placed(torch.zeros(shape, dtype=ot), pad + 1, shift)
        dx, dg, dbeta = m.norm_backward(dd, xd, gamma.to(dev()), mean.to(dev()) if layer else None, rstd.to(dev()),
                                        kind=m.NORM_LAYER if layer else m.NORM_RMS, bias=bias, out=out)
        rdx, rdg, rdb, e_dx, e_dg, e_db = ref.norm_backward(dy, x, gamma, mean, rstd, layer)
        ref.check("dx", dx, rdx, ref.store(ot, rdx, e_dx))
        ref.check("dgamma", dg, rdg, e_dg + 1e-37)
        if bias:
            ref.check("dbeta", dbeta, rdb, e_db + 1e-37)
        else:
            assert dbeta is None
        assert untouched(out, ob) and untouched(dd, db)
