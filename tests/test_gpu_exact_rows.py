"""The row operators on rows whose sums are exact in any order (exact_rows): S and the gradients' sums
have to be equal, and what follows from them within a few roundings, so that no element may be
lost or counted twice at the end of a vector, a stretch, a part or a chunk, or before a row that starts
off a 16-byte boundary.  The rows of a case start at every offset from such a boundary."""
import pytest
import torch

import exact_rows as ex
from exact_rows import TEMPERATURE, U
from gpuhelp import dev, say
from test_gpu_norm import placed

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
INF = float("inf")

# short rows, a wave a row (2057 and more rows), one stretch, several, parts of few long rows
SHAPES = [(9, 5), (9, 9), (9, 15), (9, 1000), (2057, 6), (2057, 1000), (2057, 4089), (2049, 8185), (9, 4099), (9, 32765),
          (9, 32771), (9, 49157), (9, 65529), (9, 65545), (9, 131065), (9, 131075), (9, 300007), (520, 50257),
          (520, 131075), (105, 65545), (200, 200003)]


def odd(t):
    """t placed so that its rows start at all offsets."""
    return placed(t, 1 - t.shape[1] % 2 + 2, 1)[0]


def within(what, got, want, bound):
    off = (got.double() - want).abs()
    bad = ~(off <= bound)
    assert not bool(bad.any()), (what, int(bad.sum()), bad.nonzero()[:4].tolist(), got[bad][:4].tolist(),
                                 want[bad][:4].tolist(), bound.expand_as(want)[bad][:4].tolist())


def equal(what, got, want):
    bad = got.double() != want
    assert not bool(bad.any()), (what, int(bad.sum()), bad.nonzero()[:4].tolist(), got[bad][:4].tolist(), want[bad][:4].tolist())


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
def test_logprobs(mxq_lib, shape, dtype):
    z = ex.logits(*shape, 1, dev())
    m, s, a = ex.sums(z)
    zd = odd(z.to(dtype))
    want, bound = ex.entropy(s, a)
    for k in (0, 64):
        say("exact logprobs", shape, dtype, k)
        out = mxq_lib.token_logprobs(zd, top_k=k, temperature=TEMPERATURE)
        equal("max", out[2][:, 0], m)
        equal("sum", out[2][:, 1], s)
        within("entropy", out[1], want, bound)
        if k:
            assert torch.equal(out[3].long(), ex.top(z, k)), "ids"


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
def test_distill(mxq_lib, shape, dtype):
    """One certain alternative: the cross entropy, with the gradient of every entry."""
    m = mxq_lib
    rows, vocab = shape
    z = ex.logits(*shape, 2, dev())
    ids = (torch.arange(rows, device=dev(), dtype=torch.int64) * 7919 % vocab).to(torch.int32)[:, None]
    args = ids, torch.zeros((rows, 1), device=dev())
    kw = dict(temperature=TEMPERATURE, renormalize=False)
    _, s, _ = ex.sums(z)
    want, bound = ex.loss(z, ids, s)
    dz, e_dz, _ = ex.gradient(z, ids, s)
    zd = odd(z.to(dtype))
    say("exact distill", shape, dtype)
    loss, stats = m.distill_forward(zd, *args, **kw)
    equal("sum", stats[:, 1], s)
    within("loss", loss, want, bound)
    back = m.distill_backward(zd, *args, stats, out=odd(torch.zeros(shape, device=dev())), **kw)
    within("backward", back, dz, e_dz)
    loss, both = m.distill(zd, *args, out=odd(torch.zeros(shape, device=dev())), **kw)
    within("loss of the pass", loss, want, bound)
    within("gradient of the pass", both, dz, e_dz)
    # in bf16, and over the logits: the same numbers, rounded
    for out in (odd(torch.zeros(shape, device=dev(), dtype=BF16)), zd):
        loss2, got = m.distill(zd, *args, out=out, **kw)
        assert torch.equal(loss2, loss) and torch.equal(got, both.to(got.dtype))


@pytest.mark.parametrize("vocab", [515, 8185, 32771, 50257, 131075, 300007])
@pytest.mark.parametrize("rows", [300, 2057])
@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
def test_pairs_at_boundaries(mxq_lib, rows, vocab, dtype):
    """Two logits that are not masked, side by side: across the borders of what a thread,
    a stretch, a part or a chunk holds, at the row's ends, and anywhere."""
    if rows * vocab > 2 ** 28:
        rows = 600      # more than go as parts
    say("pairs", rows, vocab, dtype)
    r = torch.arange(rows, device=dev())
    pad = 1 - vocab % 2 + 2
    lead = (1 + r * (vocab + pad)) % 8 if dtype == BF16 else 0 * r
    step = max(64, vocab // (rows // 2) // 64 * 64)
    at = torch.where(r % 2 == 0, (r // 2 + 1) * step - lead, (r * 7919 * 31) % vocab).clamp(1, vocab - 1)
    at[0], at[1] = 1, vocab - 1
    z = torch.full((rows, vocab), -INF, device=dev(), dtype=dtype)
    z[r, at - 1], z[r, at] = 0.0, -1.0
    zd = odd(z)
    out = mxq_lib.token_logprobs(zd, at.to(torch.int32), top_k=3, temperature=TEMPERATURE)
    equal("sum", out[2][:, 1], torch.full((rows,), 1.5, device=dev(), dtype=torch.float64))
    assert torch.equal(out[3].long(), torch.stack([at - 1, at, 0 * at - 1], 1))
    want = torch.full((rows,), -1.5849625007211562 / 1.4426950408889634, device=dev(), dtype=torch.float64)
    within("logprob", out[0], want, 8 * U * want.abs())
    ids, lps = at.to(torch.int32)[:, None], torch.zeros((rows, 1), device=dev())
    loss, dz = mxq_lib.distill(zd, ids, lps, temperature=TEMPERATURE, renormalize=False, out_dtype=F32)
    within("loss", loss, -want * TEMPERATURE ** 2, 12 * U * want.abs() * TEMPERATURE ** 2)
    third = TEMPERATURE / 3
    within("dz before", dz[r, at - 1], torch.full_like(want, 2 * third), torch.full_like(want, 8 * U * third))
    within("dz at", dz[r, at], torch.full_like(want, -2 * third), torch.full_like(want, 8 * U * third))
    dz[r, at - 1] = 0
    dz[r, at] = 0
    assert not dz.any()


COLS = [3, 4, 7, 9, 15, 255, 1023, 2041, 2049, 4096, 4099, 8193, 8201, 14336, 16384, 16387, 32771, 40001, 65537, 131077]


@pytest.mark.parametrize("cols", COLS)
@pytest.mark.parametrize("rows", [9, 4099])
@pytest.mark.parametrize("kind", ["layer", "rms"])
def test_norm_forward(mxq_lib, kind, rows, cols):
    m = mxq_lib
    if rows > 9 and cols > 4096:
        rows = 300
    layer = kind == "layer"
    x = ex.balanced(rows, cols, 3, dev())
    gamma = 1.0 + (torch.arange(cols, device=dev()) % 2)
    rstd = ((x.double() ** 2).sum(1) / cols + 0.5).rsqrt()
    y = x.double() * rstd[:, None] * gamma.double()
    for xt, yt in ((F32, F32), (BF16, F32), (BF16, BF16), (F32, BF16)):
        say("exact norm", kind, (rows, cols), xt, yt)
        out = odd(torch.zeros((rows, cols), device=dev(), dtype=yt))
        got, mean, rs = m.norm_forward(odd(x.to(xt)), gamma, eps=0.5, kind=m.NORM_LAYER if layer else m.NORM_RMS, out=out)
        if layer:
            equal("mean", mean, torch.zeros_like(rstd))
        # 1 / n, its product and the sum with eps: 3 u, halved by the root; the root and the reciprocal
        within("rstd", rs, rstd, 4 * U * rstd)
        half = torch.finfo(BF16).eps / 2 if yt == BF16 else 0.0
        within("y", got, y, (6 * U + half) * y.abs() * (1 + 6 * U))
        if layer:
            # one more column's worth of offset: the sum is exact still
            _, mean, _ = m.norm_forward(odd((x + 5).to(xt)), eps=0.5)
            within("mean of an offset", mean, torch.full_like(rstd, 5.0), torch.full_like(rstd, 10 * U))


@pytest.mark.parametrize("cols", COLS)
@pytest.mark.parametrize("rows", [1, 37, 2100])
@pytest.mark.parametrize("kind", ["layer", "rms"])
def test_norm_backward(mxq_lib, kind, rows, cols):
    m = mxq_lib
    if rows > 37 and cols > 16387:
        rows = 300
    layer = kind == "layer"
    x = ex.balanced(rows, cols, 4, dev()) * 2 + 1
    dy = ex.balanced(rows, cols, 5, dev())
    gamma = 1.0 + (torch.arange(cols, device=dev()) % 2)
    mean, rstd = torch.ones(rows, device=dev()), torch.full((rows,), 0.5, device=dev())
    n = (x.double() - (1.0 if layer else 0.0)) * 0.5
    w = dy.double() * gamma.double()
    along = (w * n).sum(1, keepdim=True) / cols
    rest = w.sum(1, keepdim=True) / cols if layer else torch.zeros_like(along)
    dx = 0.5 * (w - n * along - rest)
    # 1 / n and its product, n times it and the difference: 4 u; the second difference
    e_dx = 0.5 * U * (4 * (n * along).abs() + 3 * rest.abs() + 3 * w.abs())
    for dt, xt, ot in ((F32, F32, F32), (BF16, BF16, F32), (F32, BF16, BF16), (BF16, F32, F32), (BF16, BF16, BF16)):
        say("exact norm backward", kind, (rows, cols), dt, xt, ot)
        for bias in (True, False):
            out = odd(torch.zeros((rows, cols), device=dev(), dtype=ot))
            got, dg, db = m.norm_backward(odd(dy.to(dt)), odd(x.to(xt)), gamma, mean if layer else None, rstd,
                                          kind=m.NORM_LAYER if layer else m.NORM_RMS, bias=bias, out=out)
            half = torch.finfo(BF16).eps / 2 if ot == BF16 else 0.0
            within("dx", got, dx, e_dx + half * (dx.abs() + e_dx))
            equal("dgamma", dg, (dy.double() * n).sum(0))
            if bias:
                equal("dbeta", db, dy.double().sum(0))
