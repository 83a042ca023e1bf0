"""mxq_norm_forward and mxq_norm_backward against the formulas in 64 bits: row
lengths from one element to several workgroups' worth, every type, rows that
start off the vector alignment, padded leading dimensions, rows of equal
values, non-finite rows; gradients also against differences."""
import pytest
import torch

import row_refs as ref
from gpuhelp import dev, say

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
EPS = 1e-5


def rand(shape, seed, dtype=F32, scale=1.0, offset=0.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale + offset).to(dtype)


def placed(t, pad, shift):
    """t on the GPU with `pad` more columns a row and its first element `shift`
    elements after a 256-byte boundary; the buffer around it holds 7."""
    rows, cols = t.shape
    buf = torch.full((shift + rows * (cols + pad) + 64,), 7.0, dtype=t.dtype, device=dev())
    view = buf[shift:shift + rows * (cols + pad)].view(rows, cols + pad)[:, :cols]
    view.copy_(t)
    return view, buf


def untouched(view, buf):
    """Whether everything of the buffer outside the view still holds 7."""
    keep = view.clone()
    view.fill_(7.0)
    ok = bool((buf == 7.0).all())
    view.copy_(keep)
    return ok


SHAPES = [(1, 1), (3, 1), (1, 2), (5, 7), (2, 64), (3, 255), (1, 4096), (17, 1023), (4, 2048), (9, 4099),
          (2, 8192), (3, 14336), (2, 16385), (2, 40001), (1, 131072), (300, 96), (1025, 33)]


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("kind", ["layer", "rms"])
def test_forward(mxq_lib, shape, kind):
    m = mxq_lib
    layer = kind == "layer"
    rows, cols = shape
    for n, (xt, yt, affine) in enumerate([(BF16, BF16, True), (F32, BF16, False), (F32, F32, True), (BF16, F32, True)]):
        for pad, shift in ((0, 0), (5, 1), (8, 8)):
            say("norm forward", kind, shape, xt, yt, (pad, shift))
            x = rand(shape, 10 * n + 1, xt, 1.7, 0.6)
            gamma = rand((cols,), 2, scale=0.3, offset=1.0) if affine else None
            beta = rand((cols,), 3) if affine and layer else None
            xd, xb = placed(x, pad, shift)
            out, ob = placed(torch.zeros(shape, dtype=yt), pad + 1, shift)
            y, mean, rstd = m.norm_forward(xd, None if gamma is None else gamma.to(dev()),
                                           None if beta is None else beta.to(dev()), eps=EPS,
                                           kind=m.NORM_LAYER if layer else m.NORM_RMS, out=out)
            torch.cuda.synchronize()
            ry, rmean, rrstd, dy_, dmean, drstd = ref.norm(x, gamma, beta, EPS, layer)
            assert y is out and (mean is not None) == layer
            if layer:
                ref.check("mean", mean, rmean, dmean)
            ref.check("rstd", rstd, rrstd, drstd)
            ref.check("y", y, ry, ref.store(yt, ry, dy_))
            assert untouched(out, ob) and untouched(xd, xb)


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("kind", ["layer", "rms"])
def test_backward(mxq_lib, shape, kind):
    m = mxq_lib
    layer = kind == "layer"
    rows, cols = shape
    types = [(BF16, BF16, BF16), (F32, BF16, BF16), (F32, F32, F32), (BF16, F32, BF16), (F32, BF16, F32)]
    for n, (dt, xt, ot) in enumerate(types):
        pad, shift = ((0, 0), (5, 1), (8, 8))[n % 3]
        say("norm backward", kind, shape, dt, xt, ot, (pad, shift))
        x = rand(shape, 10 * n + 1, xt, 1.7, 0.6)
        dy = rand(shape, 10 * n + 2, dt, 0.1)
        gamma = rand((cols,), 4, scale=0.3, offset=1.0) if n % 2 == 0 else None
        _, mean, rstd, *_ = ref.norm(x, None, None, EPS, layer)
        mean, rstd = mean.float(), rstd.float()
        xd, _ = placed(x, pad, shift)
        dd, db = placed(dy, pad + 2, shift)
        out, ob = placed(torch.zeros(shape, dtype=ot), pad + 1, shift)
        dx, dg, dbeta = m.norm_backward(dd, xd, None if gamma is None else gamma.to(dev()),
                                        mean.to(dev()) if layer else None, rstd.to(dev()),
                                        kind=m.NORM_LAYER if layer else m.NORM_RMS, out=out)
        torch.cuda.synchronize()
        rdx, rdg, rdb, e_dx, e_dg, e_db = ref.norm_backward(dy, x, gamma, mean, rstd, layer)
        ref.check("dx", dx, rdx, ref.store(ot, rdx, e_dx))
        ref.check("dgamma", dg, rdg, e_dg + 1e-37)
        ref.check("dbeta", dbeta, rdb, e_db + 1e-37)
        assert untouched(out, ob) and untouched(dd, db)


def test_backward_parts_and_in_place(mxq_lib):
    """Only what is asked for; dx over dy and over x."""
    m = mxq_lib
    for rows, cols in ((70, 515), (33, 4096), (5, 20000)):
        x, dy = rand((rows, cols), 1, BF16), rand((rows, cols), 2, BF16)
        gamma = rand((cols,), 3).to(dev())
        y, mean, rstd = m.norm_forward(x.to(dev()), gamma, eps=EPS)
        say("norm backward in place", (rows, cols))
        dx, dg, db = m.norm_backward(dy.to(dev()), x.to(dev()), gamma, mean, rstd)
        only, none_g, none_b = m.norm_backward(dy.to(dev()), x.to(dev()), gamma, mean, rstd, weight=False, bias=False)
        assert none_g is None and none_b is None and torch.equal(only, dx)
        _, dg2, none_b = m.norm_backward(dy.to(dev()), x.to(dev()), gamma, mean, rstd, bias=False)
        assert none_b is None and torch.equal(dg2, dg)
        _, none_g, db2 = m.norm_backward(dy.to(dev()), x.to(dev()), gamma, mean, rstd, weight=False)
        assert none_g is None and torch.equal(db2, db)
        for over in ("dy", "x"):
            xd, dd = x.to(dev()), dy.to(dev())
            dx2, dg3, db3 = m.norm_backward(dd, xd, gamma, mean, rstd, out=dd if over == "dy" else xd)
            assert torch.equal(dx2, dx) and torch.equal(dg3, dg) and torch.equal(db3, db)
        xd = x.to(dev())
        y2, _, _ = m.norm_forward(xd, gamma, eps=EPS, out=xd)
        assert torch.equal(y2, y)


def test_no_rows(mxq_lib):
    m = mxq_lib
    say("norm, no rows")
    x = torch.empty((0, 100), device=dev())
    y, mean, rstd = m.norm_forward(x, eps=EPS)
    assert y.shape == (0, 100) and mean.shape == rstd.shape == (0,)
    dx, dg, db = m.norm_backward(x, x, None, mean, rstd)
    assert dx.shape == (0, 100) and torch.equal(dg, torch.zeros(100, device=dev())) and torch.equal(db, dg)


@pytest.mark.parametrize("cols", [5, 4096, 40001])
def test_special_rows(mxq_lib, cols):
    """Equal values (variance 0), tiny and large rows, a NaN, an infinity: the
    bad rows are NaN and leave the others alone."""
    m = mxq_lib
    x = rand((8, cols), 1)
    x[1] = 3.25
    x[2] = 0.0
    x[3] *= 1e-18
    x[4] *= 1e15
    x[5, cols // 2] = float("nan")
    x[6, cols - 1] = float("inf")
    for kind, layer in ((m.NORM_LAYER, True), (m.NORM_RMS, False)):
        say("norm special rows", cols, kind)
        y, mean, rstd = m.norm_forward(x.to(dev()), eps=EPS, kind=kind)
        y = y.cpu()
        ok = torch.tensor([0, 1, 2, 3, 4, 7])
        ry, _, rr, d_y, _, d_r = ref.norm(x[ok], None, None, EPS, layer)
        ref.check("y", y[ok], ry, d_y)
        ref.check("rstd", rstd.cpu()[ok], rr, d_r)
        assert y[5].isnan().all()
        # the root-mean-square norm of an infinity is inf * 0 there and 0 elsewhere
        assert y[6].isnan().all() if layer else bool(y[6, cols - 1].isnan())


def test_offsets_past_32_bits(mxq_lib):
    """Rows whose element offsets pass 2^31 and whose byte offsets pass 2^32."""
    m = mxq_lib
    cols, ld = 300, (1 << 30) + 3
    x = rand((4, cols), 1, BF16)
    buf = torch.empty(3 * ld + cols, dtype=BF16, device=dev())
    view = buf.as_strided((4, cols), (ld, 1))
    view.copy_(x)
    say("norm, far rows")
    y, mean, rstd = m.norm_forward(view, eps=EPS, out=view)
    ry, _, _, d_y, _, _ = ref.norm(x, None, None, EPS, True)
    ref.check("y", y, ry, ref.store(BF16, ry, d_y))
    view.copy_(x)
    dy = rand((4, cols), 2).to(dev())
    dx, dg, db = m.norm_backward(dy, view, None, mean, rstd, out=view)
    rdx, rdg, _, e_dx, e_dg, _ = ref.norm_backward(dy, x, None, mean, rstd, True)
    ref.check("dx", dx, rdx, ref.store(BF16, rdx, e_dx))
    ref.check("dgamma", dg, rdg, e_dg)


def test_gradient_against_differences(mxq_lib):
    """dx, dgamma, dbeta against central differences of the 64-bit forward pass:
    with step h the difference is off by h^2 / 6 of the third derivative, which
    stays under 100 rstd^3 |dy| here, and by 2^-52 / h of the value."""
    m = mxq_lib
    rows, cols, h = 4, 37, 1e-4
    x, dy = rand((rows, cols), 1), rand((rows, cols), 2)
    gamma, beta = rand((cols,), 3, offset=1.0), rand((cols,), 4)
    for kind, layer in ((m.NORM_LAYER, True), (m.NORM_RMS, False)):
        say("norm differences", kind)
        y, mean, rstd = m.norm_forward(x.to(dev()), gamma.to(dev()), beta.to(dev()), eps=EPS, kind=kind)
        got = m.norm_backward(dy.to(dev()), x.to(dev()), gamma.to(dev()), mean, rstd, kind=kind)

        def value(x_, g_, b_):
            return (ref.norm(x_, g_, b_, EPS, layer)[0] * dy.double()).sum()
        args = [x.double(), gamma.double(), beta.double()]
        tol = h * h * 100 * float(rstd.max()) ** 3 * float(dy.abs().sum()) + 2.0 ** -52 / h * 1e3
        for k, grad in enumerate(got):
            want = torch.zeros_like(args[k])
            for i in range(want.numel()):
                for sign in (1, -1):
                    moved = [a.clone() for a in args]
                    moved[k].view(-1)[i] += sign * h
                    want.view(-1)[i] += sign * value(*moved) / (2 * h)
            # the formula's bound, the differences' error, and what fp32 mean and rstd shift: about
            # (depth + 8) u = 2.5e-6 of parts that are under 8
            rs = ref.norm_backward(dy, x, gamma, mean.cpu() if layer else None, rstd.cpu(), layer)
            ref.check(("difference", k), grad, want, rs[3 + k] + tol + 2e-5 * (rs[k].abs() + 1))


def test_repeats_streams_and_graph(mxq_lib):
    """The same bits again, on another stream, and from each replay of a graph."""
    m = mxq_lib
    rows, cols = 700, 4096
    x, dy = rand((rows, cols), 1, BF16).to(dev()), rand((rows, cols), 2).to(dev())
    gamma = rand((cols,), 3).to(dev())

    def step(stream=None):
        y, mean, rstd = m.norm_forward(x, gamma, eps=EPS, stream=stream)
        return (y, mean, rstd, *m.norm_backward(dy, x, gamma, mean, rstd, stream=stream))
    say("norm repeats")
    first = [t.clone() for t in step()]
    assert all(torch.equal(a, b) for a, b in zip(first, step()))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = step(side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, other))
    say("norm graph")
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    for _ in range(3):
        for t in outs:
            t.fill_(float("nan"))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(first, outs))
        step()
