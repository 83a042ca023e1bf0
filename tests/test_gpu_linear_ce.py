"""mxq_linear_ce_forward and _backward against the formulas in 64 bits: from one
row and one entry of a vocabulary to several tiles of each, rows that do not
count, odd starts and leading dimensions, non-finite rows, tensors on a stream
of their own, replayed graphs."""
import pytest
import torch

from ce_refs import HeadLoss
from gpuhelp import dev, say
from test_gpu_norm import placed, untouched

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16
INF, NAN = float("inf"), float("nan")

# rows, hidden, vocab
SHAPES = [(1, 32, 1), (2, 64, 2), (5, 96, 63), (1, 256, 500), (16, 160, 257), (17, 544, 1000), (33, 1024, 515),
          (64, 32, 2048), (65, 288, 256), (130, 96, 3001), (255, 512, 255), (256, 256, 512), (257, 320, 513),
          (300, 64, 1031), (520, 736, 777), (700, 128, 2500)]


def case(rows, hidden, vocab, seed, ignored=0.0):
    g = torch.Generator().manual_seed(seed)
    w = (torch.randn(vocab, hidden, generator=g) * (2.5 / hidden ** 0.5)).to(BF16)
    targets = torch.randint(vocab, (rows,), generator=g, dtype=torch.int32)
    x = (torch.randn(rows, hidden, generator=g) + w[targets.long()].float()).to(BF16)
    targets[torch.rand(rows, generator=g) < ignored] = -100
    weight = 0.5 + torch.rand(rows, generator=g)
    return x, w, targets, weight


def run_both(m, x, w, targets, weight, t, want=None):
    """Both passes on the GPU, the second from its own stats, checked against the formulas."""
    d = dev()
    want = want or HeadLoss(x, w, targets, weight, t)
    xd, wd, td = x.to(d), w.to(d), targets.to(d)
    gd = None if weight is None else weight.to(d)
    what = (tuple(x.shape), w.shape[0], t)
    loss, stats = m.linear_ce_forward(xd, wd, td, gd, temperature=t)
    want.check_forward(what, loss, stats)
    dx, dw = m.linear_ce_backward(xd, wd, td, want.stats().to(d), gd, temperature=t)
    want.check_backward(what, dx, dw)
    return loss, stats, dx, dw


@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_linear_ce(mxq_lib, shape):
    for n, (t, ignored, weighted) in enumerate([(1.0, 0.0, False), (0.7, 0.3, True), (2.0, 0.9, True)]):
        say("linear ce", shape, t, ignored)
        x, w, targets, weight = case(*shape, seed=3 + n, ignored=ignored)
        run_both(mxq_lib, x, w, targets, weight if weighted else None, t)


@pytest.mark.parametrize("shape", [(3, 64, 100), (70, 160, 700), (300, 288, 1031)], ids=str)
def test_placement(mxq_lib, shape):
    """Leading dimensions and starts: x and dx at any element, w and dw at any 16 bytes; what
    lies around the outputs stays."""
    rows, hidden, vocab = shape
    x, w, targets, weight = case(*shape, seed=11, ignored=0.2)
    want = HeadLoss(x, w, targets, weight, 1.0)
    td, gd, sd = targets.to(dev()), weight.to(dev()), want.stats().to(dev())
    for pad, shift, pad_w, shift_w in ((0, 1, 0, 8), (3, 0, 8, 0), (5, 7, 40, 16), (8, 8, 0, 0), (64, 0, 8, 8)):
        say("placement", shape, pad, shift)
        xd, _ = placed(x, pad, shift)
        wd, _ = placed(w, pad_w, shift_w)
        loss, stats = mxq_lib.linear_ce_forward(xd, wd, td, gd)
        want.check_forward((shape, pad), loss, stats)
        dx, bx = placed(torch.full(x.shape, NAN, dtype=BF16), pad, shift)
        dw, bw = placed(torch.full(w.shape, NAN, dtype=BF16), pad_w, shift_w)
        mxq_lib.linear_ce_backward(xd, wd, td, sd, gd, dx=dx, dw=dw)
        want.check_backward((shape, pad), dx, dw)
        assert untouched(dx, bx) and untouched(dw, bw)


def test_one_gradient(mxq_lib):
    x, w, targets, weight = case(90, 96, 300, 5, 0.1)
    want = HeadLoss(x, w, targets, weight, 1.0)
    args = [v.to(dev()) for v in (x, w, targets, want.stats(), weight)]
    both = mxq_lib.linear_ce_backward(*args)
    dx, none = mxq_lib.linear_ce_backward(*args, dw=False)
    assert none is None and torch.equal(dx, both[0])
    none, dw = mxq_lib.linear_ce_backward(*args, dx=False)
    assert none is None and torch.equal(dw, both[1])


@pytest.mark.parametrize("rows", [1, 40, 300])
def test_nothing_counts(mxq_lib, rows):
    x, w, targets, weight = case(rows, 64, 333, 7)
    x[:] = NAN
    for targets, weight in ((torch.full_like(targets, -1), None), (targets, torch.zeros_like(weight))):
        loss, stats, dx, dw = run_both(mxq_lib, x, w, targets, weight, 1.0)
        assert not loss.any() and not dx.any() and not dw.any()
        assert torch.equal(stats.cpu(), torch.tensor([[0.0, 1.0]]).expand(rows, 2))


def test_no_rows(mxq_lib):
    d = dev()
    x, w = torch.empty(0, 64, dtype=BF16, device=d), torch.randn(70, 64, device=d).to(BF16)
    t = torch.empty(0, dtype=torch.int32, device=d)
    loss, stats = mxq_lib.linear_ce_forward(x, w, t)
    assert loss.shape == (0,) and stats.shape == (0, 2)
    dw = torch.full((70, 64), NAN, dtype=BF16, device=d)
    dx, dw = mxq_lib.linear_ce_backward(x, w, t, stats, dw=dw)
    assert dx.shape == (0, 64) and not dw.any()


@pytest.mark.parametrize("rows", [9, 290])
def test_rows_that_are_ignored_may_hold_anything(mxq_lib, rows):
    x, w, targets, weight = case(rows, 96, 515, 13, 0.3)
    weight[rows // 2] = 0
    out = (targets < 0) | (weight == 0)
    want = HeadLoss(x, w, targets, weight, 1.0)
    clean = run_both(mxq_lib, x, w, targets, weight, 1.0, want)
    n = out.nonzero()[:, 0]
    x[n[::2]], x[n[1::2]] = NAN, INF
    dirty = run_both(mxq_lib, x, w, targets, weight, 1.0, want)
    for a, b in zip(clean, dirty):
        assert torch.equal(a, b)


@pytest.mark.parametrize("rows", [6, 280])
def test_rows_without_a_distribution(mxq_lib, rows):
    """NaN and +inf logits, and a target beyond the vocabulary, stay in their row (and in dw)."""
    d = dev()
    x, w, targets, _ = case(rows, 64, 300, 17)
    want = HeadLoss(x, w, targets, None, 1.0)
    bad = [1, rows - 2, rows - 1]
    x[bad[0], 5] = NAN
    x[bad[1], 7] = INF
    targets[bad[2]] = 300
    loss, stats = mxq_lib.linear_ce_forward(x.to(d), w.to(d), targets.to(d))
    dx, dw = mxq_lib.linear_ce_backward(x.to(d), w.to(d), targets.to(d), stats)
    good = torch.ones(rows, dtype=torch.bool)
    good[bad] = False
    assert loss.cpu()[bad].isnan().all() and stats.cpu()[bad[:2], 1].isnan().all() and dx.cpu()[bad].isnan().all()
    assert dw.isnan().all()
    import row_refs as ref
    ref.check("loss", loss.cpu()[good], want.loss[good], want.d_loss[good])
    ref.check("sum", stats.cpu()[good, 1], want.s[good], want.d_s[good])
    ref.check("dx", dx.cpu()[good], want.dx[good], want.d_dx[good])


@pytest.mark.parametrize("rows", [3, 200])
@pytest.mark.parametrize("hidden,at", [(32, 0), (32, 31), (96, 95), (64, 63), (160, 130)])
def test_masked_logits(mxq_lib, rows, hidden, at):
    """-inf and +inf in w, also where a step of the product goes on behind a row of it."""
    d = dev()
    x = torch.ones(rows, hidden).to(BF16)
    w = torch.zeros(300, hidden).to(BF16)
    w[::3, at] = -INF
    targets = torch.arange(rows, dtype=torch.int32) * 3 % 300 + 1
    loss, stats = mxq_lib.linear_ce_forward(x.to(d), w.to(d), targets.to(d))
    assert stats.cpu().tolist() == [[0.0, 200.0]] * rows
    assert torch.allclose(loss.cpu(), torch.log(torch.tensor(200.0)).expand(rows), rtol=1e-6)
    dw = mxq_lib.linear_ce_backward(x.to(d), w.to(d), targets.to(d), stats, dx=False)[1].float().cpu()
    assert not dw[::3].any() and (dw[2::3] > 0).all()
    w[0, at] = INF
    loss, stats = mxq_lib.linear_ce_forward(x.to(d), w.to(d), targets.to(d))
    assert loss.isnan().all() and stats[:, 1].isnan().all()


@pytest.mark.parametrize("rows", [3, 40, 200])
@pytest.mark.parametrize("vocab", [33, 64, 321])
def test_masked_target_behind_a_step(mxq_lib, rows, vocab):
    """The vocabulary's last entry is masked by an infinity in w and is row 0's target: its dx there is
    -1 times that infinity, the others' 0 times it."""
    d = dev()
    x = torch.ones(rows, 64).to(BF16)
    w = torch.zeros(vocab, 64).to(BF16)
    w[vocab - 1, 5] = -INF
    targets = torch.zeros(rows, dtype=torch.int32)
    targets[0] = vocab - 1
    loss, stats = mxq_lib.linear_ce_forward(x.to(d), w.to(d), targets.to(d))
    dx, _ = mxq_lib.linear_ce_backward(x.to(d), w.to(d), targets.to(d), stats, dw=False)
    loss, dx = loss.cpu(), dx.float().cpu()
    assert loss[0] == INF and loss[1:].isfinite().all()
    assert dx[0, 5] == INF and dx[1:, 5].isnan().all()
    dx[:, 5] = 0
    assert not dx.any()


def test_masked_vocabulary(mxq_lib):
    """Logits of -inf: masked entries have q = 0; a row with nothing else has loss +inf, S = 0 and the
    gradient -weight / T at its target."""
    d = dev()
    x = torch.ones(3, 32).to(BF16)
    x[1] = 2
    w = torch.zeros(300, 32).to(BF16)
    w[::2, 0] = -INF
    targets = torch.tensor([1, 3, 0], dtype=torch.int32)
    loss, stats = mxq_lib.linear_ce_forward(x.to(d), w.to(d), targets.to(d))
    want = torch.log(torch.tensor(150.0))
    assert torch.allclose(loss[:2].cpu(), want.expand(2), rtol=1e-6) and loss[2].item() == INF
    assert stats.cpu().tolist() == [[0.0, 150.0]] * 3
    w[:, 0] = -INF
    loss, stats = mxq_lib.linear_ce_forward(x.to(d), w.to(d), targets.to(d))
    assert loss.cpu().tolist() == [INF] * 3 and stats.cpu().tolist() == [[-INF, 0.0]] * 3
    w[:] = 0
    weight = torch.tensor([1.0, 2.0, 4.0])
    _, dw = mxq_lib.linear_ce_backward(x.to(d), w.to(d), targets.to(d), torch.tensor([[-INF, 0.0]] * 3).to(d),
                                       weight.to(d), temperature=0.5)
    # q = 0: only the targets' rows of dw, -weight / T x
    exact = torch.zeros(300, 32)
    exact[1], exact[3], exact[0] = -2.0, -8.0, -8.0
    assert torch.equal(dw.float().cpu(), exact)


def test_gradient_against_differences(mxq_lib):
    """The change of the loss along random directions of x and w, by central differences in 64 bits."""
    x, w, targets, weight = case(40, 64, 129, 23, 0.2)
    t = 0.8
    loss, stats, dx, dw = run_both(mxq_lib, x, w, targets, weight, t)
    g = torch.Generator().manual_seed(1)

    def total(x, w):
        z = x @ w.t() / t
        keep = (targets >= 0).nonzero()[:, 0]
        return -(weight.double()[keep] * z.log_softmax(1)[keep, targets[keep].long()]).sum()
    x, w = x.double(), w.double()
    for value, grad, at in ((x, dx, lambda v: total(v, w)), (w, dw, lambda v: total(x, v))):
        for _ in range(4):
            # of one sign with the gradient, so that nothing cancels: every element off by less than 2^-6 of
            # itself or of the gradient's root mean square
            u = torch.rand(value.shape, generator=g, dtype=torch.float64) * grad.double().cpu().sign()
            e = 1e-4
            slope = (at(value + e * u) - at(value - e * u)) / (2 * e)
            got = (grad.double().cpu() * u).sum()
            rms = grad.double().square().mean().sqrt().item()
            assert abs(got - slope) <= 2.0 ** -6 * (got.abs() + rms * u.abs().sum()), (got, slope)


@pytest.mark.parametrize("weight,t", [(1 + 2.0 ** -8, 1.0), (1 / 1351, 0.7), (-3.0, 2.0)])
def test_rounding_is_not_the_same_for_all(mxq_lib, weight, t):
    """With all weights alike, dx and dw are not off by one factor.  Their best factor against the formulas
    is an average of the roundings: of dz over 600 rows, each at most 2^-8 / sqrt(3) of itself in the root
    mean square, and of the many more stored values; seven deviations of both are below 2^-8 / 3.  (Halfway
    between two bf16 numbers, 1 + 2^-8 alone would put them all off by 2^-8.)"""
    x, w, targets, _ = case(600, 128, 1031, 43)
    weight = torch.full((600,), weight)
    want = HeadLoss(x, w, targets, weight, t)
    _, _, dx, dw = run_both(mxq_lib, x, w, targets, weight, t, want)
    for got, exact in ((dx, want.dx), (dw, want.dw)):
        factor = (got.double().cpu() * exact).sum() / exact.square().sum()
        assert abs(factor - 1) <= 2.0 ** -8 / 3, factor


def test_weights_that_are_no_numbers(mxq_lib):
    """The first row's weight says nothing about the others': it may be NaN, infinite, subnormal or huge."""
    d = dev()
    x, w, targets, weight = case(70, 64, 300, 47)
    want = HeadLoss(x, w, targets, weight, 1.0)
    import row_refs as ref
    for first in (NAN, INF, 1e-42, 3e38, -1e-30):
        weight[0] = first
        dx, _ = mxq_lib.linear_ce_backward(x.to(d), w.to(d), targets.to(d), want.stats().to(d), weight.to(d))
        ref.check(("dx", first), dx[1:], want.dx[1:], want.d_dx[1:])


def test_repeats_and_graph(mxq_lib):
    """The same bits each time, and from a replayed graph, between eager calls on other data."""
    d = dev()
    x, w, targets, weight = [v.to(d) for v in case(300, 160, 700, 29, 0.2)]
    x2, w2, targets2, weight2 = [v.to(d) for v in case(300, 160, 700, 31, 0.4)]

    def both(x, w, targets, weight):
        loss, stats = mxq_lib.linear_ce_forward(x, w, targets, weight)
        return (loss, stats, *mxq_lib.linear_ce_backward(x, w, targets, stats, weight))
    first, second = both(x, w, targets, weight), both(x2, w2, targets2, weight2)
    again = both(x, w, targets, weight)
    assert all(torch.equal(a, b) for a, b in zip(first, again))
    held = [v.clone() for v in (x, w, targets, weight)]
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        both(*held)
    torch.cuda.current_stream().wait_stream(stream)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = both(*held)
    for data, want in (((x, w, targets, weight), first), ((x2, w2, targets2, weight2), second),
                       ((x, w, targets, weight), first)):
        for h, v in zip(held, data):
            h.copy_(v)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want))
        assert all(torch.equal(a, b) for a, b in zip(both(x2, w2, targets2, weight2), second))


def test_other_stream(mxq_lib):
    d = dev()
    x, w, targets, weight = [v.to(d) for v in case(100, 96, 400, 37, 0.2)]
    loss, stats = mxq_lib.linear_ce_forward(x, w, targets, weight)
    dx, dw = mxq_lib.linear_ce_backward(x, w, targets, stats, weight)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    loss2, stats2 = mxq_lib.linear_ce_forward(x, w, targets, weight, stream=s)
    dx2, dw2 = mxq_lib.linear_ce_backward(x, w, targets, stats2, weight, stream=s)
    s.synchronize()
    for a, b in ((loss, loss2), (stats, stats2), (dx, dx2), (dw, dw2)):
        assert torch.equal(a, b)
