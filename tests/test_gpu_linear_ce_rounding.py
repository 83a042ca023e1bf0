"""mxq_linear_ce_backward: what the rounding of dz to bf16 leaves in the gradients.  It is added back for the entry
at a row's target, the largest of most rows, so that neither dx nor dw is off by its rounding, whatever
the weights are; and one row's weight has no part in another row's dx."""
import pytest
import torch

import row_refs as ref
from ce_refs import H, HeadLoss
from gpuhelp import dev, say
from test_gpu_linear_ce import case

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16
INF, NAN = float("inf"), float("nan")

# rows, hidden, vocab: dw in one step, in tiles of 128 x 128 (one, two on a CU) and of 256 x 256
SHAPES = [(3, 64, 300), (64, 544, 1000), (33, 1024, 515), (100, 288, 2500), (65, 2080, 4200), (300, 64, 1031),
          (700, 736, 777), (600, 2144, 4200)]


class TargetsKept(HeadLoss):
    """HeadLoss whose bound leaves out the rounding of dz at the targets: what is left of it there is rounded once
    more, to bf16, in the product with x."""

    def __init__(self, x, w, targets, weight=None, t=1.0):
        k = (targets >= 0).nonzero()[:, 0] if weight is None else ((targets >= 0) & (weight != 0)).nonzero()[:, 0]
        self.one = torch.zeros(len(k), w.shape[0], dtype=torch.bool).scatter_(1, targets[k].long()[:, None], True)
        self.calls = 0
        super().__init__(x, w, targets, weight, t)

    def _bound(self, dz, d_dz, other, value):
        one = (self.one, self.one.t())[self.calls]
        self.calls += 1
        n = dz.shape[1]
        rest, at = torch.where(one, 0.0, dz), torch.where(one, dz, 0.0).abs()
        rounding = 4 * H * ((rest * rest) @ (other * other)).sqrt() + 2.0 ** -133 * other.abs().sum(0) + H * H * (at @ other.abs())
        more = (d_dz * (1 + H)) @ other.abs() + (n / 8 + 32) * 2 * ref.U * (dz.abs() @ other.abs())
        return ref.store(BF16, value, rounding + more)


def backward(m, x, w, targets, want, weight, t=1.0):
    d = dev()
    return m.linear_ce_backward(x.to(d), w.to(d), targets.to(d), want.stats().to(d), weight.to(d), temperature=t)


def spread(rows, hidden, vocab, seed):
    """A case whose distributions are wide: logits of about 1/4, so that no other entry is near a target's."""
    x, w, targets, weight = case(rows, hidden, vocab, seed, 0.1)
    return x, (w.float() / 16).to(BF16), targets, weight


@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_targets(mxq_lib, shape):
    say("targets", shape)
    for t in (1.0, 0.7):
        x, w, targets, weight = spread(*shape, seed=3)
        want = TargetsKept(x, w, targets, weight, t)
        want.check_backward((shape, t), *backward(mxq_lib, x, w, targets, want, weight, t))


@pytest.mark.parametrize("rows,hidden,vocab,used", [(64, 96, 300, 1), (200, 64, 300, 3), (1500, 96, 5, 5), (9000, 32, 700, 1),
                                                    (5000, 160, 257, 257)])
def test_many_rows_of_one_target(mxq_lib, rows, hidden, vocab, used):
    """More rows with their target in a tile of dw than one step of their product takes."""
    say("one target", rows, vocab, used)
    x, w, targets, weight = spread(rows, hidden, vocab, seed=5)
    targets = torch.where(targets < 0, targets, vocab - 1 - targets % used)
    want = TargetsKept(x, w, targets, weight)
    want.check_backward((rows, vocab), *backward(mxq_lib, x, w, targets, want, weight))


@pytest.mark.parametrize("first,others", [(1.0, 1 + 2.0 ** -8), (1.0, 1 + 3 * 2.0 ** -8), (0.3, 1 / 600), (1 / 600, 0.3)])
def test_weights_of_two_kinds(mxq_lib, first, others):
    """The rows of either kind are not off by one factor (see test_rounding_is_not_the_same_for_all in
    test_gpu_linear_ce.py for the bound), whichever kind comes first."""
    x, w, targets, _ = case(600, 128, 1031, 43)
    weight = torch.full((600,), others)
    weight[0] = first
    want = HeadLoss(x, w, targets, weight)
    dx, dw = backward(mxq_lib, x, w, targets, want, weight)
    for got, exact in ((dx[1:], want.dx[1:]), (dw, want.dw)):
        factor = (got.double().cpu() * exact).sum() / exact.square().sum()
        assert abs(factor - 1) <= 2.0 ** -8 / 3, factor


@pytest.mark.parametrize("shape", [(9, 64, 300), (70, 64, 300), (300, 96, 1031)], ids=str)
def test_a_row_knows_no_other_weight(mxq_lib, shape):
    x, w, targets, weight = case(*shape, seed=47)
    want = HeadLoss(x, w, targets, weight)
    dx = backward(mxq_lib, x, w, targets, want, weight)[0]
    for first in (0.3, 1.5, -2.0, 1e-42, 3e38, INF, NAN):
        weight[0] = first
        assert torch.equal(backward(mxq_lib, x, w, targets, want, weight)[0][1:], dx[1:]), first


@pytest.mark.parametrize("rows", [5, 90, 300])
def test_infinities_at_targets(mxq_lib, rows):
    """Nothing is added to an infinity: neither where w is one at a target, nor where x is one in a row whose
    logits it masks."""
    d, hidden, vocab = dev(), 64, 300
    x, w = torch.ones(rows, hidden).to(BF16), torch.ones(vocab, hidden).to(BF16)
    targets = torch.arange(rows, dtype=torch.int32) % 7
    x[1, 5] = -INF
    weight = torch.full((rows,), 1 / 3)
    loss, stats = mxq_lib.linear_ce_forward(x.to(d), w.to(d), targets.to(d), weight.to(d))
    assert stats[1].tolist() == [-INF, 0.0] and loss[1].item() == INF
    dx, dw = mxq_lib.linear_ce_backward(x.to(d), w.to(d), targets.to(d), stats, weight.to(d))
    # row 1 is -1/3 at its target and 0 elsewhere
    assert dw[1, 5].item() == INF and dw[:, 5].isnan().sum() == vocab - 1
    assert dw[:, :5].isfinite().all() and dw[:, 6:].isfinite().all()
    assert torch.equal(dx[1].float().cpu(), torch.full((hidden,), -1 / 3).to(BF16).float())
    x[1, 5] = 1
    w[2, 9] = -INF
    _, stats = mxq_lib.linear_ce_forward(x.to(d), w.to(d), targets.to(d), weight.to(d))
    dx, dw = mxq_lib.linear_ce_backward(x.to(d), w.to(d), targets.to(d), stats, weight.to(d))
    at = targets == 2
    assert (dx[:, 9].cpu()[at] == INF).all() and dx[:, 9].cpu()[~at].isnan().all()
    dx[:, 9] = 0
    assert dx.isfinite().all() and dw.isfinite().all()


def test_repeats(mxq_lib):
    """The same bits each time, with many rows to a target."""
    x, w, targets, weight = case(3000, 96, 257, 51)
    targets[::3] = 7
    want = HeadLoss(x, w, targets, weight)
    first = backward(mxq_lib, x, w, targets, want, weight)
    for _ in range(3):
        again = backward(mxq_lib, x, w, targets, want, weight)
        assert all(torch.equal(a, b) for a, b in zip(first, again))
