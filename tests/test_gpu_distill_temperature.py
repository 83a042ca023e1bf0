"""The distillation loss at temperatures whose square is no fp32 number: the formula
w T^2 sum p (log p - log q) is finite there, and so has the loss to be."""
import pytest
import torch

from gpuhelp import dev, say

pytestmark = pytest.mark.gpu

F32 = torch.float32
U = 2.0 ** -24


def losses(m, z, ids, lps, w, t):
    """The loss of the pass that gives the gradient too, and the loss alone."""
    args = z.to(dev()), ids.to(dev()), lps.to(dev()), w.to(dev())
    both, _ = m.distill(*args, temperature=t, renormalize=False)
    alone, _ = m.distill_forward(*args, temperature=t, renormalize=False)
    return {"both": both.cpu(), "alone": alone.cpu()}


@pytest.mark.parametrize("t", [2.0 ** -100, 1e-24, 3e-21, 1e-3, 1.0, 37.0])
@pytest.mark.parametrize("vocab", [2, 1000, 131072])
def test_small_temperature(mxq_lib, vocab, t):
    """One certain alternative g below the maximum, everything else masked: q = 1 at the
    maximum, log q = -g / T at the alternative (S = 1 + exp(-g / T)), the loss w T^2 (g / T + log S)."""
    say("small temperature", vocab, t)
    t = float(torch.tensor(t, dtype=F32))
    gaps = torch.tensor([0.5, 1.0, 3.0, 100.0])
    z = torch.full((4, vocab), -float("inf"))
    z[:, 0], z[:, vocab - 1] = 1.5, 1.5 - gaps
    ids = torch.full((4, 1), vocab - 1, dtype=torch.int32)
    w = torch.tensor([1.0, -2.0, 0.25, 1.0])
    g = gaps.double() / t
    want = w.double() * t * t * (g + torch.log1p((-g).exp()))
    # of the value: g / T 2 u, log S 6 u, two differences, three products; S itself 4 u, where the
    # value without w T^2 is 0.69 or more: 6 u; an fp32 subnormal's half step
    bound = 20 * U * want.abs() + 2.0 ** -149
    for what, got in losses(mxq_lib, z, ids, torch.zeros(4, 1), w, t).items():
        off = (got.double() - want).abs()
        assert bool((off <= bound).all()), (what, vocab, t, got.tolist(), want.tolist())


@pytest.mark.parametrize("t", [1e20, 1e30, 3e38])
def test_large_temperature(mxq_lib, t):
    """A single logit: q = p = 1, so the loss is T^2 times 0."""
    say("large temperature", t)
    z = torch.tensor([[0.75], [-3.0]])
    for what, got in losses(mxq_lib, z, torch.zeros((2, 1), dtype=torch.int32), torch.zeros(2, 1), torch.ones(2), t).items():
        assert got.tolist() == [0.0, 0.0], (what, t, got)
