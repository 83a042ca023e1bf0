"""The rows of exact_rows do what the tests that use them need: sums that fp32 holds in any order,
and bounds that one lost element exceeds."""
import pytest
import torch

import exact_rows as ex


@pytest.mark.parametrize("vocab", [9, 4099, 131075, 300007])
def test_logits_have_exact_sums(vocab):
    z = ex.logits(3, vocab, 1)
    m, s, a = ex.sums(z)
    g = torch.Generator().manual_seed(2)
    order = torch.randperm(vocab, generator=g)
    d = z - m[:, None].float()
    for cut in (16, 1000, vocab):
        e = torch.zeros(3)
        w = torch.zeros(3)
        for at in range(0, vocab, cut):
            e += torch.exp2(d[:, order[at:at + cut]]).sum(1)
            w += (torch.exp2(d[:, order[at:at + cut]]) * d[:, order[at:at + cut]]).sum(1)
        assert torch.equal(e.double(), s) and torch.equal(w.double(), a)
    assert 1.4426950408889634 / ex.TEMPERATURE - 1 < 2.0 ** -24   # 1 in fp32
    assert torch.tensor(ex.TEMPERATURE, dtype=torch.float32).item() == ex.TEMPERATURE
    # the largest element's gradient notices a sum without one of the smallest's eighth neighbours
    ids = torch.zeros((3, 1), dtype=torch.int32)
    dz, bound, hit = ex.gradient(z, ids, s)
    lost, _, _ = ex.gradient(z, ids, s - 0.125)
    assert bool((((lost - dz).abs() > bound) | hit).all())


@pytest.mark.parametrize("cols", [3, 4, 9, 4096, 131077])
def test_balanced_rows(cols):
    x = ex.balanced(5, cols, 1)
    assert x.shape == (5, cols) and not x.sum(1).any() and bool((x != 0).all()) and float(x.abs().max()) <= 3
    square = (x.double() ** 2).sum(1)
    assert float(square.max()) < 2 ** 24
    rstd = (square / cols + 0.5).rsqrt()
    lost = ((square - 1) / cols + 0.5).rsqrt()
    assert bool(((lost - rstd).abs() > 4 * ex.U * rstd).all())


def test_top():
    z = torch.tensor([[0.0, -1, 0, -2, 0], [-6, -6, -6, -6, -6]])
    assert ex.top(z, 4).tolist() == [[0, 2, 4, 1], [0, 1, 2, 3]] and ex.top(z, 7)[0].tolist() == [0, 2, 4, 1, 3, -1, -1]
