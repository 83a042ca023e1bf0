"""mxq_linear_ce_*: a target beyond the vocabulary makes its row's loss and dx NaN, and dw, whatever else the row
holds; also one with every logit masked, whose q is 0."""
import pytest
import torch

from gpuhelp import dev

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16
INF = float("inf")


@pytest.mark.parametrize("rows", [2, 40, 100, 300])
@pytest.mark.parametrize("beyond", [0, 1, 60, 2 ** 31 - 1 - 100])
def test_foreign_target_of_a_masked_row(mxq_lib, rows, beyond):
    d, hidden, vocab = dev(), 64, 100
    x, w = torch.zeros(rows, hidden).to(BF16), torch.ones(vocab, hidden).to(BF16)
    # row 1 has logits of -inf throughout: products of finite values, beyond fp32's lowest
    x[1, 0] = -3e38
    w[:, 0] = 3e38
    targets = torch.arange(rows, dtype=torch.int32) % vocab
    targets[1] = vocab + beyond
    loss, stats = mxq_lib.linear_ce_forward(x.to(d), w.to(d), targets.to(d))
    assert stats[1].tolist() == [-INF, 0.0] and loss.isnan().nonzero()[:, 0].tolist() == [1]
    dx, dw = mxq_lib.linear_ce_backward(x.to(d), w.to(d), targets.to(d), stats)
    assert dx[1].isnan().all() and dw.isnan().all()
    assert dx[0].isfinite().all() and dx[2:].isfinite().all()
