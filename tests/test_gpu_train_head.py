"""examples/train_head.py runs, and its gradients are those of the formulas: an FP4 layer, norm, cross entropy
without logits and clipping, one after the other as a training step uses them."""
import os
import sys

import pytest
import torch

import row_refs as ref
from ce_refs import HeadLoss
from gpuhelp import dev

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


def test_runs(mxq_lib):
    import train_head
    lines = []
    losses = train_head.train(steps=3, tokens=256, features=256, hidden=256, vocab=1000, say=lines.append)
    assert len(losses) == 3 and all(0 < v < 20 for v in losses) and len(lines) == 4


@pytest.mark.parametrize("tokens,hidden,vocab", [(128, 256, 700), (384, 512, 1501)])
def test_gradients(mxq_lib, tokens, hidden, vocab):
    """Each operator's output from the one before it, as it was handed on."""
    import train_head
    m = mxq_lib
    model = train_head.Model(features=256, hidden=hidden, vocab=vocab, max_norm=0.05, seed=3)
    g = torch.Generator(device=dev()).manual_seed(4)
    x = torch.randn(tokens, 256, generator=g, device=dev()).bfloat16()
    targets = torch.randint(vocab, (tokens,), generator=g, device=dev(), dtype=torch.int32)
    targets[5::7] = -1
    weight = torch.full((tokens,), 1.0 / tokens, device=dev())
    loss, h = model.gradients(x, targets, weight)
    du, dgamma, dw = model.du.clone(), model.dgamma.clone(), model.dw.clone()

    y, _, rstd = m.norm_forward(h, model.gamma, eps=1e-5, kind=m.NORM_RMS, out_dtype=torch.bfloat16)
    _, stats = m.linear_ce_forward(y, model.w_used, targets, weight)
    want = HeadLoss(y, model.w_used, targets, weight, 1.0, stats)
    want.check_forward("head", loss, stats)
    dy, _ = m.linear_ce_backward(y, model.w_used, targets, stats, weight, dw=False)
    want.check_backward("head", dy, dw)
    _, wg, _, _, d_wg, _ = ref.norm_backward(dy, h, model.gamma, None, rstd, False)
    ref.check("dgamma", dgamma, wg, d_wg)

    # all of them clipped by one norm
    total = sum(t.double().square().sum() for t in (du, dgamma, dw)).sqrt().item()
    norm = model.clip()
    assert abs(norm.item() / total - 1) <= 2 * ref.U
    c = min(1.0, 0.05 / (total + 1e-6))
    assert c < 1
    for before, after in ((du, model.du), (dgamma, model.dgamma), (dw, model.dw)):
        v = before.double() * c
        ref.check("clipped", after, v, ref.store(after.dtype, v, 3 * ref.U * v.abs() + 2.0 ** -149))
