"""mxq_linear_ce_backward refuses a dx or dw that shares memory with another tensor of the call, before any launch, and
takes columns of one buffer that lie between each other."""
import pytest
import torch

from gpuhelp import dev
from test_gpu_linear_ce import case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows", [9, 300])
def test_shared_outputs(mxq_lib, rows):
    x, w, targets, weight = [v.to(dev()) for v in case(rows, 64, 500, 3, 0.1)]
    loss, stats = mxq_lib.linear_ce_forward(x, w, targets, weight)
    want = mxq_lib.linear_ce_backward(x, w, targets, stats, weight)
    kept = x.clone(), w.clone()
    for name, out in (("dx", x), ("dw", w), ("dx", w[:rows]), ("dx", x.view(rows, 64))):
        with pytest.raises(ValueError, match=f"{name}: in the same memory"):
            mxq_lib.linear_ce_backward(x, w, targets, stats, weight, **{name: out})
    assert torch.equal(x, kept[0]) and torch.equal(w, kept[1])
    both = torch.zeros(500, 192, dtype=torch.bfloat16, device=dev())
    both[:, :64] = w
    dx, dw = mxq_lib.linear_ce_backward(x, both[:, :64], targets, stats, weight, dw=both[:, 64:128], dx=both[:rows, 128:])
    assert torch.equal(dx, want[0]) and torch.equal(dw, want[1]) and torch.equal(both[:, :64], w)
