"""mxq_linear_ce_forward and _backward at sizes for each tile of their products: the
smallest sizes that are large enough for the larger tiles."""
import os

import pytest
import torch

from gpuhelp import say
from test_gpu_linear_ce import case, run_both
from test_gpu_linear_ce_exact import case as exact_case, check_forward, given, gradients

pytestmark = pytest.mark.gpu

# rows, hidden, vocab: small tiles over rows that are not packed; few rows; up to 128; more.  A hidden size that ends
# within a step, and one that does not.
SHAPES = [(33, 64, 700), (65, 128, 300), (128, 64, 1000), (20, 96, 16385), (32, 64, 16448), (100, 96, 8321), (70, 64, 8192 + 64), (128, 96, 32833), (100, 64, 33024),
          (200, 96, 8257), (256, 64, 8320), (600, 96, 11077), (530, 64, 11136), (600, 288, 16451), (513, 320, 16512), (700, 288, 23045)]


@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_tiles(mxq_lib, shape):
    say("tiles", shape)
    x, w, targets, weight = case(*shape, seed=31, ignored=0.1)
    run_both(mxq_lib, x, w, targets, weight, 0.7)


@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_tiles_exact(mxq_lib, shape):
    say("tiles exact", shape)
    x, w, targets = exact_case(*shape, seed=6, ignored=0.3)
    check_forward(mxq_lib, x, w, targets)
    dx, dw = mxq_lib.linear_ce_backward(x, w, targets, given(shape[0]))
    want = gradients(x, w, targets)
    assert torch.equal(dx, want[0]) and torch.equal(dw, want[1])


@pytest.mark.parametrize("shape", [(8200, 1120, 515), (40, 96, 1031), (8200, 64, 600)], ids=str)
def test_tiles_of_pieces(mxq_lib, monkeypatch, shape):
    """The library built for pieces of 256 of the vocabulary: dx grows over several of them in large tiles too."""
    from fp4_microscaling_quantization_amd import build
    assert os.path.exists(build.LOOP_LIB), "libmxq_loop.so is not built"
    x, w, targets = exact_case(*shape, seed=12, ignored=0.1)
    want = gradients(x, w, targets)
    say("tiles of pieces", shape)
    with monkeypatch.context() as p:
        p.setattr(mxq_lib, "LIB_PATH", build.LOOP_LIB)
        p.setattr(mxq_lib, "_lib", None)
        dx, dw = mxq_lib.linear_ce_backward(x, w, targets, given(shape[0]))
        torch.cuda.synchronize()
    assert torch.equal(dx, want[0]) and torch.equal(dw, want[1])
