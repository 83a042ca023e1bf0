"""mxq_linear_ce_backward where its plan is large: the largest tiles for dx, several pieces of the vocabulary with
several slabs of dx in the library itself, and every kind of large tile over several pieces in the build whose
pieces are 256 wide.  That the sizes take the kernels they are listed for is tested on the CPU
(test_linear_ce_kernels_host.py)."""
import os

import pytest
import torch

from gpuhelp import dev, say
from test_gpu_linear_ce import case, run_both
from test_gpu_linear_ce_exact import case as exact_case, check_forward, given, gradients
from test_gpu_linear_ce_rounding import TargetsKept, backward, spread

pytestmark = pytest.mark.gpu

# (rows, hidden, vocab): what it is listed for
LARGE = {
    (2600, 544, 4160): dict(dx=("Many", False)),
    (2048, 96, 65700): dict(dx=("Many", True), dz=("Many", True), dw=("Many", False), pieces=2, slabs=32),
    (2048, 64, 65728): dict(dx=("Many", False), dz=("Many", False), dw=("Many", False), pieces=2, slabs=32),
    (20, 64, 600001): dict(dx=("Few", True), dz=("Few", False), dw=("Outer", False), pieces=2),
    (100, 96, 600064): dict(dx=("Twin", False), dz=("Twin", True), dw=("Twin", False), pieces=2),
}
# in the build for pieces of 256
PIECES = {
    (8200, 2048, 576): dict(dx=("Many", False), dz=("Half", False), pieces=3),
    (8200, 2048, 515): dict(dx=("Many", True), pieces=3),
    (130, 33024, 576): dict(dw=("Many", False), dx=("Deep", False), pieces=3),
    (33025, 64, 600): dict(dz=("Many", False), pieces=3),
}
PIECES_ROUNDED = [(20, 96, 700), (100, 160, 1031), (700, 512, 769), (8200, 96, 515)]


@pytest.fixture
def pieces(mxq_lib, monkeypatch):
    from fp4_microscaling_quantization_amd import build
    assert os.path.exists(build.LOOP_LIB), "libmxq_loop.so is not built"
    monkeypatch.setattr(mxq_lib, "LIB_PATH", build.LOOP_LIB)
    monkeypatch.setattr(mxq_lib, "_lib", None)
    yield mxq_lib
    torch.cuda.synchronize()


def check_exact(m, shape):
    x, w, targets = exact_case(*shape, seed=15, ignored=0.1)
    dx, dw = m.linear_ce_backward(x, w, targets, given(shape[0]))
    want = gradients(x, w, targets)
    assert torch.equal(dx, want[0]), (shape, (dx != want[0]).nonzero()[:4].tolist())
    assert torch.equal(dw, want[1]), (shape, (dw != want[1]).nonzero()[:4].tolist())
    return x, w, targets


@pytest.mark.parametrize("shape", LARGE, ids=str)
def test_large(mxq_lib, shape):
    say("large", shape)
    check_forward(mxq_lib, *check_exact(mxq_lib, shape))


def test_large_tiles_of_dx(mxq_lib):
    x, w, targets, weight = case(2600, 544, 4160, seed=33, ignored=0.1)
    run_both(mxq_lib, x, w, targets, weight, 0.7)


@pytest.mark.parametrize("shape", PIECES, ids=str)
def test_pieces(pieces, shape):
    say("pieces", shape)
    check_exact(pieces, shape)


@pytest.mark.parametrize("shape", PIECES_ROUNDED, ids=str)
def test_rounding_over_pieces(pieces, shape):
    """Every row's target is in one piece; what its rounding left is added in that one, to dx behind the last."""
    say("rounding over pieces", shape)
    x, w, targets, weight = spread(*shape, seed=35)
    want = TargetsKept(x, w, targets, weight)
    want.check_backward(shape, *backward(pieces, x, w, targets, want, weight))


def test_rounding_over_pieces_of_the_library(mxq_lib):
    """Two pieces in the library: the gradients of 2048 rows under 65700 entries, of which the first and the last
    2000 have the targets, against the formulas on the GPU, in 64 bits."""
    d, rows, hidden, vocab = dev(), 2048, 64, 65700
    say("rounding over pieces of the library")
    g = torch.Generator(device=d).manual_seed(37)
    x = torch.randn(rows, hidden, generator=g, device=d).bfloat16()
    w = (torch.randn(vocab, hidden, generator=g, device=d) / 64).bfloat16()
    targets = torch.randint(4000, (rows,), generator=g, device=d, dtype=torch.int32)
    targets = torch.where(targets < 2000, targets, targets + (vocab - 4000)).to(torch.int32)
    loss, stats = mxq_lib.linear_ce_forward(x, w, targets)
    weight = torch.full((rows,), 1 + 2.0 ** -8, device=d)
    dx, dw = mxq_lib.linear_ce_backward(x, w, targets, stats, weight)
    z = x.double() @ w.double().t()
    dz = (z - stats[:, :1].double()).exp_().div_(stats[:, 1:].double())
    dz[torch.arange(rows, device=d), targets.long()] -= 1
    dz.mul_(weight.double()[:, None])
    # Off by: the stored values by 2^-8 of theirs, what is not at a target by 2^-8 of itself, what is left at a
    # target by 2^-8 of 2^-8 of it; dz before its rounding by 2^-18 of itself (its logits by 2^-20: 8 instructions of
    # 2^-23 of at most 1), and the fp32 sums as in ce_refs.py.  A target's entry is above 0.99: q is below 2^-12.
    assert stats[:, 1].min() > 2 ** 12 and (x.double().abs() @ w.double().abs().t()).max() < 2
    u, one = 2.0 ** -24, dz.abs().amax(1)[:, None]
    wide, tall, at = w.double(), x.double(), w[targets.long()].double().abs()
    want, reach = dz @ wide, dz.abs() @ wide.abs()
    bound = 2.0 ** -8 * (want.abs() + reach - one * at) + 2.0 ** -16 * one * at + (2.0 ** -18 + (vocab / 8 + 32) * 2 * u) * reach
    assert ((dx.double() - want).abs() <= bound * (1 + 2.0 ** -7)).all()
    want, reach = dz.t() @ tall, dz.abs().t() @ tall.abs()
    at = torch.zeros(vocab, hidden, dtype=torch.float64, device=d).index_add_(0, targets.long(), tall.abs())
    bound = 2.0 ** -8 * (want.abs() + (reach - 0.99 * at).clamp(min=0)) + 2.0 ** -15 * at + (2.0 ** -18 + (rows / 8 + 32) * 2 * u) * reach
    assert ((dw.double() - want).abs() <= bound * (1 + 2.0 ** -7)).all()
