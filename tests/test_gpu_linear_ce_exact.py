"""mxq_linear_ce_* on data whose every sum is exact in fp32 in any order, so that one row, one entry of the
vocabulary or one hidden value lost or counted twice shows at any size: at sizes that take every form of the
kernels, with pieces of the vocabulary, and with fewer rows that count than there are.

x lives in the first half of the hidden values and w in the second, so that all logits are 0: S is the
size of the vocabulary and the loss its logarithm.  The backward pass is given S = 256 whatever the
vocabulary is: dz is then 2^-8, and 2^-8 - 1 at the target, both exact in bf16, and with integers of up to 3
in x and w every sum of dx and dw is a multiple of 2^-8 below 2^16: exact in fp32, rounded once to bf16.
A logit that is not 0 is tested by one integer in each row's target: z = 1, 2 or 3 there."""
import math
import os

import pytest
import torch

import row_refs as ref
from gpuhelp import dev, say

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16

# rows, hidden, vocab: tiles of 128 x 32; 128 x 128 once and twice a CU; 128 x 256; 256 x 256, and of dw
SHAPES = [(1, 64, 1), (1, 4096, 700), (20, 160, 4099), (32, 96, 33000), (33, 64, 130), (64, 512, 8193), (65, 352, 5000),
          (128, 160, 32768), (100, 96, 33001), (128, 288, 40000), (129, 64, 257), (300, 96, 5000), (513, 1024, 1000),
          (130, 128, 33000), (1500, 64, 12345), (2600, 544, 4111), (900, 2048, 9001), (257, 8192, 300)]


def integers(shape, seed, most=3):
    g = torch.Generator(device=dev()).manual_seed(seed)
    return torch.randint(-most, most + 1, shape, generator=g, device=dev()).to(BF16)


def case(rows, hidden, vocab, seed, ignored):
    """x, w, targets (some < 0), with all logits 0."""
    half = hidden // 2
    x, w = torch.zeros(rows, hidden, dtype=BF16, device=dev()), torch.zeros(vocab, hidden, dtype=BF16, device=dev())
    x[:, :half] = integers((rows, half), seed)
    w[:, half:] = integers((vocab, hidden - half), seed + 1)
    g = torch.Generator(device=dev()).manual_seed(seed + 2)
    targets = torch.randint(vocab, (rows,), generator=g, device=dev(), dtype=torch.int32)
    targets[torch.rand(rows, generator=g, device=dev()) < ignored] = -1
    return x, w, targets


def given(rows):
    return torch.tensor([[0.0, 256.0]], device=dev()).expand(rows, 2).contiguous()


def gradients(x, w, targets):
    """dx and dw by the formulas, in fp64 on the GPU, rounded to bf16."""
    keep = (targets >= 0).nonzero()[:, 0]
    t = targets[keep].long()
    dx = torch.zeros_like(x, dtype=torch.float64)
    dx[keep] = w.double().sum(0) / 256 - w.double()[t]
    dw = (x.double()[keep].sum(0) / 256).expand(w.shape).clone()
    dw.index_add_(0, t, -x.double()[keep])
    return dx.to(BF16), dw.to(BF16)


def check_forward(m, x, w, targets):
    vocab = w.shape[0]
    counts = targets >= 0
    loss, stats = m.linear_ce_forward(x, w, targets)
    assert torch.equal(stats[counts], torch.tensor([0.0, float(vocab)], device=dev()).expand(int(counts.sum()), 2))
    assert torch.equal(stats[~counts], torch.tensor([0.0, 1.0], device=dev()).expand(int((~counts).sum()), 2))
    # the logarithm is good to an ulp or two, and the same for every row
    assert torch.unique(loss[counts]).numel() <= 1 and not loss[~counts].any()
    if counts.any():
        assert abs(loss[counts][0].item() - math.log(vocab)) <= 4 * ref.U * (math.log(vocab) + 1)


@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_exact(mxq_lib, shape):
    for ignored in (0.0, 0.4):
        say("exact", shape, ignored)
        x, w, targets = case(*shape, seed=5, ignored=ignored)
        check_forward(mxq_lib, x, w, targets)
        dx, dw = mxq_lib.linear_ce_backward(x, w, targets, given(shape[0]))
        want = gradients(x, w, targets)
        assert torch.equal(dx, want[0]), (shape, (dx != want[0]).nonzero()[:4].tolist())
        assert torch.equal(dw, want[1]), (shape, (dw != want[1]).nonzero()[:4].tolist())


@pytest.mark.parametrize("rows", [600, 4096])
@pytest.mark.parametrize("count", [1, 31, 64, 257])
def test_few_rows_count(mxq_lib, rows, count):
    """The rows that count are few, and anywhere; how many the kernels learn on the GPU."""
    x, w, targets = case(rows, 288, 3001, 7, 0.0)
    g = torch.Generator().manual_seed(count)
    out = torch.ones(rows, dtype=torch.bool)
    out[torch.randperm(rows, generator=g)[:count]] = False
    targets[out.to(dev())] = -7
    say("few rows count", rows, count)
    check_forward(mxq_lib, x, w, targets)
    dx, dw = mxq_lib.linear_ce_backward(x, w, targets, given(rows))
    want = gradients(x, w, targets)
    assert torch.equal(dx, want[0]) and torch.equal(dw, want[1])


@pytest.mark.parametrize("shape", [(20, 96, 700), (100, 160, 1031), (300, 96, 1500), (700, 512, 769)], ids=str)
def test_pieces(mxq_lib, monkeypatch, shape):
    """The library built for pieces of 256 of the vocabulary: dx grows over several of them."""
    from fp4_microscaling_quantization_amd import build
    assert os.path.exists(build.LOOP_LIB), "libmxq_loop.so is not built"
    x, w, targets = case(*shape, seed=11, ignored=0.3)
    want = gradients(x, w, targets)
    say("pieces", shape)
    with monkeypatch.context() as p:
        p.setattr(mxq_lib, "LIB_PATH", build.LOOP_LIB)
        p.setattr(mxq_lib, "_lib", None)
        dx, dw = mxq_lib.linear_ce_backward(x, w, targets, given(shape[0]))
        torch.cuda.synchronize()
    assert torch.equal(dx, want[0]) and torch.equal(dw, want[1])


@pytest.mark.parametrize("shape", [(9, 64, 300), (128, 96, 1000), (300, 64, 5000), (1500, 64, 12345)], ids=str)
def test_target_logits(mxq_lib, shape):
    """One integer logit in each row, at its target: the loss knows it, and no other."""
    rows, hidden, vocab = shape
    targets = torch.arange(rows, device=dev(), dtype=torch.int32) * 7919 % vocab
    first = torch.unique(targets.long(), return_inverse=True)[1]
    x, w = torch.zeros(rows, hidden, dtype=BF16, device=dev()), torch.zeros(vocab, hidden, dtype=BF16, device=dev())
    z = (first % 3 + 1).to(BF16)
    # row r is 1 at a hidden value of its target's class, whose weight there is the logit
    w[targets.long(), 5] = z
    x[:, 5] = 1
    # ... which all other rows see too: their sums have every target's entry
    loss, stats = mxq_lib.linear_ce_forward(x, w, targets)
    logits = w[:, 5].double()
    s = (logits - logits.max()).exp().sum()
    assert (stats[:, 0] == logits.max().float()).all()
    ref.check("sum", stats[:, 1], s.expand(rows).cpu(), (s * (vocab / 64 + 64) * ref.U).expand(rows).cpu())
    want = (s.log() + logits.max() - z.double()).cpu()
    ref.check("loss", loss, want, (vocab / 64 + 64) * ref.U * (want.abs() + 4))
