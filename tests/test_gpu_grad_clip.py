"""mxq_grad_norm and mxq_grad_clip against the formulas in 64 bits: lists from one
element to hundreds of tensors, mixed types, tensors at any element, values
whose squares leave fp32, non-finite ones, in place and elsewhere, replayed
graphs.

Integers up to 64 have squares whose sums are exact in fp64 in any order: sum_sq
is compared for equality there, so an element lost or counted twice shows.
With u = 2^-24, norm is off by u (its rounding) and c g by 3 u (c, the product and
max_norm / eps as fp32 numbers), then half a step of out's type; below the normal
numbers a step is 2^-149."""
import pytest
import torch

import row_refs as ref
from gpuhelp import dev, say

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
INF, NAN = float("inf"), float("nan")
EPS = 2.0 ** -20

LISTS = {
    "one": [1], "seven": [7], "empty ones": [0, 3, 0, 0, 9, 0], "around a chunk": [4095, 4096, 4097, 8192, 8193],
    "a batch": [5 + i % 9 for i in range(128)], "a batch and one": [300 - i for i in range(129)],
    "three batches": [(i * 37) % 5000 + 1 for i in range(300)], "long": [1_000_003, 64, 2_000_001],
    "longer chunks": [40_000_001, 17],
}


def integers(sizes, dtype, seed):
    g = torch.Generator(device=dev()).manual_seed(seed)
    return [torch.randint(-64, 65, (n,), generator=g, device=dev()).to(dtype) for n in sizes]


def squares(grads):
    return sum(g.double().square().sum() for g in grads)


def check_norm(what, norm, sum_sq, grads):
    want = squares(grads)
    assert sum_sq.item() == want.item(), (what, sum_sq.item(), want.item())
    ref.check((what, "norm"), norm, want.sqrt(), want.sqrt() * ref.U)


def check_clip(what, grads, out, max_norm, eps=EPS):
    norm = squares(grads).sqrt().item()
    c = min(1.0, max_norm / (norm + eps)) if norm + eps > 0 else NAN
    for g, o in zip(grads, out):
        want = g.double() * c
        bound = 3 * ref.U * want.abs() + 2.0 ** -149 if c < 1 else 0 * want
        ref.check((what, c), o, want, ref.store(o.dtype, want, bound))


@pytest.mark.parametrize("name", LISTS)
@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
def test_norm_and_clip(mxq_lib, name, dtype):
    say("grad", name, dtype)
    grads = integers(LISTS[name], dtype, 3)
    norm, sum_sq = mxq_lib.grad_norm(grads)
    check_norm(name, norm, sum_sq, grads)
    for out_dtype in (F32, BF16):
        out = [torch.full_like(g, NAN, dtype=out_dtype) for g in grads]
        mxq_lib.grad_clip(grads, sum_sq, 2.5, eps=EPS, out=out)
        check_clip((name, out_dtype), grads, out, 2.5)
        # nothing to clip: the values themselves
        mxq_lib.grad_clip(grads, sum_sq, 1e9, eps=EPS, out=out)
        assert all(torch.equal(o, g.to(out_dtype)) for g, o in zip(grads, out))
    kept = [g.clone() for g in grads]
    assert mxq_lib.clip_grad_norm(grads, 1e9, eps=EPS).item() == norm.item()
    assert all(torch.equal(a, b) for a, b in zip(grads, kept))
    assert mxq_lib.clip_grad_norm(grads, 2.5, eps=EPS).item() == norm.item()
    check_clip((name, "in place"), kept, grads, 2.5)


def test_mixed_types_and_places(mxq_lib):
    """fp32 and bf16 in one list, each at an odd element of a buffer whose rest stays."""
    d = dev()
    bufs, grads, outs = [], [], []
    for i, n in enumerate([3, 4099, 17, 70_001, 1, 8, 33]):
        dtype, out_dtype = (F32, BF16)[i % 2], (F32, BF16)[i // 2 % 2]
        g = torch.full((n + 40,), 7.0, dtype=dtype, device=d)
        o = torch.full((n + 40,), 9.0, dtype=out_dtype, device=d)
        g[1 + i:1 + i + n] = integers([n], dtype, i)[0]
        bufs.append((g, o, 1 + i, n))
        grads.append(g[1 + i:1 + i + n])
        outs.append(o[11 - i:11 - i + n])
    norm, sum_sq = mxq_lib.grad_norm(grads)
    check_norm("mixed", norm, sum_sq, grads)
    mxq_lib.grad_clip(grads, sum_sq, 1.5, eps=EPS, out=outs)
    check_clip("mixed", grads, outs, 1.5)
    for i, (g, o, at, n) in enumerate(bufs):
        assert (g[:at] == 7).all() and (g[at + n:] == 7).all()
        assert (o[:11 - i] == 9).all() and (o[11 - i + n:] == 9).all()


def test_shapes_and_orders(mxq_lib):
    """Matrices, a transposed one (dense in memory), a scalar; views that skip memory are refused."""
    d = dev()
    a, b, c = integers([60 * 70], F32, 1)[0].view(60, 70), integers([31 * 9], BF16, 2)[0].view(31, 9).t(), torch.tensor(3.0, device=d)
    grads = [a, b, c]
    check_norm("shapes", *mxq_lib.grad_norm(grads), grads)
    kept = [g.clone() for g in grads]
    mxq_lib.clip_grad_norm(grads, 1.0, eps=EPS)
    check_clip("shapes", kept, grads, 1.0)
    with pytest.raises(ValueError):
        mxq_lib.grad_norm([a[:, ::2]])
    with pytest.raises(ValueError):
        mxq_lib.clip_grad_norm([a, c, a], 1.0, eps=EPS)
    with pytest.raises(ValueError):
        mxq_lib.clip_grad_norm([b], 1.0, eps=EPS, out=[torch.empty(9, 31, dtype=BF16, device=d)])
    with pytest.raises(ValueError):
        mxq_lib.grad_norm([a.double()])
    # a gradient may be counted twice
    assert mxq_lib.grad_norm([a, a])[1].item() == 2 * squares([a]).item()


@pytest.mark.parametrize("scale", [2.0 ** 90, 2.0 ** 110, 2.0 ** -100, 2.0 ** -140])
def test_range(mxq_lib, scale):
    """Squares beyond fp32's range, and a factor below its normal numbers."""
    grads = [g * scale for g in integers([500, 4100], F32, 9)]
    want = squares(grads)
    norm, sum_sq = mxq_lib.grad_norm(grads)
    assert sum_sq.item() == want.item() and abs(norm.item() / want.sqrt().item() - 1) <= 2 * ref.U + 2.0 ** -149 / want.sqrt().item()
    for max_norm in (2.0 ** -60, 2.0 ** -20, 1.0):
        out = [torch.empty_like(g) for g in grads]
        mxq_lib.grad_clip(grads, sum_sq, max_norm, eps=0, out=out)
        check_clip((scale, max_norm), grads, out, max_norm, 0.0)


def test_not_finite(mxq_lib):
    for bad, c in ((INF, 0.0), (-INF, 0.0), (NAN, NAN)):
        grads = integers([300, 5000], F32, 5)
        grads[1][77] = bad
        norm, sum_sq = mxq_lib.grad_norm(grads)
        assert (norm.isnan() and sum_sq.isnan()) if bad != bad else (norm.item() == INF and sum_sq.item() == INF)
        want = [g * c for g in grads]
        mxq_lib.clip_grad_norm(grads, 1.0, eps=EPS)
        for g, w in zip(grads, want):
            assert torch.equal(g.isnan(), w.isnan()) and torch.equal(g.nan_to_num(), w.nan_to_num())


def test_largest_norm_of_zero(mxq_lib):
    grads = integers([300, 5000], BF16, 5)
    mxq_lib.clip_grad_norm(grads, 0, eps=EPS)
    assert not any(g.any() for g in grads)
    mxq_lib.clip_grad_norm(grads, 1, eps=0)      # a norm of 0 is not over it
    assert not any(g.any() for g in grads)
    mxq_lib.clip_grad_norm(grads, 0, eps=0)      # 0 / 0
    assert all(g.isnan().all() for g in grads)


def test_parts_of_a_norm(mxq_lib):
    """Ranks that hold a part each: their sums added, every part clipped by the whole norm."""
    a, b = integers([700, 3], F32, 1), integers([5000], F32, 2)
    total = mxq_lib.grad_norm(a)[1] + mxq_lib.grad_norm(b)[1]
    assert total.item() == squares(a + b).item()
    out = [torch.empty_like(g) for g in a + b]
    mxq_lib.grad_clip(a, total, 3.0, eps=EPS, out=out[:2])
    mxq_lib.grad_clip(b, total, 3.0, eps=EPS, out=out[2:])
    check_clip("parts", a + b, out, 3.0)


def test_prepared_streams_and_graph(mxq_lib):
    """A prepared call follows its gradients' values, on whichever stream is current, and in a graph that is
    replayed between eager calls."""
    sizes = [(i * 53) % 3000 + 1 for i in range(150)]
    first, second = integers(sizes, F32, 1), integers(sizes, F32, 2)
    grads = [g.clone() for g in first]
    out = [torch.empty_like(g, dtype=BF16) for g in grads]
    call = mxq_lib.prepare_clip_grad_norm(grads, 2.0, eps=EPS, out=out)
    measure = mxq_lib.prepare_grad_norm(grads)

    def load(values):
        for g, v in zip(grads, values):
            g.copy_(v)

    def check(what, norm):
        ref.check((what, "norm"), norm, squares(grads).sqrt(), squares(grads).sqrt() * ref.U)
        check_clip(what, grads, out, 2.0)
    check("eager", call())
    load(second)
    check("again", call())
    check_norm("measure", *measure(), grads)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        load(first)
        norm = call()
    s.synchronize()
    check("stream", norm)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        norm = call()
    for values in (second, first, second):
        load(values)
        graph.replay()
        torch.cuda.synchronize()
        check("graph", norm)
        assert mxq_lib.grad_norm(first)[1].item() == squares(first).item()
