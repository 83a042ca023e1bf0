"""mxq_grad_norm and mxq_grad_clip on lists around the numbers of tensors that a launch takes (32, 256 and 1024),
and over several launches: integers, so that sum_sq is exact in fp64 and a tensor that is lost or counted twice
shows (see test_gpu_grad_clip.py)."""
import pytest
import torch

from gpuhelp import dev, say
from test_gpu_grad_clip import EPS, check_clip, check_norm, integers, squares

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
COUNTS = [31, 32, 33, 255, 256, 257, 1023, 1024, 1025, 2048, 2049, 2500]


def sizes(count):
    """Short tensors of mixed sizes, some of more than one chunk, some empty."""
    return [0 if i % 11 == 5 else 9000 + i if i % 97 == 3 else (i * 37) % 700 + 1 for i in range(count)]


@pytest.mark.parametrize("count", COUNTS)
def test_lists(mxq_lib, count):
    for n, (dtype, out_dtype) in enumerate([(F32, BF16), (BF16, F32)]):
        say("list", count, dtype)
        grads = integers(sizes(count), dtype, 3 + n)
        norm, sum_sq = mxq_lib.grad_norm(grads)
        check_norm(count, norm, sum_sq, grads)
        out = [torch.full_like(g, float("nan"), dtype=out_dtype) for g in grads]
        mxq_lib.grad_clip(grads, sum_sq, 2.5, eps=EPS, out=out)
        check_clip((count, out_dtype), grads, out, 2.5)
        kept = [g.clone() for g in grads]
        assert mxq_lib.clip_grad_norm(grads, 2.5, eps=EPS).item() == norm.item()
        check_clip((count, "in place"), kept, grads, 2.5)


@pytest.mark.parametrize("tensors", [0, 1, 1024, 2500])
def test_tensors_that_count(mxq_lib, tensors):
    """As many tensors with elements as launches take, among empty ones; each element once in the sum."""
    count = max(2500, tensors)
    has = set(range(0, count, count // tensors)[:tensors]) if tensors else set()
    grads = [torch.full((1 if i in has else 0,), float(i % 50 + 1), device=dev()) for i in range(count)]
    norm, sum_sq = mxq_lib.grad_norm(grads)
    assert sum_sq.item() == sum((i % 50 + 1) ** 2 for i in has) == squares(grads)
    mxq_lib.grad_clip(grads, sum_sq, 0, eps=EPS)
    assert not any(g.any() for g in grads)


def test_a_prepared_list_over_several_launches(mxq_lib):
    """And from a graph, replayed between eager calls."""
    first, second = integers(sizes(1500), F32, 1), integers(sizes(1500), F32, 2)
    grads = [g.clone() for g in first]
    out = [torch.empty_like(g, dtype=BF16) for g in grads]
    call = mxq_lib.prepare_clip_grad_norm(grads, 2.0, eps=EPS, out=out)
    check_clip("eager", grads, (call(), out)[1], 2.0)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        norm = call()
    for values in (second, first, second):
        for g, v in zip(grads, values):
            g.copy_(v)
        graph.replay()
        torch.cuda.synchronize()
        assert abs(norm.item() / squares(grads).sqrt().item() - 1) <= 2.0 ** -23
        check_clip("graph", grads, out, 2.0)
        assert mxq_lib.grad_norm(first)[1].item() == squares(first).item()
