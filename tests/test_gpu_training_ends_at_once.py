"""The ends of a training step where calls meet: two at once on streams of their own, two
captured graphs replayed in turn, the same tensor twice; and where offsets pass 32 bits."""
import pytest
import torch

from gpuhelp import dev, say
from test_gpu_linear_ce import case

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16
SHAPES = [(20, 96, 1000), (100, 64, 9000), (700, 128, 3000)]


def step(m, x, w, targets, weight, out):
    """Loss, gradients, and the gradients' clipping into new tensors."""
    loss, stats = m.linear_ce_forward(x, w, targets, weight)
    dx, dw = m.linear_ce_backward(x, w, targets, stats, weight)
    norm = m.clip_grad_norm([dx, dw], 0.5, eps=1e-6, out=out)
    return loss, stats, norm, *out


def outputs(x, w):
    return [torch.empty_like(t, dtype=torch.float32) for t in (x, w)]


@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_two_streams(mxq_lib, shape):
    say("two streams", shape)
    d = dev()
    data = [[v.to(d) for v in case(*shape, seed=51 + i, ignored=0.2)] for i in range(2)]
    outs = [outputs(*v[:2]) for v in data]
    want = [[t.clone() for t in step(mxq_lib, *v, o)] for v, o in zip(data, outs)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = [[], []]
    for n in range(4):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append([t.clone() for t in step(mxq_lib, *data[i], outs[i])])
    torch.cuda.synchronize()
    for i in range(2):
        for g in got[i]:
            assert all(torch.equal(a, b) for a, b in zip(g, want[i]))


def test_two_graphs(mxq_lib):
    """Two graphs of one pool, replayed in turn with eager calls between them."""
    say("two graphs")
    d = dev()
    data = [[v.to(d) for v in case(*shape, seed=61, ignored=0.1)] for shape in SHAPES[:2]]
    outs = [outputs(*v[:2]) for v in data]
    want = [[t.clone() for t in step(mxq_lib, *v, o)] for v, o in zip(data, outs)]
    torch.cuda.synchronize()
    graphs, got = [], []
    for v, o in zip(data, outs):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, pool=graphs[0].pool() if graphs else None):
            got.append(step(mxq_lib, *v, o))
        graphs.append(g)
    for n in range(3):
        for i in (0, 1):
            for o in outs[i]:
                o.fill_(7)
            graphs[i].replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(got[i], want[i])), (n, i)
            step(mxq_lib, *data[1 - i], outs[1 - i])
            torch.cuda.synchronize()


def test_the_same_tensor_twice(mxq_lib):
    """A tensor that is listed twice counts twice; it cannot be written twice."""
    g = torch.arange(-50, 51, device=dev(), dtype=torch.float32)
    assert mxq_lib.grad_norm([g, g])[1].item() == 2 * (g.double() ** 2).sum().item()
    with pytest.raises(ValueError):
        mxq_lib.clip_grad_norm([g, g], 1.0, eps=1e-6)
    out = [torch.empty_like(g), torch.empty_like(g)]
    mxq_lib.clip_grad_norm([g, g], 1e9, eps=1e-6, out=out)
    assert torch.equal(out[0], g) and torch.equal(out[1], g)


@pytest.mark.parametrize("rows", [30, 130, 12000])
def test_far_rows(mxq_lib, rows):
    """Leading dimensions of 2^22, the largest: rows of w and dw gigabytes apart, the same bits."""
    say("far rows", rows)
    d, vocab, hidden, ld = dev(), 600, 96, 1 << 22
    x, w, targets, weight = [v.to(d) for v in case(rows, hidden, vocab, 71, 0.1)]
    loss, stats = mxq_lib.linear_ce_forward(x, w, targets, weight)
    dx, dw = mxq_lib.linear_ce_backward(x, w, targets, stats, weight)
    far = torch.empty(vocab, ld, dtype=BF16, device=d)
    far[:, :hidden] = w
    far[:, hidden:hidden + 64] = float("nan")
    far_w = far[:, :hidden]
    got = mxq_lib.linear_ce_forward(x, far_w, targets, weight)
    assert torch.equal(got[0], loss) and torch.equal(got[1], stats)
    far_dw = far[:, hidden + 64:2 * hidden + 64]
    far_dx, _ = mxq_lib.linear_ce_backward(x, far_w, targets, stats, weight, dw=far_dw)
    assert torch.equal(far_dx, dx) and torch.equal(far_dw, dw)
    assert torch.equal(far_w, w) and far[:, hidden:hidden + 64].isnan().all()
