"""CPU checks of the ends of a training step (cross entropy of an output layer, gradient norm and
clipping): the entry points refuse bad arguments with the documented status before any launch, the
binding refuses tensors that the entry points cannot see through, and the 64-bit reference agrees
with an independent route."""
import ctypes as C

import pytest
import torch

from ce_refs import HeadLoss

A, B, D, E, F = 0x10000, 0x20000, 0x30000, 0x40000, 0x50000   # addresses that nothing reads
NAN, INF = float("nan"), float("inf")


def ce_refusals(m, f):
    for t in (0.0, -1.0, NAN, INF, 1e-40):
        assert f(t=t) == m.ERR_UNSUPPORTED
    assert f(rows=-1) == f(rows=(1 << 22) + 1) == f(vocab=0) == f(vocab=-5) == f(vocab=(1 << 24) + 1) == m.ERR_SHAPE
    assert f(rows=1 << 20, vocab=(1 << 17) + 1) == f(rows=1 << 62, vocab=1 << 62) == m.ERR_SHAPE
    assert f(hidden=0) == f(hidden=48) == f(hidden=-32) == f(ldx=95) == f(ldw=95) == m.ERR_SHAPE
    assert f(hidden=(1 << 16) + 32, ldx=1 << 20, ldw=1 << 20, lddx=1 << 20, lddw=1 << 20) == f(ldw=(1 << 22) + 8) == m.ERR_SHAPE
    assert f(x=None) == f(w=None) == f(targets=None) == m.ERR_NULL
    assert f(x=A + 1) == f(w=B + 8) == f(ldw=100) == f(targets=D + 2) == f(weight=D + 1) == m.ERR_ALIGN


def test_linear_ce_forward_refusals(mxq_lib):
    m, L = mxq_lib, mxq_lib.lib()
    need = L.mxq_linear_ce_forward_workspace_size(4, 96, 100)
    assert need > 0
    for bad in ((-1, 96, 100), (0, 96, 100), (4, 95, 100), (4, 0, 100), (4, 96, 0), (4, 96, 1 << 31), (1 << 31, 96, 100), (1 << 20, 96, 1 << 18), (4, 1 << 17, 100)):
        assert L.mxq_linear_ce_forward_workspace_size(*bad) == 0

    def f(x=A, ldx=96, w=B, ldw=96, rows=4, hidden=96, vocab=100, t=1.0, targets=D, weight=None, loss=E, stats=F, ws=A, size=need, **_):
        return L.mxq_linear_ce_forward(x, ldx, w, ldw, rows, hidden, vocab, t, targets, weight, loss, stats, ws, size, None)
    ce_refusals(m, f)
    assert f(loss=None) == f(stats=None) == m.ERR_NULL
    assert f(loss=E + 2) == f(stats=F + 4) == f(ws=A + 8) == m.ERR_ALIGN
    assert f(ws=None) == f(size=need - 1) == f(size=0) == m.ERR_WORKSPACE
    assert f(rows=0) == f(rows=0, x=None, targets=None, loss=None, stats=None, ws=None, size=0) == m.OK


def test_linear_ce_backward_refusals(mxq_lib):
    m, L = mxq_lib, mxq_lib.lib()
    need = L.mxq_linear_ce_backward_workspace_size(4, 96, 100)
    assert need > 0 and L.mxq_linear_ce_backward_workspace_size(0, 96, 100) > 0
    for bad in ((-1, 96, 100), (4, 95, 100), (4, 0, 100), (4, 96, 0), (4, 96, 1 << 31)):
        assert L.mxq_linear_ce_backward_workspace_size(*bad) == 0

    def f(x=A, ldx=96, w=B, ldw=96, rows=4, hidden=96, vocab=100, t=1.0, targets=D, weight=None, stats=E, dx=F, lddx=96,
          dw=A, lddw=96, ws=A, size=need):
        return L.mxq_linear_ce_backward(x, ldx, w, ldw, rows, hidden, vocab, t, targets, weight, stats, dx, lddx, dw, lddw,
                                        ws, size, None)
    ce_refusals(m, f)
    assert f(lddx=95) == f(lddw=95) == f(lddw=(1 << 22) + 8) == m.ERR_SHAPE
    assert f(stats=None) == f(dx=None, dw=None) == m.ERR_NULL
    assert f(stats=E + 4) == f(dx=F + 1) == f(dw=A + 8) == f(lddw=100) == f(ws=A + 8) == m.ERR_ALIGN
    assert f(ws=None) == f(size=need - 1) == f(size=0) == m.ERR_WORKSPACE
    assert f(rows=0, dw=None) == f(rows=0, dw=None, dx=None, x=None, targets=None, stats=None, ws=None, size=0) == m.OK


def grads_of(m, *entries):
    return (m.Grad * max(1, len(entries)))(*[m.Grad(*e) for e in entries]), len(entries)


def test_grad_norm_refusals(mxq_lib):
    m, L = mxq_lib, mxq_lib.lib()

    def f(*entries, norm=D, sum_sq=E, ws=F, size=1 << 20, count=None):
        arr, n = grads_of(m, *entries)
        return L.mxq_grad_norm(arr, n if count is None else count, norm, sum_sq, ws, size, None)
    good = (A, None, 100, 0, 0)
    assert L.mxq_grad_norm_workspace_size(*grads_of(m, good)) == 8
    assert L.mxq_grad_norm_workspace_size(*grads_of(m, good, (B, None, 0, 1, 0), (B, None, 10, 1, 0))) == 16
    assert L.mxq_grad_norm_workspace_size(*grads_of(m)) == L.mxq_grad_norm_workspace_size(None, 0) == 0
    assert L.mxq_grad_norm_workspace_size(None, 1) == L.mxq_grad_norm_workspace_size(*grads_of(m, (A, None, -1, 0, 0))) == 0
    assert f(good, count=-1) == f((A, None, -1, 0, 0)) == f((A, None, 1 << 49, 0, 0)) == f(good, (A, None, 1 << 48, 0, 0)) == m.ERR_SHAPE
    assert f((A, None, 5, 2, 0)) == f((A, None, 0, -1, 0)) == m.ERR_UNSUPPORTED
    assert f((None, None, 5, 0, 0)) == f(good, norm=None, sum_sq=None) == L.mxq_grad_norm(None, 1, D, E, F, 8, None) == m.ERR_NULL
    assert f((A + 2, None, 5, 0, 0)) == f((A + 1, None, 5, 1, 0)) == f(good, norm=D + 2) == f(good, sum_sq=E + 4) == f(good, ws=F + 4) == m.ERR_ALIGN
    assert f(good, ws=None) == f(good, size=7) == f(good, (B, None, 10, 1, 0), size=8) == m.ERR_WORKSPACE


def test_most_elements(mxq_lib):
    """Above any memory, and within what a launch counts its workgroups in."""
    m, L = mxq_lib, mxq_lib.lib()
    most = 1 << 38
    assert L.mxq_grad_norm_workspace_size(*grads_of(m, (A, None, most, 1, 0))) == 8 * (most // 32768)
    for list_ in [((A, None, most + 1, 1, 0),), ((A, None, most, 0, 0), (B, None, 1, 0, 0))]:
        arr, n = grads_of(m, *list_)
        assert L.mxq_grad_norm_workspace_size(arr, n) == 0
        assert L.mxq_grad_norm(arr, n, D, E, F, 1 << 40, None) == m.ERR_SHAPE


def test_grad_clip_refusals(mxq_lib):
    m, L = mxq_lib, mxq_lib.lib()

    def f(*entries, sum_sq=E, most=1.0, eps=1e-6, count=None):
        arr, n = grads_of(m, *entries)
        return L.mxq_grad_clip(arr, n if count is None else count, sum_sq, most, eps, None)
    good = (A, B, 100, 0, 1)
    assert f(good, count=-1) == f((A, B, -1, 0, 0)) == m.ERR_SHAPE
    assert f((A, B, 5, 0, 2)) == f((A, B, 5, 3, 0)) == f((A, A, 5, 0, 1)) == m.ERR_UNSUPPORTED
    for v in (-1.0, NAN, INF):
        assert f(good, most=v) == f(good, eps=v) == m.ERR_UNSUPPORTED
    assert f((A, None, 5, 0, 0)) == f((None, B, 5, 0, 0)) == f(good, sum_sq=None) == m.ERR_NULL
    assert f((A, B + 2, 5, 0, 0)) == f((A, B + 1, 5, 0, 1)) == f(good, sum_sq=E + 4) == m.ERR_ALIGN
    # nothing to do
    assert f() == f((A, B, 0, 0, 0), (None, None, 0, 1, 1)) == L.mxq_grad_clip(None, 0, E, 1.0, 0.0, None) == m.OK


def test_binding_refuses_what_it_cannot_pass_on(mxq_lib):
    m = mxq_lib
    x, w = torch.zeros(4, 64, dtype=torch.bfloat16), torch.zeros(9, 64, dtype=torch.bfloat16)
    t = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError, match="GPU"):
        m.linear_ce_forward(x, w, t)
    with pytest.raises(ValueError, match="GPU"):
        m.linear_ce_backward(x, w, t, torch.zeros(4, 2))
    with pytest.raises(ValueError, match="GPU"):
        m.grad_norm([x])
    with pytest.raises(ValueError, match="no gradients"):
        m.grad_norm([])
    with pytest.raises(ValueError, match="same memory"):
        m._grad_list([x, w, x])
    with pytest.raises(ValueError, match="2 outputs"):
        m._grad_list([x], [x, w])
    with pytest.raises(ValueError, match="output 0"):
        m._grad_list([x], [torch.zeros(64, 4, dtype=torch.bfloat16)])
    with pytest.raises(ValueError, match="dense"):
        m._grad_list([x[:, ::2]])
    with pytest.raises(ValueError, match="dense"):
        m._grad_list([x[:1].expand(4, 64)])
    with pytest.raises(ValueError, match="float32 or bfloat16"):
        m._grad_list([x.double()])
    arr, _ = m._grad_list([x, w.float(), x], write=False)
    assert [(a.g, a.out, a.n, a.dtype, a.out_dtype) for a in arr][0] == (x.data_ptr(), x.data_ptr(), 256, 1, 1)
    assert arr[1].dtype == 0 and arr[2].g == arr[0].g


def test_reference_agrees_with_autograd():
    g = torch.Generator().manual_seed(3)
    x = torch.randn(9, 32, generator=g).bfloat16()
    w = (torch.randn(50, 32, generator=g) / 4).bfloat16()
    targets = torch.randint(50, (9,), generator=g, dtype=torch.int32)
    targets[2] = -1
    weight = torch.rand(9, generator=g)
    weight[5] = 0
    want = HeadLoss(x, w, targets, weight, 0.7)
    xd, wd = x.double().requires_grad_(), w.double().requires_grad_()
    loss = torch.nn.functional.cross_entropy(xd @ wd.t() / 0.7, targets.long(), reduction="none", ignore_index=-1) * weight.double()
    loss.sum().backward()
    assert torch.allclose(loss.detach(), want.loss, rtol=1e-12, atol=0)
    assert torch.allclose(xd.grad, want.dx, rtol=1e-10, atol=1e-14) and torch.allclose(wd.grad, want.dw, rtol=1e-10, atol=1e-14)
