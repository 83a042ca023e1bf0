"""CPU checks of the row operators (norm, token log probabilities, distillation):
the entry points refuse bad arguments with the documented status before any
launch, the binding refuses tensors that the entry points cannot see through,
and the 64-bit references agree with an independent route."""
import ctypes as C

import pytest
import torch

import row_refs as ref

A, B, D, E = 0x10000, 0x20000, 0x30000, 0x40000   # addresses that nothing reads
NAN, INF = float("nan"), float("inf")


def test_norm_forward_refusals(mxq_lib):
    m, L = mxq_lib, mxq_lib.lib()

    def f(kind=0, x=A, xt=1, ldx=64, rows=4, cols=64, g=None, b=None, eps=1e-5, y=B, yt=1, ldy=64, mean=None, rstd=None):
        return L.mxq_norm_forward(kind, x, xt, ldx, rows, cols, g, b, eps, y, yt, ldy, mean, rstd, None)
    assert f(kind=2) == f(kind=-1) == f(xt=2) == f(yt=-1) == m.ERR_UNSUPPORTED
    assert f(eps=-1.0) == f(eps=NAN) == f(eps=INF) == m.ERR_UNSUPPORTED
    assert f(rows=-1) == f(cols=0) == f(cols=1 << 31, ldx=1 << 32, ldy=1 << 32) == f(ldx=63) == f(ldy=63) == m.ERR_SHAPE
    assert f(x=None) == f(y=None) == m.ERR_NULL
    assert f(x=A + 1) == f(y=B + 1) == f(xt=0, x=A + 2) == f(g=D + 2) == f(b=D + 2) == f(mean=D + 1) == f(rstd=D + 2) == m.ERR_ALIGN
    assert f(rows=0) == f(rows=0, x=None, y=None) == m.OK


def test_norm_backward_refusals(mxq_lib):
    m, L = mxq_lib, mxq_lib.lib()
    need = L.mxq_norm_backward_workspace_size(4, 64)
    assert need > 0 and L.mxq_norm_backward_workspace_size(-1, 64) == 0 and L.mxq_norm_backward_workspace_size(4, 0) == 0

    def f(kind=0, dy=A, dt=1, ldd=64, x=B, xt=1, ldx=64, rows=4, cols=64, g=None, mean=D, rstd=D, dx=E, ot=1, ldo=64,
          dg=A, db=A, ws=B, size=need):
        return L.mxq_norm_backward(kind, dy, dt, ldd, x, xt, ldx, rows, cols, g, mean, rstd, dx, ot, ldo, dg, db, ws, size, None)
    assert f(kind=3) == f(dt=2) == f(xt=2) == f(ot=2) == m.ERR_UNSUPPORTED
    assert f(rows=-1) == f(cols=0) == f(ldd=63) == f(ldx=63) == f(ldo=63) == m.ERR_SHAPE
    assert f(dy=None) == f(x=None) == f(rstd=None) == f(mean=None) == m.ERR_NULL
    assert f(dy=A + 1) == f(x=B + 1) == f(dx=E + 1) == f(g=D + 2) == f(dg=A + 2) == f(db=A + 1) == f(ws=B + 2) == m.ERR_ALIGN
    assert f(ws=None) == f(size=need - 1) == f(dg=None, size=0) == f(db=None, ws=None) == m.ERR_WORKSPACE
    # nothing to do: no dx and no sums, or no rows and no sums
    assert f(rows=0, dg=None, db=None, ws=None) == m.OK
    assert f(dx=None, dg=None, db=None, ws=None, size=0) == m.OK


def logits_refusals(m, f):
    assert f(zt=2) == f(zt=-1) == m.ERR_UNSUPPORTED
    for t in (0.0, -1.0, NAN, INF):
        assert f(t=t) == m.ERR_UNSUPPORTED
    assert f(rows=-1) == f(vocab=0) == f(vocab=1 << 31, ld=1 << 32) == f(ld=99) == m.ERR_SHAPE
    assert f(z=None) == m.ERR_NULL
    assert f(z=A + 1) == f(zt=0, z=A + 2) == m.ERR_ALIGN
    assert f(rows=0) == f(rows=0, z=None) == m.OK


def test_token_logprobs_refusals(mxq_lib):
    m, L = mxq_lib, mxq_lib.lib()
    need = L.mxq_vocab_workspace_size(4, 100, 5)

    def f(z=A, zt=1, ld=100, rows=4, vocab=100, t=1.0, tok=B, lp=D, ent=D, st=D, k=5, ids=E, lps=E, ws=B, size=None):
        return L.mxq_token_logprobs(z, zt, ld, rows, vocab, t, tok, lp, ent, st, k, ids, lps, ws, need if size is None else size, None)
    logits_refusals(m, f)
    assert f(k=-1) == f(k=m.TOP_MAX + 1) == m.ERR_UNSUPPORTED
    assert f(tok=None) == f(st=None) == f(ids=None) == f(lps=None) == m.ERR_NULL
    assert f(tok=B + 2) == f(lp=D + 2) == f(ent=D + 1) == f(st=D + 2) == f(ids=E + 2) == f(lps=E + 1) == f(ws=B + 4) == m.ERR_ALIGN
    for rows, vocab, k in ((1, 131072, 0), (4, 131072, 20), (2, 10 ** 6, 64)):
        need = L.mxq_vocab_workspace_size(rows, vocab, k)
        if need:
            assert f(rows=rows, vocab=vocab, ld=vocab, k=k, size=need - 1) == m.ERR_WORKSPACE
            assert f(rows=rows, vocab=vocab, ld=vocab, k=k, ws=None, size=need) == m.ERR_WORKSPACE
    assert L.mxq_vocab_workspace_size(-1, 100, 5) == L.mxq_vocab_workspace_size(4, 0, 5) == L.mxq_vocab_workspace_size(4, 100, 65) == 0


def test_token_logprobs_backward_refusals(mxq_lib):
    m, L = mxq_lib, mxq_lib.lib()

    def f(z=A, zt=1, ld=100, rows=4, vocab=100, t=1.0, tok=B, st=D, ent=D, gl=D, gh=D, o=E, ot=1, ldo=100):
        return L.mxq_token_logprobs_backward(z, zt, ld, rows, vocab, t, tok, st, ent, gl, gh, o, ot, max(ldo, 0) if ldo != 100 else max(100, vocab), None)
    logits_refusals(m, f)
    assert f(ot=2) == m.ERR_UNSUPPORTED and f(ldo=99) == m.ERR_SHAPE
    assert f(st=None) == f(tok=None) == f(ent=None) == f(o=None) == m.ERR_NULL
    assert f(tok=B + 2) == f(st=D + 2) == f(ent=D + 2) == f(gl=D + 2) == f(gh=D + 2) == f(o=E + 1) == m.ERR_ALIGN


@pytest.mark.parametrize("entry", ["forward", "backward", "both"])
def test_distill_refusals(mxq_lib, entry):
    m, L = mxq_lib, mxq_lib.lib()

    def f(z=A, zt=1, ld=100, rows=4, vocab=100, t=1.0, ids=B, lps=D, k=5, renorm=1, w=D, loss=E, st=E, o=E, ot=1, ldo=None, ws=B, size=1 << 40):
        ldo = max(100, vocab) if ldo is None else ldo
        head = (z, zt, ld, rows, vocab, t, ids, lps, k, renorm, w)
        if entry == "forward":
            return L.mxq_distill_forward(*head, loss, st, ws, size, None)
        if entry == "backward":
            return L.mxq_distill_backward(*head, st, o, ot, ldo, None)
        return L.mxq_distill(*head, loss, o, ot, ldo, ws, size, None)
    logits_refusals(m, f)
    assert f(k=0) == f(k=65) == f(renorm=2) == f(renorm=-1) == m.ERR_UNSUPPORTED
    assert f(ids=None) == f(lps=None) == m.ERR_NULL
    assert f(ids=B + 2) == f(lps=D + 1) == f(w=D + 2) == m.ERR_ALIGN
    if entry != "backward":
        assert f(loss=None) == m.ERR_NULL and f(loss=E + 2) == f(ws=B + 4) == m.ERR_ALIGN
        need = L.mxq_vocab_workspace_size(1, 131072, 0)
        if need:
            assert f(rows=1, vocab=131072, ld=131072, size=need - 1) == m.ERR_WORKSPACE
    if entry != "both":
        assert f(st=None) == m.ERR_NULL and f(st=E + 2) == m.ERR_ALIGN
    if entry != "forward":
        assert f(ot=2) == m.ERR_UNSUPPORTED and f(ldo=99) == m.ERR_SHAPE
        assert f(o=None) == m.ERR_NULL and f(o=E + 1) == m.ERR_ALIGN


def test_binding_refuses_what_the_entry_points_cannot_see(mxq_lib):
    m = mxq_lib
    x = torch.zeros((4, 8))
    assert m._matrix("x", x)[1:] == (m.OUT_F32, 8)
    assert m._matrix("x", torch.zeros((4, 9), dtype=torch.bfloat16)[:, :8])[1:] == (m.OUT_BF16, 9)
    assert m._matrix("x", x[:1])[2] == 8 and m._matrix("x", x[:, :1])[2] == 8
    for bad in (x.t(), x[:, ::2], x[:1].expand(3, 8), x.half(), x.double(), x.int(), x[0], x[None]):
        with pytest.raises(ValueError):
            m._matrix("x", bad)
    with pytest.raises(ValueError):
        m._matrix("out", torch.zeros((4, 7)), x)
    assert m._vector("v", None, (4,), x) is None
    v = torch.zeros(8)
    assert m._vector("v", v, (8,), x) == v.data_ptr()
    for bad in (v[::2], v.double(), v[:3], v.int(), v[:4].bfloat16(), torch.zeros((4, 1))):
        with pytest.raises(ValueError):
            m._vector("v", bad, (4,), x)
    with pytest.raises(ValueError):
        m.norm_forward(x, eps=1e-5)               # not on a GPU
    with pytest.raises(ValueError):
        m.token_logprobs(x)
    with pytest.raises(TypeError):
        m.norm_forward(x)                         # eps has to be said


def test_references_against_autograd():
    """The formulas of row_refs against automatic differentiation in 64 bits."""
    g = torch.Generator().manual_seed(1)
    x = torch.randn(5, 33, generator=g, dtype=torch.float64, requires_grad=True)
    gamma = torch.randn(33, generator=g, dtype=torch.float64, requires_grad=True)
    beta = torch.randn(33, generator=g, dtype=torch.float64, requires_grad=True)
    dy = torch.randn(5, 33, generator=g, dtype=torch.float64)
    y = torch.nn.functional.layer_norm(x, (33,), gamma, beta, 1e-5)
    y.backward(dy)
    ry, mean, rstd, *_ = ref.norm(x.detach(), gamma.detach(), beta.detach(), 1e-5, True)
    got = ref.norm_backward(dy, x.detach(), gamma.detach(), mean, rstd, True)
    assert torch.allclose(ry, y.detach(), atol=1e-12)
    for a, b in zip(got, (x.grad, gamma.grad, beta.grad)):
        assert torch.allclose(a, b, atol=1e-11)
    x.grad = None
    z = (3 * torch.randn(5, 40, generator=g, dtype=torch.float64)).requires_grad_()
    tok = torch.randint(0, 40, (5,), generator=g)
    gl, gh = torch.randn(5, generator=g, dtype=torch.float64), torch.randn(5, generator=g, dtype=torch.float64)
    lq = (z / 1.7).log_softmax(1)
    ent = -(lq.exp() * lq).sum(1)
    ((lq.gather(1, tok[:, None])[:, 0] * gl).sum() + (ent * gh).sum()).backward()
    d = ref.Distribution(z.detach(), 1.7)
    assert torch.allclose(d.logq, lq.detach(), atol=1e-12) and torch.allclose(d.entropy, ent.detach(), atol=1e-12)
    assert torch.allclose(ref.logprobs_backward(d, tok, d.entropy, gl, gh)[0], z.grad, atol=1e-12)
    z.grad = None
    ids = torch.randint(0, 40, (5, 6), generator=g).int()
    ids[2, 3] = -1
    ids[1, 1] = ids[1, 0]
    lps = torch.randn(5, 6, generator=g, dtype=torch.float64)
    w = torch.randn(5, generator=g, dtype=torch.float64)
    for renorm in (True, False):
        z.grad = None
        lp = lps.masked_fill(ids < 0, -INF)
        lp = lp.log_softmax(1) if renorm else lp
        p = lp.exp()
        lq = (z / 1.7).log_softmax(1)
        terms = p * (lp.masked_fill(ids < 0, 0.0) - lq.gather(1, ids.long().clamp(min=0)))
        loss = w * 1.7 * 1.7 * terms.sum(1)
        loss.sum().backward()
        rl, rz, *_ = ref.distill(ref.Distribution(z.detach(), 1.7), ids, lps, w, renorm)
        assert torch.allclose(rl, loss.detach(), atol=1e-12) and torch.allclose(rz, z.grad, atol=1e-12)


def test_structs_unchanged(mxq_lib):
    """The new entry points take plain arguments only: the structures keep their sizes."""
    assert C.sizeof(mxq_lib.QConfig) == 48 and C.sizeof(mxq_lib.QTensor) == 32
