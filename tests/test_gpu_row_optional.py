"""Outputs and operands of the row operators that a caller leaves out: what is left has the bits
that it has with them, and buffers that are not named stay as they were."""
import pytest
import torch

from gpuhelp import dev, say
from test_gpu_norm import EPS, placed, rand

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


def stream():
    return torch.cuda.current_stream().cuda_stream


@pytest.mark.parametrize("shape", [(7, 5), (70, 515), (33, 4096), (600, 2048), (40, 9001), (5, 20000)], ids=str)
@pytest.mark.parametrize("kind", ["layer", "rms"])
def test_norm_sums_alone(mxq_lib, kind, shape):
    """mxq_norm_backward without dx: the sums over the rows only."""
    m = mxq_lib
    rows, cols = shape
    code = m.NORM_LAYER if kind == "layer" else m.NORM_RMS
    for dt, xt in ((F32, BF16), (BF16, BF16), (F32, F32)):
        say("norm sums alone", kind, shape, dt, xt)
        x, dy = placed(rand(shape, 1, xt), 3, 1)[0], placed(rand(shape, 2, dt), 2, 3)[0]
        gamma = rand((cols,), 3, offset=1.0).to(dev())
        _, mean, rstd = m.norm_forward(x, gamma, eps=EPS, kind=code)
        _, dg, db = m.norm_backward(dy, x, gamma, mean, rstd, kind=code)
        for want_g, want_b in ((True, True), (True, False), (False, True)):
            got_g, got_b = torch.full((2, cols), 7.0, device=dev())
            size = m.lib().mxq_norm_backward_workspace_size(rows, cols)
            ws = torch.empty(size, dtype=torch.uint8, device=dev())
            status = m.lib().mxq_norm_backward(
                code, dy.data_ptr(), m._dtype(dy), dy.stride(0), x.data_ptr(), m._dtype(x), x.stride(0), rows, cols,
                gamma.data_ptr(), None if mean is None else mean.data_ptr(), rstd.data_ptr(), None, m.OUT_F32, 0,
                got_g.data_ptr() if want_g else None, got_b.data_ptr() if want_b else None, ws.data_ptr(), size, stream())
            assert status == m.OK
            assert torch.equal(got_g, dg if want_g else torch.full_like(dg, 7.0))
            assert torch.equal(got_b, db if want_b else torch.full_like(db, 7.0))


@pytest.mark.parametrize("shape", [(7, 5), (70, 515), (4099, 1024), (3, 9001), (2, 70001)], ids=str)
def test_norm_forward_parts(mxq_lib, shape):
    """Without mean and rstd; beta without gamma, gamma without beta."""
    m = mxq_lib
    rows, cols = shape
    x = placed(rand(shape, 1, BF16), 3, 1)[0]
    ones, zeros = torch.ones(cols, device=dev()), torch.zeros(cols, device=dev())
    gamma, beta = rand((cols,), 3, offset=1.0).to(dev()), rand((cols,), 4).to(dev())
    for code in (m.NORM_LAYER, m.NORM_RMS):
        say("norm parts", shape, code)
        y, _, _ = m.norm_forward(x, gamma, beta, eps=EPS, kind=code, out_dtype=F32)
        out = torch.empty(shape, device=dev())
        assert m.lib().mxq_norm_forward(code, x.data_ptr(), m.OUT_BF16, x.stride(0), rows, cols, gamma.data_ptr(), beta.data_ptr(),
                                        EPS, out.data_ptr(), m.OUT_F32, cols, None, None, stream()) == m.OK
        assert torch.equal(out, y)
        for g, b in ((gamma, None), (None, beta), (None, None)):
            got, _, _ = m.norm_forward(x, g, b, eps=EPS, kind=code, out_dtype=F32)
            want, _, _ = m.norm_forward(x, ones if g is None else g, zeros if b is None else b, eps=EPS, kind=code, out_dtype=F32)
            assert torch.equal(got, want)


@pytest.mark.parametrize("shape", [(3, 6), (2051, 515), (70, 5000), (3, 131072), (520, 50257)], ids=str)
def test_logprobs_parts(mxq_lib, shape):
    """Each output of token log probabilities alone."""
    m = mxq_lib
    rows, vocab = shape
    say("logprobs parts", shape)
    z = placed(rand(shape, 1, BF16, 2.0), 3, 1)[0]
    tokens = (torch.arange(rows, device=dev()) * 31 % vocab).to(torch.int32)
    lp, ent, stats, ids, lps = m.token_logprobs(z, tokens, top_k=9)
    for with_tokens, with_entropy, k in ((True, False, 0), (False, True, 0), (False, False, 0), (False, False, 9), (True, False, 9)):
        got = m.token_logprobs(z, tokens if with_tokens else None, entropy=with_entropy, top_k=k)
        assert len(got) == (5 if k else 3)
        for have, want in zip(got, (lp if with_tokens else None, ent if with_entropy else None, stats, ids, lps)):
            assert (have is None) == (want is None) and (have is None or torch.equal(have, want))
