"""mxq_token_logprobs, mxq_distill_* and their gradients against the formulas in
64 bits: vocabularies from one entry to several workgroups' worth, every type,
rows off the vector alignment, masked entries and rows, non-finite rows, equal
logits, absent, repeated and foreign ids, rows that are ignored."""
import pytest
import torch

import row_refs as ref
from gpuhelp import dev, say
from test_gpu_norm import placed, rand, untouched

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
INF, NAN = float("inf"), float("nan")

SHAPES = [(1, 1), (2, 2), (3, 7), (2, 63), (5, 100), (2, 1000), (70, 515), (3, 4096), (2, 8191), (1, 32003),
          (6, 32768), (3, 50257), (1, 131072), (2, 131075), (1, 160001), (2, 300007)]


def logits_of(shape, seed, dtype, scale=2.5):
    return rand(shape, seed, dtype, scale)


def tokens_of(z, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randint(0, z.shape[1], (z.shape[0],), generator=g, dtype=torch.int32)


def check_logprobs(what, out, z, t, tokens, k, dist=None):
    d = dist or ref.Distribution(z, t)
    lp, ent, stats = out[:3]
    idx = tokens.long()[:, None]
    bad = idx >= z.shape[1]
    pick = torch.where(bad, -1, idx)
    want, bound = d.pick(d.logq, pick, 0.0), d.pick(d.d_logq, pick, 0.0)
    want = torch.where(bad, NAN, want)
    ref.check((what, "logprob"), lp, want[:, 0], bound[:, 0])
    ref.check((what, "entropy"), ent, d.entropy, d.d_entropy)
    ok = ~d.none
    ref.check((what, "max"), stats[:, 0].cpu()[ok], d.m[ok], torch.zeros(int(ok.sum())))
    ref.check((what, "sum"), stats[:, 1], d.s, d.d_s.nan_to_num() * d.s.abs().nan_to_num() + 2 * ref.U * d.s.abs().nan_to_num())
    if k:
        ids = d.top(k)
        assert torch.equal(out[3].cpu().long(), ids), (what, "ids", (out[3].cpu().long() != ids).nonzero()[:4].tolist())
        w, b = d.pick(d.logq, ids, -INF), d.pick(d.d_logq, ids, 0.0)
        w[d.none] = NAN
        ref.check((what, "top"), out[4], w, b)


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
def test_logprobs(mxq_lib, shape, dtype):
    for n, (t, k, pad, shift) in enumerate([(1.0, 0, 0, 0), (0.7, 1, 3, 1), (2.0, 20, 8, 8), (1.0, 64, 1, 3)]):
        say("logprobs", shape, dtype, (t, k, pad, shift))
        z = logits_of(shape, 5 + n, dtype)
        tokens = tokens_of(z, n)
        zd, zb = placed(z, pad, shift)
        out = mxq_lib.token_logprobs(zd, tokens.to(dev()), top_k=k, temperature=t)
        check_logprobs((shape, t, k), out, z, t, tokens, k)
        assert untouched(zd, zb)


def special(vocab, dtype):
    """Rows where a softmax goes wrong, and what each is."""
    z = rand((16, vocab), 3, F32, 2.0)
    low = torch.finfo(dtype).min
    z[1] = -INF                                # every entry masked
    z[2, : vocab - vocab // 8] = -INF          # few left
    z[3] = low                                 # masked by the lowest value, all of it
    z[4, 1::2] = low                           # half of it
    z[5] = 1.5                                 # all equal
    z[6] = z[6].round()                        # many equal
    z[7, vocab // 2] = NAN
    z[8, vocab - 1] = INF
    z[9, 0], z[9, vocab - 1] = -INF, -low      # the largest value there is
    z[10] = 0.0
    z[10, ::2] = -0.0                          # zeros of both signs are equal
    z[11] = torch.arange(vocab).float() / vocab * 8       # rising
    z[12] = -torch.arange(vocab).float() / vocab * 8      # falling
    z[13] = -INF
    z[13, vocab // 3] = -4.0                   # a single one left
    z[14] = NAN
    z[15] = z[15] * 40                         # peaked
    return z.to(dtype)


@pytest.mark.parametrize("vocab", [9, 1000, 32768, 50257, 131072, 200003])
@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
def test_logprobs_special_rows(mxq_lib, vocab, dtype):
    z = special(vocab, dtype)
    tokens = tokens_of(z, 1)
    tokens[0], tokens[5], tokens[6] = -1, vocab, vocab - 1
    tokens[13] = vocab // 3
    for t, k in ((1.0, 64), (2.0, 7)):
        say("logprobs special", vocab, dtype, t, k)
        out = mxq_lib.token_logprobs(z.to(dev()), tokens.to(dev()), top_k=k, temperature=t)
        check_logprobs(("special", vocab, t), out, z, t, tokens, k)


@pytest.mark.parametrize("vocab,rows", [(40000, 2), (131072, 1), (131072, 300)])
def test_top_clustered(mxq_lib, vocab, rows):
    """The largest logits where one thread, one wave or one stretch of the row
    holds them all."""
    for step in (1, 8, 64, 512, 1024, 2048, 4096, 8192, 16384):
        for dtype in (F32, BF16):
            say("clustered", vocab, rows, step, dtype)
            z = rand((1, vocab), step, F32, 0.5)
            at = torch.arange(3, vocab, step)[:200]
            z[0, at] = 20.0 + 4 * rand((len(at),), 9)
            z = z.to(dtype)
            out = mxq_lib.token_logprobs(z.to(dev()).expand(rows, vocab).contiguous(), top_k=64)
            ids = ref.Distribution(z, 1.0).top(64)
            assert out[0] is None
            assert torch.equal(out[3].cpu().long(), ids.expand(rows, 64)), (vocab, step, dtype)


@pytest.mark.parametrize("vocab", [20000, 131072, 300007])
def test_top_stretches(mxq_lib, vocab):
    """Long stretches of large logits, one every few thousand entries: a few
    threads hold far more of them than are asked for; and rows of equal ones."""
    for step, width in ((2048, 128), (4096, 300), (8192, 128), (8192, 1000), (16384, 4096)):
        for dtype in (F32, BF16):
            for equal in (False, True):
                say("stretches", vocab, step, width, dtype, equal)
                z = rand((2, vocab), step, F32, 0.5)
                at = torch.arange(vocab) % step < width
                z[:, at] = 20.0 if equal else 20.0 + 4 * rand((2, int(at.sum())), 9)
                z = z.to(dtype)
                out = mxq_lib.token_logprobs(z.to(dev()), top_k=64)
                assert torch.equal(out[3].cpu().long(), ref.Distribution(z, 1.0).top(64)), (vocab, step, dtype)


@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_logprobs_backward(mxq_lib, shape):
    m = mxq_lib
    rows, vocab = shape
    types = [(F32, BF16), (BF16, BF16), (F32, F32), (BF16, F32)]
    for n, (zt, ot) in enumerate(types):
        pad, shift, t = [(0, 0, 1.0), (3, 1, 0.7), (8, 8, 2.0), (1, 3, 1.0)][n]
        say("logprobs backward", shape, zt, ot, (pad, shift))
        z = logits_of(shape, 15 + n, zt)
        tokens = tokens_of(z, n)
        if rows > 2:
            tokens[1] = -1
        gl, gh = rand((rows,), 1), rand((rows,), 2, scale=0.1)
        _, ent, stats = m.token_logprobs(z.to(dev()), tokens.to(dev()), temperature=t)
        zd, _ = placed(z, pad, shift)
        out, ob = placed(torch.zeros(shape, dtype=ot), pad + 1, shift)
        d = ref.Distribution(z, t, stats)
        for use_l, use_h in ((True, True), (True, False), (False, True)):
            m.token_logprobs_backward(zd, tokens.to(dev()), stats, ent if use_h else None, gl.to(dev()) if use_l else None,
                                      gh.to(dev()) if use_h else None, temperature=t, out=out)
            want, bound = ref.logprobs_backward(d, tokens, ent, gl * use_l, gh * use_h)
            ref.check("dlogits", out, want, ref.store(ot, want, bound))
        assert untouched(out, ob)


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
def test_logprobs_backward_special_rows(mxq_lib, dtype):
    m = mxq_lib
    for vocab in (9, 5000, 131072):
        say("logprobs backward special", vocab, dtype)
        z = special(vocab, dtype)
        tokens = tokens_of(z, 1)
        tokens[0], tokens[5], tokens[6] = -1, vocab, vocab - 1
        gl, gh = rand((16,), 1), rand((16,), 2, scale=0.1)
        zd = z.to(dev())
        _, ent, stats = m.token_logprobs(zd, tokens.to(dev()))
        d = ref.Distribution(z, 1.0, stats)
        out = m.token_logprobs_backward(zd, tokens.to(dev()), stats, ent, gl.to(dev()), gh.to(dev()), out=zd)
        assert out is zd
        want, bound = ref.logprobs_backward(d, tokens, ent, gl, gh)
        ref.check("dlogits", out, want, ref.store(dtype, want, bound))


def teacher_of(z, k, seed, ragged=True):
    """Alternatives of a teacher near the student, some rows with fewer, some
    ids twice, in an order of their own."""
    rows, vocab = z.shape
    zt = z.float().nan_to_num(0.0, 30.0, -30.0).clamp(-30, 30) + rand(z.shape, seed, F32, 0.7)
    g = torch.Generator().manual_seed(seed + 1)
    n = min(k, vocab)
    values, ids = zt.topk(n, 1)
    lps = torch.full((rows, k), -1.0)
    all_ids = torch.full((rows, k), -1, dtype=torch.int32)
    lps[:, :n] = values - zt.logsumexp(1, keepdim=True)
    all_ids[:, :n] = ids.int()
    if ragged:
        gone = torch.rand((rows, k), generator=g) < 0.2
        all_ids[gone] = -1
        lps[torch.rand((rows, k), generator=g) < 0.1] = -INF
        if k > 2:
            all_ids[::3, 2] = all_ids[::3, 0]
    return all_ids, lps


def run_distill(m, z, zd, ids, lps, w, t, renorm, ot, out):
    """All three entry points on one case: checked against 64 bits and each other."""
    args = ids.to(dev()), lps.to(dev())
    wd = None if w is None else w.to(dev())
    loss, stats = m.distill_forward(zd, *args, wd, temperature=t, renormalize=renorm)
    d = ref.Distribution(z, t)
    rl, rz, e_l, e_z = ref.distill(d, ids, lps, w, renorm)
    ref.check("loss", loss, rl, e_l.nan_to_num() + 1e-37)
    dz = m.distill_backward(zd, *args, stats, wd, temperature=t, renormalize=renorm, out_dtype=ot)
    ref.check("backward", dz, rz, ref.store(ot, rz, e_z.nan_to_num()))
    loss2, both = m.distill(zd, *args, wd, temperature=t, renormalize=renorm, out_dtype=ot, out=out)
    ref.check("loss of the pass", loss2, rl, e_l.nan_to_num() + 1e-37)
    ref.check("gradient of the pass", both, rz, ref.store(ot, rz, e_z.nan_to_num()))
    return both


@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_distill(mxq_lib, shape):
    rows, vocab = shape
    for n, (zt, ot) in enumerate([(F32, BF16), (BF16, BF16), (F32, F32), (BF16, F32)]):
        k, t, renorm, pad, shift = [(8, 1.0, True, 0, 0), (64, 2.0, False, 3, 1), (1, 1.0, True, 8, 8), (33, 0.7, False, 1, 3)][n]
        say("distill", shape, zt, ot, (k, t, renorm, pad, shift))
        z = logits_of(shape, 25 + n, zt)
        ids, lps = teacher_of(z, k, n)
        w = rand((rows,), 4)
        if rows > 3:
            w[1] = 0.0
        zd, zb = placed(z, pad, shift)
        out, ob = placed(torch.zeros(shape, dtype=ot), pad + 1, shift)
        run_distill(mxq_lib, z, zd, ids, lps, w if n % 2 else None, t, renorm, ot, out)
        assert untouched(out, ob) and untouched(zd, zb)


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("vocab", [9, 5000, 50257, 131072, 200003])
def test_distill_special_rows(mxq_lib, vocab, dtype):
    z = special(vocab, dtype)
    z = torch.cat([z, z])
    ids, lps = teacher_of(z, 12, 3, ragged=False)
    ids[0] = -1                                     # nothing known
    lps[5] = -INF                                   # nothing probable
    ids[6, 3] = vocab                               # not of this vocabulary
    ids[15, :] = ids[15, 0].clone()                 # one id in every place
    lps[12, 1] = NAN
    w = torch.ones(32)
    w[16:] = 0.0                                    # ignored, whatever they hold
    ids[20, 0] = vocab + 5
    w[4] = -2.0
    for renorm in (True, False):
        say("distill special", vocab, dtype, renorm)
        zd = z.to(dev())
        out = run_distill(mxq_lib, z, zd, ids, lps, w, 1.0, renorm, dtype, None)
        assert not out[16:].any() and not out[0].any() and not out[5].any()
        loss, over = mxq_lib.distill(zd, ids.to(dev()), lps.to(dev()), w.to(dev()), renormalize=renorm, out=zd)
        assert over is zd and torch.equal(over.view(torch.int16 if dtype == BF16 else torch.int32),
                                          out.view(torch.int16 if dtype == BF16 else torch.int32))


def test_cross_entropy_is_a_case(mxq_lib):
    """One certain alternative: -log q and q - 1[v = id]."""
    z = logits_of((50, 777), 1, F32)
    tokens = tokens_of(z, 2)
    say("cross entropy")
    loss, dz = mxq_lib.distill(z.to(dev()), tokens[:, None].to(dev()), torch.zeros((50, 1), device=dev()))
    lp, _, _ = mxq_lib.token_logprobs(z.to(dev()), tokens.to(dev()))
    d = ref.Distribution(z, 1.0)
    idx = tokens.long()[:, None]
    ref.check("loss", loss, -d.logq.gather(1, idx)[:, 0], 2 * d.d_logq.gather(1, idx)[:, 0])
    ref.check("loss and logprob", loss, -lp.double(), 2 * d.d_logq.gather(1, idx)[:, 0])
    want = d.q - torch.nn.functional.one_hot(tokens.long(), 777)
    ref.check("gradient", dz, want, d.d_q + 12 * ref.U * want.abs())


def test_gradients_against_differences(mxq_lib):
    """Central differences of the 64-bit forward passes: with step h they are off
    by h^2 / 6 of the third derivative, under 8 / t^3 of the outer gradients'
    magnitudes here, and by 2^-52 / h of the value."""
    m = mxq_lib
    rows, vocab, t, h = 3, 29, 1.3, 1e-4
    z = logits_of((rows, vocab), 1, F32, 1.0)
    tokens = tokens_of(z, 2)
    ids, lps = teacher_of(z, 6, 3)
    w, gl, gh = rand((rows,), 4), rand((rows,), 5), rand((rows,), 6)
    say("differences over a vocabulary")

    def difference(value):
        want = torch.zeros(rows, vocab, dtype=torch.float64)
        for i in range(rows * vocab):
            for sign in (1, -1):
                moved = z.double().clone()
                moved.view(-1)[i] += sign * h
                want.view(-1)[i] += sign * value(ref.Distribution(moved, t)) / (2 * h)
        return want
    zd = z.to(dev())
    _, ent, stats = m.token_logprobs(zd, tokens.to(dev()), temperature=t)
    got = m.token_logprobs_backward(zd, tokens.to(dev()), stats, ent, gl.to(dev()), gh.to(dev()), temperature=t)
    want = difference(lambda d: (gl.double() * d.logq.gather(1, tokens.long()[:, None])[:, 0]).sum() + (gh.double() * d.entropy).sum())
    _, bound = ref.logprobs_backward(ref.Distribution(z, t, stats), tokens, ent, gl, gh)
    # entropy and S are fp32 values: 4 u of log q + H and 4 u of q more
    more = 8 * h * h / t ** 3 * float((gl.abs() + 4 * gh.abs()).sum()) + 2.0 ** -52 / h * 100 + 60 * ref.U * float(gl.abs().max() + 4 * gh.abs().max())
    ref.check("logprob and entropy", got, want, bound + more)
    for renorm in (True, False):
        _, got = m.distill(zd, ids.to(dev()), lps.to(dev()), w.to(dev()), temperature=t, renormalize=renorm)
        want = difference(lambda d: ref.distill(d, ids, lps, w, renorm)[0].sum())
        _, _, _, bound = ref.distill(ref.Distribution(z, t), ids, lps, w, renorm)
        more = 8 * h * h / t * float(w.abs().sum()) + 2.0 ** -52 / h * 100
        ref.check("distillation", got, want, bound + more)


def test_offsets_past_32_bits(mxq_lib):
    """Rows whose element offsets pass 2^31 and whose byte offsets pass 2^32."""
    m = mxq_lib
    vocab, ld = 3001, (1 << 30) + 3
    z = logits_of((4, vocab), 1, BF16)
    buf = torch.empty(3 * ld + vocab, dtype=BF16, device=dev())
    view = buf.as_strided((4, vocab), (ld, 1))
    view.copy_(z)
    tokens = tokens_of(z, 1)
    say("far rows over a vocabulary")
    check_logprobs("far", m.token_logprobs(view, tokens.to(dev()), top_k=5), z, 1.0, tokens, 5)
    ids, lps = teacher_of(z, 5, 2)
    loss, out = m.distill(view, ids.to(dev()), lps.to(dev()), out=view)
    rl, rz, e_l, e_z = ref.distill(ref.Distribution(z, 1.0), ids, lps, None, True)
    ref.check("loss", loss, rl, e_l)
    ref.check("dlogits", out, rz, ref.store(BF16, rz, e_z))


def test_no_rows(mxq_lib):
    m = mxq_lib
    say("no rows over a vocabulary")
    z = torch.empty((0, 100), device=dev())
    none = torch.empty((0,), dtype=torch.int32, device=dev())
    lp, ent, stats, ids, lps = m.token_logprobs(z, none, top_k=3)
    assert lp.shape == ent.shape == (0,) and ids.shape == lps.shape == (0, 3)
    assert m.token_logprobs_backward(z, none, stats, ent, lp, ent).shape == (0, 100)
    loss, stats = m.distill_forward(z, ids, lps)
    assert loss.shape == (0,) and m.distill_backward(z, ids, lps, stats).shape == (0, 100)
    loss, dz = m.distill(z, ids, lps)
    assert loss.shape == (0,) and dz.shape == (0, 100)


@pytest.mark.parametrize("rows,vocab", [(2, 131072), (600, 5003)])
def test_repeats_streams_and_graph(mxq_lib, rows, vocab):
    """The same bits again, on another stream, and from each replay of a graph."""
    m = mxq_lib
    z = logits_of((rows, vocab), 1, F32)
    tokens = tokens_of(z, 2).to(dev())
    z = z.to(dev())

    def step(stream=None):
        lp, ent, stats, ids, lps = m.token_logprobs(z, tokens, top_k=16, stream=stream)
        back = m.token_logprobs_backward(z, tokens, stats, ent, lp, ent, stream=stream)
        loss, dz = m.distill(z, ids, lps, out_dtype=BF16, stream=stream)
        loss2, stats2 = m.distill_forward(z, ids, lps, stream=stream)
        return [lp, ent, stats, ids, lps, back, loss, dz, loss2, stats2, m.distill_backward(z, ids, lps, stats2, stream=stream)]
    say("repeats over a vocabulary", (rows, vocab))
    first = [x.clone() for x in step()]
    assert all(torch.equal(a, b) for a, b in zip(first, step()))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = step(side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, other))
    say("graph over a vocabulary", (rows, vocab))
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    for _ in range(3):
        for x in outs:
            x.fill_(3)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(first, outs))
        step()
