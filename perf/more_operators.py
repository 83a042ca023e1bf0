"""The loss of an output layer without its logits, and the clipping of all gradients: cases to time and to compare.

Two operators that close a training step around the quantized products:

- softmax cross entropy from the hidden states and the output layer's weight, over a large
  vocabulary, without the logits ever being kept: the loss of each token forward, and the
  gradients of the hidden states and of the weight backward;
- the global norm of a list of gradients, and the gradients scaled down to a largest norm.

`run` computes them in plain torch operations, or, where `own` is true, through the library.
"""
import torch

own = False

EPS = 1e-6
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "bf16": 2}


def listed():
    return [
        # the loss of one token after a prompt: latency, and a weight of 64 MB to read
        dict(name="head loss: one token", op="ce", rows=1, hidden=1024, vocab=32000, ignored=0.0, temperature=1.0),
        # scoring a few continuations with a large vocabulary: one read of the weight
        dict(name="head loss: a few tokens", op="ce", rows=24, hidden=4096, vocab=128256, ignored=0.0, temperature=1.0),
        # evaluation of a text in windows of odd length, with a vocabulary that is no multiple of anything
        dict(name="head loss: odd", op="ce", rows=1501, hidden=1600, vocab=50257, ignored=0.0, temperature=1.0),
        # a training step of 8192 tokens, a tenth of them padding
        dict(name="head loss: step", op="ce", rows=8192, hidden=4096, vocab=128256, ignored=0.1, temperature=1.0),
        # the backward pass of a few tokens: the weight and its gradient are all there is to move
        dict(name="head loss backward: a few tokens", op="ce_bwd", rows=16, hidden=4096, vocab=32003, ignored=0.0, temperature=1.0),
        # a micro-batch with an odd vocabulary, at a temperature
        dict(name="head loss backward: odd", op="ce_bwd", rows=1501, hidden=1600, vocab=50257, ignored=0.1, temperature=0.7),
        # fine-tuning on answers: more than half of the tokens are prompt and do not count
        dict(name="head loss backward: answers", op="ce_bwd", rows=4096, hidden=4096, vocab=32000, ignored=0.6, temperature=1.0),
        # the backward pass of the training step
        dict(name="head loss backward: step", op="ce_bwd", rows=8192, hidden=4096, vocab=128256, ignored=0.1, temperature=1.0),
        # the norm of one small layer's gradients, for a log: latency
        dict(name="gradient norm: small layer", op="norm", layers=1, hidden=512, inner=1024, vocab=0, g="f32"),
        # a shard of a large model's gradients in bf16, whose squares are summed over the ranks next
        dict(name="gradient norm: shard", op="norm", layers=4, hidden=4096, inner=14336, vocab=32000, g="bf16"),
        # some hundred tensors of odd sizes, adapters and norms among them, clipped into fp32
        dict(name="clipping: odd tensors", op="clip", count=700, largest=200003, g="bf16", out="f32", over=True),
        # the fp32 gradients of layers and output layer, clipped into the bf16 that the optimizer reads
        dict(name="clipping: layers and head", op="clip", layers=4, hidden=4096, inner=14336, vocab=128256, g="f32", out="bf16", over=True),
    ]


def _size(rng, low, high, step=1):
    """A size in low..high, spread over its logarithm, a multiple of `step`."""
    n = int(round(low * (high / low) ** rng.random()))
    return min(high, max(low, n // step * step))


def draw(rng):
    op = rng.choice(("ce", "ce_bwd", "ce", "ce_bwd", "norm", "clip"))
    if op in ("ce", "ce_bwd"):
        hidden = _size(rng, 64, 8192, rng.choice((32, 64, 256)))
        vocab = _size(rng, 500, min(160000, 2 ** 29 // hidden), rng.choice((1, 1, 128)))
        rows = _size(rng, 1, max(1, min(8192, 2 ** 41 // (hidden * vocab))))
        return dict(op=op, rows=rows, hidden=hidden, vocab=vocab, ignored=rng.choice((0.0, 0.1, rng.random())), temperature=rng.choice((1.0, 1.0, 0.7, 2.0)))
    case = dict(op=op, g=rng.choice(("f32", "bf16")))
    if rng.random() < 0.5:
        case.update(layers=rng.randint(1, 4), hidden=_size(rng, 64, 4096, 8), inner=_size(rng, 128, 14336, 8), vocab=rng.choice((0, _size(rng, 500, 128256))))
    else:
        case.update(count=_size(rng, 1, 1500), largest=_size(rng, 16, 1000000))
    if op == "clip":
        case["out"], case["over"] = rng.choice(("f32", "bf16")), rng.random() < 0.75
    return case


# ---- inputs ----------------------------------------------------------------------------------

def _used(case):
    """The rows that count."""
    return case["rows"] - int(case["rows"] * case["ignored"])


def _shapes(case):
    """The shapes of the gradients: layers of attention and a gated block with their norms, and an
    output layer; or `count` vectors of lengths up to `largest`, spread over their logarithm."""
    if "layers" in case:
        h, f, kv = case["hidden"], case["inner"], max(1, case["hidden"] // 4)
        layer = [(h, h), (kv, h), (kv, h), (h, h), (f, h), (f, h), (h, f), (h,), (h,)]
        return layer * case["layers"] + ([(case["vocab"], h)] if case["vocab"] else []) + [(h,)]
    return [(int(case["largest"] ** ((i * 0.6180339887) % 1)),) for i in range(1, case["count"] + 1)]


def _count(shape):
    return shape[0] * (shape[1] if len(shape) > 1 else 1)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda")

    if case["op"] in ("norm", "clip"):
        shapes = _shapes(case)
        # gradients whose size differs from tensor to tensor; together they have the norm `want`
        size = torch.rand(len(shapes), generator=g, device="cuda") + 0.1
        total = torch.stack([size[i] ** 2 * _count(s) for i, s in enumerate(shapes)]).sum().sqrt()
        want = 2.7 if case.get("over", True) else 0.4
        grads = [(normal(*s) * (size[i] * want / total)).to(DT[case["g"]]) for i, s in enumerate(shapes)]
        state = dict(case=case, grads=grads)
        if case["op"] == "clip":
            # the optimizer's one buffer, with a view for each gradient
            state["max_norm"] = 1.0
            state["flat"] = torch.empty(sum(t.numel() for t in grads), dtype=DT[case["out"]], device="cuda")
            state["out"] = [v.view(t.shape) for v, t in zip(state["flat"].split([t.numel() for t in grads]), grads)]
        if own:
            from fp4_microscaling_quantization_amd import mxq
            # the buffers of a training run stay where they are, so the list of them is made once
            state["call"] = (mxq.prepare_grad_norm(grads) if case["op"] == "norm" else
                             mxq.prepare_clip_grad_norm(grads, state["max_norm"], eps=EPS, out=state["out"]))
        return state
    rows, hidden, vocab = case["rows"], case["hidden"], case["vocab"]
    w = (normal(vocab, hidden) * (2.5 / hidden ** 0.5)).to(torch.bfloat16)
    targets = torch.randint(vocab, (rows,), generator=g, device="cuda", dtype=torch.int32)
    # hidden states that lean towards their target, as a trained model's do: losses of about 3 with all
    # vocabularies, from well under 1 to over 10
    lean = 1 + 0.4 * normal(rows, 1)
    x = (normal(rows, hidden) + lean * w[targets.long()].float()).to(torch.bfloat16)
    weight = torch.full((rows,), 1.0 / _used(case), device="cuda")
    # tokens that do not count lie in stretches: prompts and padding
    start = torch.randint(rows, (1,), generator=g, device="cuda")
    place = (torch.arange(rows, device="cuda") - start) % rows
    targets = torch.where(place < rows - _used(case), -100, targets).to(torch.int32)
    s = dict(case=case, x=x, w=w, targets=targets, weight=weight)
    if case["op"] == "ce_bwd":
        t = case["temperature"]
        stats = []
        for part in x.split(1024):
            z = part.float() @ w.float().t()
            top = z.amax(1, keepdim=True)
            stats.append(torch.cat([top, ((z - top) / t).exp().sum(1, keepdim=True)], 1))
        s["stats"] = torch.cat(stats)
    return s


# ---- one pass --------------------------------------------------------------------------------

def run(state):
    return (_run_own if own else _run_plain)(state)


def _run_own(s):
    from fp4_microscaling_quantization_amd import mxq
    c = s["case"]
    if c["op"] == "norm":
        return s["call"]()
    if c["op"] == "clip":
        return s["call"](), s["flat"]
    if c["op"] == "ce":
        return mxq.linear_ce_forward(s["x"], s["w"], s["targets"], s["weight"], temperature=c["temperature"])
    return mxq.linear_ce_backward(s["x"], s["w"], s["targets"], s["stats"], s["weight"], temperature=c["temperature"])


def _run_plain(s):
    c = s["case"]
    if c["op"] in ("norm", "clip"):
        squares = [t.double().square().sum() for t in s["grads"]]
        total = torch.stack(squares).sum()
        norm = total.sqrt().float()
        if c["op"] == "norm":
            return norm, total
        scale = (s["max_norm"] / (norm + EPS)).clamp(max=1.0)
        for t, out in zip(s["grads"], s["out"]):
            out.copy_(t.float() * scale)
        return norm, s["flat"]
    t = c["temperature"]
    x, w = s["x"].float(), s["w"].float()
    counts = s["targets"] >= 0
    at = s["targets"].clamp(min=0).long()[:, None]
    z = x @ w.t()
    if c["op"] == "ce":
        top = z.amax(1, keepdim=True)
        total = ((z - top) / t).exp().sum(1, keepdim=True)
        loss = total.log() - (z.gather(1, at) - top) / t
        loss = torch.where(counts, s["weight"] * loss[:, 0], 0.0)
        # what does not count has the maximum 0 and the sum 1
        return loss, torch.where(counts[:, None], torch.cat([top, total], 1), torch.tensor([0.0, 1.0], device=x.device))
    d = ((z - s["stats"][:, :1]) / t).exp() / s["stats"][:, 1:]
    d.scatter_add_(1, at, torch.full_like(at, -1, dtype=torch.float32))
    d *= torch.where(counts, s["weight"] / t, 0.0)[:, None]
    return (d @ w).to(torch.bfloat16), (d.t() @ x).to(torch.bfloat16)


# ---- the bytes and operations that a pass cannot do without ----------------------------------

def work(case):
    if case["op"] in ("norm", "clip"):
        n = sum(_count(s) for s in _shapes(case))
        return {"bytes": n * (SIZE[case["g"]] + SIZE.get(case.get("out"), 0)), "flops": n * (3 if case["op"] == "clip" else 2)}
    rows, hidden, vocab, used = case["rows"], case["hidden"], case["vocab"], _used(case)
    product = 2 * used * hidden * vocab
    if case["op"] == "ce":
        return {"bytes": 2 * hidden * (vocab + used) + rows * 20, "flops": product + 4 * used * vocab}
    # the logits again, then both gradients; all rows of dx are written
    return {"bytes": 2 * hidden * (2 * vocab + used + rows) + rows * 16, "flops": 3 * product + 6 * used * vocab}


# ---- the definitions, in 64 bits -------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] in ("norm", "clip"):
        norms = torch.stack([torch.linalg.vector_norm(t.double()) for t in s["grads"]])
        norm = torch.linalg.vector_norm(norms)
        if case["op"] == "norm":
            return norm, norm * norm
        scale = min(1.0, s["max_norm"] / (norm.item() + EPS))
        return norm, torch.cat([t.double().flatten() * scale for t in s["grads"]])
    # the tokens that count, some at a time: log q by logsumexp, gradients from the one-hot target
    rows, t = case["rows"], case["temperature"]
    w = s["w"].double()
    keep = (s["targets"] >= 0).nonzero()[:, 0]
    loss = torch.zeros(rows, dtype=torch.float64, device="cuda")
    stats = torch.zeros(rows, 2, dtype=torch.float64, device="cuda")
    stats[:, 1] = 1
    dx = torch.zeros(rows, case["hidden"], dtype=torch.float64, device="cuda")
    dw = torch.zeros_like(w)
    for part in keep.split(max(1, 2 ** 28 // case["vocab"])):
        x, target, weight = s["x"][part].double(), s["targets"][part].long(), s["weight"][part].double()
        y = torch.mm(x, w.t()).div_(t)
        if case["op"] == "ce":
            norm = torch.logsumexp(y, 1)
            loss[part] = weight * (norm - torch.einsum("rh,rh->r", x, w[target]) / t)
            top = y.amax(1)
            stats[part] = torch.stack([top * t, (norm - top).exp()], 1)
        else:
            given = s["stats"][part].double()
            y = y.sub_((given[:, 0] / t + given[:, 1].log())[:, None]).exp_()
            y[torch.arange(len(part), device="cuda"), target] -= 1
            y = y.mul_((weight / t)[:, None])
            dx[part] = torch.mm(y, w)
            dw.addmm_(y.t(), x)
    return (loss, stats) if case["op"] == "ce" else (dx, dw)
