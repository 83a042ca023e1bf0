"""Quantization-aware distillation of an output layer, on one GPU.

A teacher's output layer in bf16 hands on its top alternatives for each token;
the student's output layer runs in MXFP4 (all three products), behind a
root-mean-square norm whose weight is trained too:

    teacher   log probabilities of the top alternatives      mxq.token_logprobs
    forward   Y = norm(X), both of its operands              mxq.norm_forward, mxq.quantize
              logits = Y W^T                                  mxq.gemm_abt  (Fprop)
    loss      and the gradient of the logits, one pass        mxq.distill
    backward  dY = dL W, dW = dL^T Y                          mxq.gemm_abt  (Dgrad, Wgrad)
              dX and the norm weight's gradient               mxq.norm_backward

    python examples/distill_head.py [--steps 30]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from fp4_microscaling_quantization_amd import mxq  # noqa: E402

FP4 = dict(grid=mxq.GRID_E2M1, hadamard_n=16)


def product(a, b):
    """A B^T of two FP4 operands, fp32."""
    return mxq.gemm_abt(*a, mxq.FMT_FP4, mxq.GRID_E2M1, *b, mxq.FMT_FP4, mxq.GRID_E2M1)


def operands(t, **kw):
    """A tensor's operands along its rows and along its columns, from one read."""
    q = mxq.quantize(t, row=True, col=True, sign_mask=mxq.rht_sign_mask(3, 16), **FP4, **kw)
    return q["row"], q["col"]


def train(steps=30, tokens=1024, hidden=1024, vocab=8192, top_k=32, temperature=2.0, rate=3.0, seed=1, say=print):
    """The mean loss of each step."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda")
    x = normal(tokens, hidden).bfloat16()
    teacher = (3 * normal(vocab, hidden) / hidden ** 0.5).bfloat16()
    w = teacher.float() + 1.5 * normal(vocab, hidden) / hidden ** 0.5   # the student's, in fp32
    gamma = torch.ones(hidden, device="cuda")
    # tokens of padding at the end count for nothing
    weight = torch.full((tokens,), 1.0 / (tokens - tokens // 16), device="cuda")
    weight[tokens - tokens // 16:] = 0

    y, _, _ = mxq.norm_forward(x, eps=1e-5, kind=mxq.NORM_RMS)
    _, _, _, ids, logprobs = mxq.token_logprobs(y @ teacher.t(), top_k=top_k, temperature=temperature)

    losses = []
    for step in range(steps):
        y, _, rstd = mxq.norm_forward(x, gamma, eps=1e-5, kind=mxq.NORM_RMS)
        y_row, y_col = operands(y)
        w_row, w_col = operands(w.bfloat16())
        logits = product(y_row, w_row)
        loss, dlogits = mxq.distill(logits, ids, logprobs, weight, temperature=temperature, out_dtype=torch.bfloat16)
        d_row, d_col = operands(dlogits, round=mxq.SR, sr_seed=step)
        dy, dw = product(d_row, w_col), product(d_col, y_col)
        _, dgamma, _ = mxq.norm_backward(dy, x, gamma, None, rstd, kind=mxq.NORM_RMS, bias=False, out_dtype=torch.bfloat16)
        w -= rate * dw
        gamma -= 0.001 * rate * dgamma
        losses.append(loss.sum())
    losses = [v.item() for v in losses]
    for step in range(0, steps, max(1, steps // 10)):
        say(f"step {step:3d}  loss {losses[step]:.4f}")
    say(f"last      loss {losses[-1]:.4f}")
    return losses


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--steps", type=int, default=30)
    train(ap.parse_args().steps)
