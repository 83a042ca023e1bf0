"""A training step from a layer's input to clipped gradients, on one GPU.

A linear layer in MXFP4 (all three products) feeds a root-mean-square norm and an output layer in
bf16, whose cross entropy is taken without its logits; all gradients are clipped to a largest norm
together, then stepped along:

    forward   H = X U^T, both operands in MXFP4              mxq.quantize, mxq.gemm_abt  (Fprop)
              Y = norm(H)                                     mxq.norm_forward
              loss = cross entropy of Y W^T                   mxq.linear_ce_forward
    backward  dY, dW                                          mxq.linear_ce_backward
              dH, the norm weight's gradient                  mxq.norm_backward
              dU = dH^T X                                     mxq.quantize, mxq.gemm_abt  (Wgrad)
    clipping  all of dU, dgamma, dW to one norm, in place     mxq.prepare_clip_grad_norm

    python examples/train_head.py [--steps 30]
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


def operand(t, axis, **kw):
    """A tensor's FP4 operand along its rows ("row") or its columns ("col")."""
    q = mxq.quantize(t, row=axis == "row", col=axis == "col", sign_mask=mxq.rht_sign_mask(3, 16), **FP4, **kw)
    return q[axis]


class Model:
    """The parameters, the buffers of their gradients, and the clipping of those."""

    def __init__(self, features=1024, hidden=1024, vocab=8192, max_norm=1.0, seed=1):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        self.u = torch.randn(hidden, features, generator=g, device="cuda") / features ** 0.5
        self.gamma = torch.ones(hidden, device="cuda")
        self.w = torch.randn(vocab, hidden, generator=g, device="cuda") / hidden ** 0.5    # fp32; bf16 in the products
        self.w_used = self.w.bfloat16()
        self.du, self.dgamma, self.dw = torch.empty_like(self.u), torch.empty_like(self.gamma), torch.empty_like(self.w_used)
        self.clip = mxq.prepare_clip_grad_norm([self.du, self.dgamma, self.dw], max_norm, eps=1e-6)

    def gradients(self, x, targets, weight, seed=0):
        """The losses of the rows, and what went into the norm; the gradients are left in their buffers."""
        h = product(operand(x, "row"), operand(self.u.bfloat16(), "row"))
        y, _, rstd = mxq.norm_forward(h, self.gamma, eps=1e-5, kind=mxq.NORM_RMS, out_dtype=torch.bfloat16)
        loss, stats = mxq.linear_ce_forward(y, self.w_used, targets, weight)
        dy, _ = mxq.linear_ce_backward(y, self.w_used, targets, stats, weight, dw=self.dw)
        dh, dgamma, _ = mxq.norm_backward(dy, h, self.gamma, None, rstd, kind=mxq.NORM_RMS, bias=False, out_dtype=torch.bfloat16)
        self.dgamma.copy_(dgamma)
        self.du.copy_(product(operand(dh, "col", round=mxq.SR, sr_seed=seed), operand(x, "col")))
        return loss, h

    def step(self, rate):
        self.u -= rate * self.du
        self.gamma -= rate * self.dgamma
        self.w -= rate * self.dw.float()
        self.w_used.copy_(self.w)


def train(steps=30, tokens=1024, rate=1.0, seed=1, say=print, **sizes):
    """The mean loss of each step."""
    model = Model(seed=seed, **sizes)
    g = torch.Generator(device="cuda")
    g.manual_seed(seed + 1)
    x = torch.randn(tokens, model.u.shape[1], generator=g, device="cuda").bfloat16()
    targets = torch.randint(model.w.shape[0], (tokens,), generator=g, device="cuda", dtype=torch.int32)
    targets[tokens - tokens // 16:] = -1     # padding
    weight = torch.full((tokens,), 1.0 / (tokens - tokens // 16), device="cuda")
    losses, norms = [], []
    for step in range(steps):
        loss, _ = model.gradients(x, targets, weight, seed=step)
        norms.append(model.clip().clone())
        model.step(rate)
        losses.append(loss.sum())
    losses, norms = [v.item() for v in losses], [v.item() for v in norms]
    for step in range(0, steps, max(1, steps // 10)):
        say(f"step {step:3d}  loss {losses[step]:.4f}  gradient norm {norms[step]:.3f}")
    say(f"last      loss {losses[-1]:.4f}")
    return losses


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--steps", type=int, default=30)
    train(ap.parse_args().steps)
