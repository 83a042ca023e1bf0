"""Cross entropy of an output layer in 64 bits, with bounds on how far the
library's computation may be from it (not a test module).

u = 2^-24 is fp32's rounding, h = 2^-8 is half a bf16 step.

A logit is a sum of `hidden` exact products of bf16 values in fp32, 32 of them
an instruction: at most hidden / 8 roundings, each of at most 2 u of the sum of
the products' magnitudes (`reach`).  exp of an argument of magnitude a that was
formed in three roundings is off by (3 a + 4) u of itself, and by the logits'
own error over the temperature.

dz is rounded to bf16 before the second products.  Its roundings are as good as
independent, each uniform within half a step, so a sum of n terms t_i is off by
h / sqrt(3) sqrt(sum t_i^2) in the root mean square: 4 h sqrt(sum t_i^2) is
seven of those deviations, and no less than the worst case, h sum |t_i|, where
there are up to 16 terms.  Everything else (dz's own error, fp32 sums) is in
the bound as the worst case, and the store rounds once more."""
import torch

import row_refs as ref

U, H = 2.0 ** -24, 2.0 ** -8


class HeadLoss:
    """loss, stats, dx, dw of the rows x [rows, hidden] under w [vocab, hidden], on the CPU; the gradients
    from `stats` where they are given."""

    def __init__(self, x, w, targets, weight=None, t=1.0, stats=None):
        x, w = x.double().cpu(), w.double().cpu()
        targets = targets.long().cpu()
        rows, hidden = x.shape
        vocab = w.shape[0]
        weight = torch.ones(rows, dtype=torch.float64) if weight is None else weight.double().cpu()
        self.counts = (targets >= 0) & ~(weight == 0)
        k = self.counts.nonzero()[:, 0]
        x1, t1, w1 = x[k], targets[k], weight[k, None]
        foreign = t1 >= vocab
        z = x1 @ w.t()
        d_z = hidden / 8 * 2 * U * (x1.abs() @ w.abs().t())
        self.z = z
        m = z.amax(1, keepdim=True)
        base = torch.where(m == -ref.INF, 0.0, m)
        a = (z - base) / t
        e = a.exp()
        s = e.sum(1, keepdim=True)
        # both ends of a difference are off, and the maximum itself is within the rows' error
        d_a = (d_z + d_z.amax(1, keepdim=True)) / t
        d_e = e * ((3 * a.abs().nan_to_num(posinf=0.0) + 4) * U + d_a)
        d_s = d_e.sum(1, keepdim=True) + (vocab / 64 + 64) * U * s
        logq = a - s.log()
        d_logq = d_a + d_s / s + 4 * U * (a.abs() + s.log().abs() + 1)
        at = t1.clamp(max=vocab - 1)[:, None]
        pick, d_pick = logq.gather(1, at)[:, 0], d_logq.gather(1, at)[:, 0]
        self.loss, self.d_loss = torch.zeros(rows, dtype=torch.float64), torch.zeros(rows, dtype=torch.float64)
        self.loss[k] = torch.where(foreign, float("nan"), -w1[:, 0] * pick)
        self.d_loss[k] = w1[:, 0].abs() * (d_pick + 2 * U * pick.abs())
        self.m, self.d_m = torch.zeros(rows, dtype=torch.float64), torch.zeros(rows, dtype=torch.float64)
        self.s, self.d_s = torch.ones(rows, dtype=torch.float64), torch.zeros(rows, dtype=torch.float64)
        self.m[k], self.d_m[k] = m[:, 0], d_z.amax(1)
        self.s[k], self.d_s[k] = s[:, 0], d_s[:, 0]
        if stats is not None:
            given = stats.double().cpu()[k]
            a, s = (z - given[:, :1]) / t, given[:, 1:]
            e, d_a, d_s = a.exp(), d_z / t, 0 * s
        q = e / s
        one = torch.zeros_like(q).scatter_(1, at, 1.0)
        dz = w1 / t * (q - one)
        dz[foreign] = float("nan")
        d_q = q * ((3 * a.abs().nan_to_num(posinf=0.0) + 8) * U + d_a + d_s / s)
        d_dz = w1.abs() / t * (d_q + 4 * U * (q + one))
        self.dx = torch.zeros(rows, hidden, dtype=torch.float64)
        self.d_dx = torch.zeros_like(self.dx)
        self.dx[k] = dz @ w
        self.d_dx[k] = self._bound(dz, d_dz, w, self.dx[k])
        self.dw = dz.t() @ x1
        self.d_dw = self._bound(dz.t(), d_dz.t(), x1, self.dw)

    @staticmethod
    def _bound(dz, d_dz, other, value):
        n = dz.shape[1]
        # subnormal bf16 values have no smaller step than 2^-133
        rounding = 4 * H * ((dz * dz) @ (other * other)).sqrt() + 2.0 ** -133 * other.abs().sum(0)
        rest = (d_dz * (1 + H)) @ other.abs() + (n / 8 + 32) * 2 * U * (dz.abs() @ other.abs())
        return ref.store(torch.bfloat16, value, rounding + rest)

    def check_forward(self, what, loss, stats):
        ref.check((what, "loss"), loss, self.loss, self.d_loss)
        ref.check((what, "max"), stats[:, 0], self.m, self.d_m)
        ref.check((what, "sum"), stats[:, 1], self.s, self.d_s)

    def check_backward(self, what, dx, dw):
        if dx is not None:
            ref.check((what, "dx"), dx, self.dx, self.d_dx)
        if dw is not None:
            ref.check((what, "dw"), dw, self.dw, self.d_dw)

    def stats(self):
        """The stats in fp32, as the backward pass takes them."""
        return torch.stack([self.m, self.s], 1).float()
