"""The row operators (norm, token log probabilities, distillation) in 64 bits
on the CPU, each with a bound on how far an fp32 computation may be from it
(not a test module).

u = 2^-24 is fp32's rounding.  A sum of n terms, held per thread over at most
n / 64 of them and then joined in a tree, is off by at most depth(n) u times
the sum of the terms' magnitudes.  exp of an argument of magnitude a that was
formed in three roundings is off by (3 a + 4) u of itself.  What is stored in
16 bits may be off by half a step more: finfo.eps / 2 of the value."""
import torch

U = 2.0 ** -24
INF = float("inf")


def depth(n):
    return n / 64 + 32


def store(dtype, value, bound):
    """The bound with the rounding of a value (off by `bound` already) to dtype.
    Below the smallest normal number a step is that of the smallest normal."""
    half = torch.finfo(dtype).eps / 2 if dtype != torch.float32 else 0.0
    return bound + half * (value.abs() + bound) + torch.finfo(torch.float32).tiny


def check(what, got, want, bound):
    got, want, bound = got.detach().double().cpu(), want.double().cpu(), bound.double().cpu()
    assert got.shape == want.shape, (what, got.shape, want.shape)
    same = (got == want) | (got.isnan() & want.isnan())
    off = torch.where(same, 0.0, (got - want).abs())
    bad = ~same & ~(off <= bound)
    assert not bad.any(), (what, int(bad.sum()), bad.nonzero()[:4].tolist(), got[bad][:4].tolist(),
                           want[bad][:4].tolist(), bound.expand_as(got)[bad][:4].tolist())


# ---- norm --------------------------------------------------------------------

def norm(x, gamma, beta, eps, layer):
    """y, mean, rstd and their bounds (y's for fp32 storage)."""
    x = x.double().cpu()
    n = x.shape[1]
    mean = x.mean(1) if layer else torch.zeros(x.shape[0], dtype=torch.float64)
    d_mean = (depth(n) + 2) * U * x.abs().mean(1) if layer else 0 * mean
    c = x - mean[:, None]
    var = (c * c).mean(1)
    rstd = 1 / (var + eps).sqrt()
    # (c + d)^2 is off by 2 |c| d + d^2 in the mean; then the sum, the division, eps, root and reciprocal
    d_c = d_mean[:, None] + U * c.abs()
    d_var = (2 * c.abs() * d_c + d_c * d_c).mean(1) + (depth(n) + 4) * U * var
    d_rstd = rstd * (0.5 * (d_var + U * eps) / (var + eps) + 4 * U)
    # a variance that is off by more than itself: the root's full range
    wide = d_var > 0.5 * (var + eps)
    d_rstd = torch.where(wide, torch.full_like(rstd, INF), d_rstd)
    g = torch.ones(n, dtype=torch.float64) if gamma is None else gamma.double().cpu()
    b = torch.zeros(n, dtype=torch.float64) if beta is None else beta.double().cpu()
    y = c * rstd[:, None] * g + b
    d_y = (d_c * rstd[:, None] + (c.abs() + d_c) * d_rstd[:, None]) * g.abs() + 4 * U * ((y - b).abs() + b.abs())
    return y, mean, rstd, d_y, d_mean, d_rstd


def norm_backward(dy, x, gamma, mean, rstd, layer):
    """dx, dgamma, dbeta and their bounds, from the fp32 mean and rstd."""
    dy, x, rstd = dy.double().cpu(), x.double().cpu(), rstd.double().cpu()[:, None]
    mu = mean.double().cpu()[:, None] if layer else 0.0
    rows, n = x.shape
    g = torch.ones(n, dtype=torch.float64) if gamma is None else gamma.double().cpu()
    h = (x - mu) * rstd                      # off by 2 u of itself
    w = dy * g                               # off by u of itself
    along = (w * h).mean(1, keepdim=True)
    rest = w.mean(1, keepdim=True) if layer else 0.0
    dx = rstd * (w - h * along - rest)
    d_along = (depth(n) + 6) * U * (w * h).abs().mean(1, keepdim=True)
    d_rest = (depth(n) + 3) * U * w.abs().mean(1, keepdim=True) if layer else 0.0
    parts = w.abs() + (h * along).abs() + (abs(rest) if layer else 0.0)
    d_dx = rstd * (h.abs() * d_along + d_rest + 6 * U * parts)
    d_h = 2 * U * h.abs()
    dgamma, dbeta = (dy * h).sum(0), dy.sum(0)
    d_gamma = (dy.abs() * d_h).sum(0) + (depth(rows) + rows / 8 + 2) * U * (dy * h).abs().sum(0)
    d_beta = (depth(rows) + rows / 8 + 2) * U * dy.abs().sum(0)
    return dx, dgamma, dbeta, d_dx, d_gamma, d_beta


# ---- over a vocabulary ---------------------------------------------------------

class Distribution:
    """q = softmax(z / t) of each row; with `stats` from the maximum and sum given."""

    def __init__(self, logits, t, stats=None):
        z = logits.double().cpu()
        self.z, self.t = z, t
        nan = z.isnan().any(1) | (z == INF).any(1)
        self.m = z.nan_to_num(nan=-INF, posinf=INF, neginf=-INF).amax(1) if stats is None else stats[:, 0].double().cpu()
        base = torch.where(self.m == -INF, 0.0, self.m)[:, None]
        self.d = (z - base) / t
        self.e = self.d.exp()
        self.s = self.e.sum(1) if stats is None else stats[:, 1].double().cpu()
        self.s = torch.where(nan, float("nan"), self.s)
        self.none, self.empty = nan, self.s == 0
        n = z.shape[1]
        far = torch.where(self.e > 0, self.d.abs(), 0.0)
        weigh = (self.e * far).sum(1) / self.s.clamp(min=1e-300)
        self.far = far
        self.d_s = U * (3 * weigh + 4 + depth(n)) if stats is None else 0 * weigh     # of itself
        self.log_s = self.s.log()
        self.logq = torch.where(self.empty[:, None], -INF, self.d - self.log_s[:, None])
        self.logq[self.none] = float("nan")
        # the difference, the division, the logarithm (2 u of itself) and the last difference
        self.d_logq = (3 * U * far + (self.d_s + 3 * U * self.log_s.abs())[:, None] + U * self.logq.abs())
        self.d_logq = torch.where(self.d_logq.isfinite(), self.d_logq, 0.0)
        self.q = torch.where(self.empty[:, None], 0.0, self.logq.exp())
        # exp, the reciprocal and product; an exp below the smallest normal number may be 0
        self.d_q = self.q * (U * (3 * far + 8) + self.d_s[:, None]) + torch.finfo(torch.float32).tiny
        self.entropy = torch.where(self.empty, 0.0, -torch.where(self.q > 0, self.q * self.logq, 0.0 * self.q).sum(1))
        self.entropy[self.none] = float("nan")
        mean_d = weigh
        err_a = U * ((self.e * far * (3 * far + 6)).sum(1) / self.s.clamp(min=1e-300) + (depth(n) + 2) * mean_d)
        self.d_entropy = self.d_s * (1 + mean_d) + 3 * U * self.log_s.abs() + err_a + 2 * U * self.entropy.abs()

    def top(self, k):
        """ids (-1: none left) of the k largest logits, equal ones by index."""
        rows, n = self.z.shape
        z = torch.where(self.z.isnan(), 0.0, self.z)
        values, order = z.sort(dim=1, descending=True, stable=True)
        ids = torch.full((rows, k), -1, dtype=torch.int64)
        ids[:, :min(k, n)] = order.masked_fill(values == -INF, -1)[:, :k]
        ids[self.none] = -1
        return ids

    def pick(self, a, ids, absent):
        return torch.where(ids < 0, absent, a.gather(1, ids.clamp(min=0)))


def distill(dist, ids, lps, weight, renormalize):
    """loss, dlogits and their bounds."""
    ids, lps, t = ids.long().cpu(), lps.double().cpu(), dist.t
    rows, n = dist.z.shape
    w = torch.ones(rows, dtype=torch.float64) if weight is None else weight.double().cpu()
    lp = torch.where(ids < 0, -INF, lps)
    spread = torch.zeros(rows, 1, dtype=torch.float64)
    if renormalize:
        m = lp.amax(1, keepdim=True)
        some = m > -INF
        total = (lp - m).exp().sum(1, keepdim=True)
        spread = torch.where(some, total.log().abs(), 0.0)
        lp = torch.where(some, lp - m - total.log(), lp)
        # the difference to the maximum, then exp, a sum of 64, its logarithm
        d_lp = U * (3 * torch.where(lp > -INF, (lp.abs() + spread), 0.0) + 12 + 4 * spread)
    else:
        d_lp = torch.zeros_like(lp)
    p = lp.exp()
    d_p = p * (d_lp + U * (torch.where(p > 0, lp.abs(), 0.0) + 4))
    bad = (ids >= n).any(1)
    zero = (w == 0) | (~bad & (p == 0).all(1))
    safe = torch.where(ids >= n, -1, ids)
    logq = dist.pick(dist.logq, safe, 0.0)
    d_logq = dist.pick(dist.d_logq, safe, 0.0)
    terms = torch.where(p != 0, p * (lp - logq), 0.0)
    d_terms = torch.where(p != 0, p * (d_lp + d_logq) + d_p * (lp - logq).abs() + 3 * U * terms.abs(), 0.0)
    loss = w * t * t * terms.sum(1)
    d_loss = (w * t * t).abs() * (d_terms.sum(1) + 8 * U * terms.abs().sum(1)) + 4 * U * loss.abs()
    big = p.sum(1, keepdim=True)
    d_big = d_p.sum(1, keepdim=True) + 8 * U * big
    dense = torch.zeros(rows, n, dtype=torch.float64).scatter_add_(1, safe.clamp(min=0), torch.where(safe < 0, 0.0, p))
    d_dense = torch.zeros(rows, n, dtype=torch.float64).scatter_add_(1, safe.clamp(min=0), torch.where(safe < 0, 0.0, d_p))
    wt = (w * t)[:, None]
    dz = wt * (big * dist.q - dense)
    d_dz = wt.abs() * (big * dist.d_q + dist.q * d_big + d_dense + 6 * U * (big * dist.q) + 70 * U * dense) + 2 * U * dz.abs()
    loss, dz = torch.where(bad, float("nan"), loss), torch.where(bad[:, None], float("nan"), dz)
    loss, dz = torch.where(zero, 0.0, loss), torch.where(zero[:, None], 0.0, dz)
    return loss, dz, d_loss, d_dz


def logprobs_backward(dist, tokens, entropy, gl, gh):
    """dlogits and its bound."""
    tokens, gl, gh, h = tokens.long().cpu(), gl.double().cpu(), gh.double().cpu(), entropy.double().cpu()
    n = dist.z.shape[1]
    gl = torch.where(tokens < 0, 0.0, torch.where(tokens >= n, float("nan"), gl))[:, None]
    gh = gh[:, None]
    lq = torch.where(dist.q == 0, 0.0, dist.logq + h[:, None])
    hit = torch.arange(n) == tokens[:, None]
    one = torch.where(hit, gl, 0.0)
    dz = (one - dist.q * (gl + gh * lq)) / dist.t
    parts = (one.abs() + dist.q * (gl.abs() + (gh * lq).abs())) / dist.t
    d_lq = dist.d_logq + U * (dist.far + h.abs()[:, None] + 4 * lq.abs())
    d_dz = (dist.d_q * (gl.abs() + (gh * lq).abs()) + dist.q * gh.abs() * d_lq) / dist.t + 6 * U * parts
    return dz, d_dz
