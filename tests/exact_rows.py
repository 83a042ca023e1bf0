"""Rows whose sums are exact in fp32, in whatever order they are added (not a test module).

Over a vocabulary: integer logits from -6 to 0 at the temperature TEMPERATURE, at which exp is a
power of two and of which the kernels' factor log2(e) / T is 1.  Every term of S, and of
sum 2^d d, is a multiple of 2^-6, and the sums stay below 2^18: all partial sums are fp32 numbers.  A
norm's rows hold small integers, none of them 0.  One element that is lost, counted twice or taken
from another row therefore changes the result by more than its bound, at any length here."""
import torch

U = 2.0 ** -24
TEMPERATURE = 1.4426950216293335   # log2(e) as fp32


def spread(rows, cols, seed, device):
    g = torch.Generator(device=device)
    g.manual_seed(seed)
    return lambda low, high: torch.randint(low, high + 1, (rows, cols), generator=g, device=device, dtype=torch.float32)


def logits(rows, vocab, seed, device="cpu"):
    return spread(rows, vocab, seed, device)(-6, 0)


def sums(z):
    """m, S and sum 2^d d of the rows, exact (in 64 bits)."""
    z = z.double()
    m = z.amax(1)
    d = z - m[:, None]
    e = torch.exp2(d)
    return m, e.sum(1), (e * d).sum(1)


def top(z, k):
    """The ids of the k largest, equal ones by index; -1 where there are no more."""
    n = z.shape[1]
    key = (z.long() + 8) * 2 ** 21 + (2 ** 21 - 1 - torch.arange(n, device=z.device))
    ids = 2 ** 21 - 1 - (key.topk(min(k, n), 1).values & (2 ** 21 - 1))
    return torch.nn.functional.pad(ids, (0, k - min(k, n)), value=-1)


def entropy(s, a):
    """log S - sum 2^d d ln 2 / S and its bound from exact sums: the logarithm (6 u), the quotient, ln 2
    and its product, and the difference."""
    log_s, rest = s.log(), a / s * 0.6931471805599453
    return log_s - rest, U * (6 * log_s + 4 * rest.abs() + (log_s - rest))


def gradient(z, ids, s):
    """T (q - 1[v = id]) and its bound: T P, over S, times a power of two; then the difference."""
    m = z.double().amax(1, keepdim=True)
    q = TEMPERATURE * torch.exp2(z.double() - m) / s[:, None]
    hit = torch.arange(z.shape[1], device=z.device) == ids
    dz = torch.where(hit, q - TEMPERATURE, q)
    return dz, U * (4 * q + torch.where(hit, 2 * dz.abs(), 0.0)), hit


def loss(z, ids, s):
    """-T^2 log q at the id, and its bound: the logarithm, log q, T twice."""
    m = z.double().amax(1, keepdim=True)
    gap = (m - z.double().gather(1, ids.long()))[:, 0] / TEMPERATURE
    value = gap + s.log()
    return TEMPERATURE ** 2 * value, TEMPERATURE ** 2 * U * (6 * s.log() + 3 * gap + 4 * value)


def balanced(rows, cols, seed, device="cpu"):
    """Integers from -3 to 3, none of them 0, that add up to 0 in each row of three or more."""
    draw = spread(rows, cols, seed, device)
    half = cols // 2 - cols % 2
    a = draw(1, 3)[:, :half]
    x = torch.cat([a, -a, torch.tensor([1.0, 1.0, -2.0], device=device).expand(rows, 3)[:, :cols - 2 * half]], 1)
    return x.gather(1, draw(0, 1 << 20).argsort(1))
