"""The gated product, its gradient and 4-bit weights in 64 bits, and how far a
kernel may be from them."""
import math

import torch

ACTS = ("silu", "gelu", "gelu_tanh")
EPS = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}   # half a step, relative
TINY = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25}  # half the smallest subnormal
GROUP_SHIFT = {32: 5, 64: 6, 128: 7}


def act64(g, kind):
    """Value and slope of an activation, in 64 bits."""
    if kind == "silu":
        p = torch.sigmoid(g)
        d = p * (1 - p)
    elif kind == "gelu":
        p = torch.special.ndtr(g)
        d = torch.exp(-g * g / 2) / math.sqrt(2 * math.pi)
    else:
        v = math.sqrt(2 / math.pi) * (g + 0.044715 * g ** 3)
        p = torch.sigmoid(2 * v)
        d = p * (1 - p) * 2 * math.sqrt(2 / math.pi) * (1 + 3 * 0.044715 * g * g)
    return g * p, p + g * d


def sum_error(mag, k):
    """Bound on a product's fp32 sum of k exact terms whose magnitudes add up to
    mag: at most a step of 2^-23 of it for each 16 terms added together, and for
    the few partial sums of a split."""
    return (k / 16 + 16) * 2.0 ** -23 * mag


def w4_values(q, s, z, group, k):
    """What codes, scales and zero points stand for, in 64 bits."""
    codes = torch.stack((q & 15, q >> 4), -1).reshape(q.shape[0], -1)[:, :k].double()
    of = torch.arange(k, device=q.device) // group
    zero = 8.0 if z is None else z.double()[:, of]
    return (codes - zero) * s.double()[:, of]


def gated_bound(x, w, kind, weight_eps=0.0):
    """h, [g u] in 64 bits and how far the kernel's may be, before rounding; the
    weights may have been rounded by weight_eps, relative."""
    x, w = x.double(), w.double()
    n, k = w.shape[0] // 2, x.shape[1]
    y, mag = x @ w.t(), x.abs() @ w.abs().t()
    err = sum_error(mag, k) + weight_eps * mag
    g, u, eg, eu = y[:, :n], y[:, n:], err[:, :n], err[:, n:]
    a, _ = act64(g, kind)
    # |act'| < 1.13; the activation is computed to 2^-19 of |g| (its exponential's
    # argument, below 88 where the result counts, is rounded to 2^-24 of itself)
    ea = 1.13 * eg + 2.0 ** -19 * g.abs()
    return a * u, y, ea * u.abs() + a.abs() * eu + ea * eu, err


def rounded(bound, ref, dtype):
    """The bound with the result's rounding to dtype added."""
    return bound * (1 + EPS[dtype]) + EPS[dtype] * ref.abs() + TINY[dtype]


def check(out, ref, bound, what=""):
    d = (out.double() - ref).abs()
    bad = ~(d <= bound)
    assert not bad.any(), "%s: %d of %d off, worst %.3g of its bound" % (
        what, int(bad.sum()), bad.numel(), float((d / bound).nan_to_num(math.inf).max()))
