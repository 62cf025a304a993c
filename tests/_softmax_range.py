"""A 64-bit reference of the softmax with a relative position bias whose bound
stays tight whatever the mask: lowest values, -1e10, +-infinity.

The operator forms z = fl(fl(scale * x + bias) + mask) in fp32.  For inputs on a
coarse grid (``grid``), with a scale that is a power of two, scale * x + bias is
exact in 64 bits, so rounding it once to fp32 and adding the mask in fp32 gives
the operator's own z, and what is left to bound are the weights
w_j = e^(z_j - m), m the row's maximum.

Bound, u = 2^-24.  z_j - m, its product with log2 e and the constant itself are
off by u each, relative to the exponent: 3 u |z_j - m| in w_j; where the product
comes first, m * log2 e is rounded, which multiplies the whole row by one number
and leaves the quotient alone.  ex2.approx and rcp.approx add 4 u each.  The sum
adds its weights' own errors (their mean, weighted) and one u for each term of
its chain, six in an online pass that rescales at every term; the chain has
Tk / 32 + 10 terms at most.  Beyond |z_j - m| = 110 a weight is below 2^-149.
One rounding to storage adds half a step, and half a subnormal step of fp16."""
import torch

from _position_ref import U, half_step, relpos_pairs, relpos_visible, tiny


def grid(t, step=2.0 ** -10):
    """t rounded to multiples of ``step``."""
    return (t / step).round() * step


def scores(x, table, buckets, mask, causal, scale):
    """(z as the operator forms it, in 64 bits and -inf at invisible keys; visible)"""
    B, H, Tq, Tk = x.shape
    ids, seen = relpos_pairs(Tq, Tk, buckets, table.shape[0], causal, x.device)
    assert bool((ids >= 0).all())
    a, b = x.double() * scale, table.double()[ids].permute(2, 0, 1)
    z = a + b
    assert bool(((z - a) == b).all()) and bool(((z - b) == a).all()), "not on the grid"
    z = z.float()
    if mask is not None:
        z = z + mask.float()[:, None, None, :]
    vis = relpos_visible(x.shape, mask, seen)
    return torch.where(vis, z.double(), -torch.inf), vis


def biased_softmax(x, table, buckets, mask, causal, scale):
    """(y, tol)"""
    Tk = x.shape[-1]
    z, _ = scores(x, table, buckets, mask, causal, scale)
    m = z.amax(-1, keepdim=True)
    gap = torch.where(m.isneginf(), torch.inf, m - z)
    e = torch.exp(-gap)
    s = e.sum(-1, keepdim=True)
    y = torch.where(s == 0, 0.0, e / s)
    gap = gap.clamp(max=110.0)
    mean = (y * gap).sum(-1, keepdim=True)
    rel = half_step(x.dtype) + U * (3 * gap + 3 * mean + 6 * (Tk / 32) + 70)
    return y, y * rel + tiny(x.dtype)
