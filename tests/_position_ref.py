"""64-bit references of the softmax with a relative position bias, the per-head
norm with rotation and the gradient clipping, written from their definitions
in plain torch, with the error bound of each fp32 kernel output beside it.

Bounds.  u = 2^-24 is half a step of fp32 at 1; h = finfo(dtype).eps / 2 half
a step of the storage type.  A sum of fp32 terms along a chain of L additions
is off by at most L u times the sum of their magnitudes; an fp32 product or
sum adds u relative; ex2.approx and rcp.approx at most 4 u; one rounding to
storage h (plus half a subnormal step of fp16, 2^-25, or a flushed fp32
subnormal)."""
import torch

U = 2.0 ** -24


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def tiny(dtype):
    return 2.0 ** -25 if dtype == torch.float16 else 2.0 ** -125


def check(got, want, tol, what):
    """Elementwise |got - want| <= tol; infinities and NaN have to agree."""
    g = got.double()
    want = want.to(g.device)
    assert g.shape == want.shape, f"{what}: shape {tuple(g.shape)} for {tuple(want.shape)}"
    same = (g == want) | (g.isnan() & want.isnan())
    bad = ~(same | ((g - want).abs() <= tol.to(g.device)))
    if bool(bad.any()):
        i = tuple(int(v) for v in bad.nonzero()[0])
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} off, first at {i}: "
                             f"{float(g[i])!r} for {float(want[i])!r}, allowed "
                             f"{float(tol.expand_as(want)[i]):.3g}")


# -- softmax with a relative position bias --------------------------------------
def relpos_pairs(Tq, Tk, buckets, num_buckets, causal, device):
    """(bucket of each pair, or -1 for none; visible by causality) [Tq, Tk]."""
    R = buckets.numel() // 2
    i = torch.arange(Tq, device=device)[:, None] + Tk - Tq
    r = torch.arange(Tk, device=device)[None, :] - i
    ids = buckets.to(device).long()[r.clamp(-R, R) + R]
    ids = torch.where((ids >= 0) & (ids < num_buckets), ids, -1)
    return ids, (r <= 0) if causal else torch.ones_like(r, dtype=torch.bool)


def relpos_visible(shape, mask, seen):
    B, H, Tq, Tk = shape
    vis = seen[None, None].expand(B, 1, Tq, Tk)
    if mask is not None:
        vis = vis & ~torch.isneginf(mask.double())[:, None, None, :]
    return vis.expand(B, H, Tq, Tk)


def relpos_fw(x, table, buckets, mask, causal, scale):
    B, H, Tq, Tk = x.shape
    ids, seen = relpos_pairs(Tq, Tk, buckets, table.shape[0], causal, x.device)
    bias = torch.cat((table.double(), torch.zeros(1, H, dtype=torch.float64, device=x.device)))
    z = x.double() * scale + bias[ids].permute(2, 0, 1)
    if mask is not None:
        z = z + mask.double()[:, None, None, :]
    vis = relpos_visible(x.shape, mask, seen)
    z = torch.where(vis, z, -torch.inf)
    m = z.amax(-1, keepdim=True)
    e = torch.exp(z - torch.where(m.isneginf(), 0.0, m))
    s = e.sum(-1, keepdim=True)
    y = torch.where(s == 0, 0.0, e / s)
    # z carries the rounding of its three terms, z - m and the exponent's
    # argument one each: 5 u max|z|, in the weight and in the sum; the sum's
    # chain has Tk / 32 + 10 terms at most (a warp or more per row)
    big = torch.where(vis, z, 0.0).abs().amax(-1, keepdim=True)
    tol = y * (half_step(x.dtype) + U * (10 * big + Tk / 32 + 24)) + tiny(x.dtype)
    return y, tol


def relpos_bw(dout, y, buckets, num_buckets, mask, causal, scale):
    """((dinp, tol), (dtable, tol))"""
    B, H, Tq, Tk = y.shape
    ids, seen = relpos_pairs(Tq, Tk, buckets, num_buckets, causal, y.device)
    vis = relpos_visible(y.shape, mask, seen)
    yd = torch.where(vis, y.double(), 0.0)
    g = torch.where(vis, dout.double(), 0.0)
    s = (yd * g).sum(-1, keepdim=True)
    dz = yd * (g - s)
    dinp = scale * dz
    s_err = U * (Tk / 32 + 12) * (yd * g).abs().sum(-1, keepdim=True)
    dz_err = yd.abs() * (s_err + 2 * U * (g.abs() + s.abs())) + tiny(torch.float32)
    tol = half_step(y.dtype) * dinp.abs() + scale * 1.01 * dz_err + 2 * U * dinp.abs() + tiny(y.dtype)
    flat = ids.reshape(-1) + 1

    def by_bucket(v):  # [H, Tq, Tk] -> [num_buckets, H]
        out = torch.zeros(num_buckets + 1, H, dtype=torch.float64, device=y.device)
        return out.index_add_(0, flat, v.permute(1, 2, 0).reshape(-1, H))[1:]

    # the longest chain: a group's rows times a lane's clipped keys of a row,
    # its block's groups, the head's blocks, a lane's distances
    W = buckets.numel()
    rows = H * B * Tq
    chain = (rows / 1216 + 1) * (Tk / 32 + 1) + B * Tq / 2 + 2 + W / 32 + 80
    dtable = by_bucket(dz.sum(0))
    dtol = by_bucket(dz_err.sum(0)) + U * chain * by_bucket(dz.abs().sum(0)) + 1e-30
    return (dinp, tol), (dtable, dtol)


# -- per-head norm with rotation -------------------------------------------------
def rotate(x, cos, sin, positions, interleaved, back=False):
    """x [tokens, heads, D] in 64 bits, its first 2 cos.shape[1] features turned."""
    if cos is None:
        return x
    rot = 2 * cos.shape[1]
    bad = (positions < 0) | (positions >= cos.shape[0])
    p = positions.long().clamp(0, cos.shape[0] - 1)
    c, s = (torch.where(bad[:, None], torch.nan, t.double()[p])[:, None, :] for t in (cos, sin))
    s = -s if back else s
    a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if interleaved else \
        (x[..., :rot // 2], x[..., rot // 2:rot])
    ya, yb = a * c - b * s, b * c + a * s
    y = torch.stack((ya, yb), -1).flatten(-2) if interleaved else torch.cat((ya, yb), -1)
    return torch.cat((y, x[..., rot:]), -1)


def _reach(x, cos, positions, interleaved):
    """Bound of a rotated feature: |a| + |b| over its pair, |x| where not rotated."""
    if cos is None:
        return x.abs()
    rot = 2 * cos.shape[1]
    if interleaved:
        t = (x[..., 0:rot:2].abs() + x[..., 1:rot:2].abs()).repeat_interleave(2, -1)
    else:
        t = (x[..., :rot // 2].abs() + x[..., rot // 2:rot].abs()).repeat(1, 1, 2)
    return torch.cat((t, x[..., rot:].abs()), -1)


def qk_fw(x, gamma, cos, sin, positions, interleaved, eps):
    """((y, tol), (rstd, tol)) of one side"""
    D = x.shape[-1]
    xd = x.double()
    rstd = ((xd * xd).sum(-1) / D + eps) ** -0.5
    n = xd * rstd[..., None] * gamma.double()
    y = rotate(n, cos, sin, positions, interleaved)
    k = U * (D / 8 + 24)  # the sum of squares (all positive) and a few roundings
    tol = half_step(x.dtype) * y.abs() + k * _reach(n, cos, positions, interleaved) + tiny(x.dtype)
    return (y, tol), (rstd, k * rstd)


def qk_bw(dout, x, gamma, rstd, cos, sin, positions, interleaved):
    """((dx, tol), (dgamma, tol)) of one side"""
    T, Hn, D = x.shape
    dd = dout.double()
    dn = rotate(dd, cos, sin, positions, interleaved, back=True)
    r = rstd.double()[..., None]
    xh = x.double() * r
    g = dn * gamma.double()
    S = (g * xh).sum(-1, keepdim=True) / D
    dx = r * (g - xh * S)
    far = _reach(dd, cos, positions, interleaved)  # magnitude that dn's rounding goes by
    ga = far * gamma.double().abs()
    mean = (ga * xh.abs()).sum(-1, keepdim=True) / D
    k = U * (D / 8 + 24)
    tol = half_step(x.dtype) * dx.abs() + k * r * (ga + 2 * xh.abs() * mean) + tiny(x.dtype)
    dgamma = (dn * xh).sum((0, 1))
    rows = T * Hn
    chain = rows / 32 + 700  # a lane's rows of a block's run, and at most 609 blocks
    return (dx, tol), (dgamma, U * (chain + 8) * (far * xh.abs()).sum((0, 1)) + 1e-30)


# -- clipping ---------------------------------------------------------------------
def clip(grads, max_norm, eps):
    """((norm, tol), [(out, tol)])"""
    norm = sum((g.double() ** 2).sum() for g in grads) ** 0.5
    k = 24 * U  # 32 terms of a lane pair in FP32 (halved by the root), then FP64, one rounding
    ratio = max_norm / (norm + eps)
    coef = torch.where(ratio >= 1, torch.ones_like(ratio), ratio)
    outs = []
    for g in grads:
        w = g.double() * coef
        outs.append((w, w.abs() * (half_step(g.dtype) + k + 4 * U) + tiny(g.dtype)))
    # (the rounding to fp32 is half a step of 2^-149 where the norm is subnormal)
    return (norm.reshape(1), k * norm.reshape(1) + 2.0 ** -150), outs
