"""64-bit references of the difference of two softmax maps, the norms around a
block and the cross entropy from hidden states, written from their definitions
in plain torch, with the error bound of each output beside it.

Bounds.  u = 2^-24 is half a step of fp32 at 1; h = finfo(dtype).eps / 2 half a
step of the storage type.  A sum of fp32 terms along a chain of L additions is
off by at most L u times the sum of their magnitudes; an fp32 product or sum
adds u relative; ex2.approx and rcp.approx at most 4 u; one rounding to storage
h (plus half a subnormal step).  The tensor cores add exact products of 16-bit
operands into an FP32 accumulator that is cut off, not rounded: at most 2 u of
the sum of magnitudes per step of 16."""
import torch

from _position_ref import U, check, half_step, tiny  # noqa: F401

D64 = torch.float64


def wide(*ts):
    return tuple(None if t is None else t.to(D64) for t in ts)


# -- difference of two softmax maps ----------------------------------------------
def visible(shape, mask, causal, device):
    B, H, Tq, Tk = shape
    vis = torch.ones(B, 1, Tq, Tk, dtype=torch.bool, device=device)
    if causal:
        vis = vis & torch.ones(Tq, Tk, dtype=torch.bool, device=device).tril(Tk - Tq)
    if mask is not None:
        vis = vis & ~torch.isneginf(mask.to(D64))[:, None, None, :]
    return vis.expand(B, H, Tq, Tk)


def one_map(x, mask, causal, scale):
    """(z, -inf at invisible keys; visible; largest z, 0 if there is none; 1 / sum or 0;
    largest |z| of the row)"""
    vis = visible(x.shape, mask, causal, x.device)
    z = x.to(D64) * scale
    if mask is not None:
        z = z + mask.to(D64)[:, None, None, :]
    z = torch.where(vis, z, -torch.inf)
    m = z.amax(-1, keepdim=True)
    m = torch.where(m.isneginf(), 0.0, m)
    s = torch.exp(z - m).sum(-1, keepdim=True)
    inv = torch.where(s == 0, 0.0, 1 / s)
    big = torch.where(vis & z.isfinite(), z, 0.0).abs().amax(-1, keepdim=True)
    return z, vis, m, inv, big


def diff_fw(x1, x2, lam, mask, causal, scale):
    """((y, tol), (stats, tol))"""
    B, H, Tq, Tk = x1.shape
    lam_h = lam.to(D64).expand(H)[None, :, None, None]
    ps, tols, stats, stat_tols = [], [], [], []
    for x in (x1, x2):
        z, vis, m, inv, big = one_map(x, mask, causal, scale)
        p = torch.where(vis, torch.exp(z - m) * inv, 0.0)
        # z: the product, the sum and the exponent's argument (5 u |z|), in the
        # weight and in the sum; the sum's chain has Tk / 32 + 10 terms at most
        k = U * (10 * big + Tk / 32 + 24)
        ps.append(p)
        tols.append(p * k)
        stats += [m, inv]
        # up to |z| = 64 the saved sum also carries the rounding of 64 log2 e
        stat_tols += [4 * U * m.abs(), inv * (k + 100 * U)]
    y = ps[0] - lam_h * ps[1]
    tol = half_step(x1.dtype) * y.abs() + tols[0] + lam_h.abs() * tols[1] + \
        3 * U * (ps[0] + lam_h.abs() * ps[1]) + 2 * tiny(x1.dtype)
    return (y, tol), (torch.cat(stats, -1), torch.cat(stat_tols, -1) + tiny(torch.float32))


def diff_bw(dout, x1, x2, lam, stats, mask, causal, scale):
    """((dx1, tol), (dx2, tol), (dlam, tol)) from given fp32 statistics"""
    B, H, Tq, Tk = x1.shape
    lam_h = lam.to(D64).expand(H)[None, :, None, None]
    out = []
    for a, (x, f) in enumerate(((x1, 1.0), (x2, -lam_h))):
        z, vis, _, _, big = one_map(x, mask, causal, scale)
        m, inv = stats[..., 2 * a:2 * a + 1].to(D64), stats[..., 2 * a + 1:2 * a + 2].to(D64)
        p = torch.where(vis, torch.exp(z - m) * inv, 0.0)
        g = torch.where(vis, dout.to(D64), 0.0)
        D = (p * g).sum(-1, keepdim=True)
        p_err = p * U * (10 * big + 130)
        D_err = (p_err * g.abs()).sum(-1, keepdim=True) + \
            U * (Tk / 32 + 14) * (p * g).abs().sum(-1, keepdim=True)
        dx = scale * f * p * (g - D)
        w = scale * (abs(f) if isinstance(f, float) else f.abs())
        err = w * (p_err * (g.abs() + D.abs()) + p * (D_err + 6 * U * (g.abs() + D.abs())))
        out.append((dx, half_step(x.dtype) * dx.abs() + 1.01 * err + tiny(x.dtype)))
    dlam = -D.sum((0, 2, 3))
    # the fold adds 32 rows in FP32, the rest in FP64
    lam_tol = (D_err + 12 * U * D.abs()).sum((0, 2, 3)) + 2 * U * dlam.abs() + 1e-30
    if lam.numel() == 1:
        dlam, lam_tol = dlam.sum().reshape(1), lam_tol.sum().reshape(1)
    return out[0], out[1], (dlam, lam_tol)


# -- norms around a block ---------------------------------------------------------
def _stats(v, layer, eps):
    mean = v.mean(-1, keepdim=True) if layer else torch.zeros_like(v[:, :1])
    rstd = ((v - mean).square().mean(-1, keepdim=True) + eps) ** -0.5
    return mean, rstd


def block_fw(x, r, g_pre, b_pre, g_post, b_post, gate, a, layer, eps):
    """((h, tol), (y, tol) or None, (stats, tol))"""
    rows, D = x.shape
    dtype = x.dtype
    hs = half_step(dtype)
    x, r, g_pre, b_pre, g_post, b_post, gate = wide(x, r, g_pre, b_pre, g_post, b_post, gate)
    k = U * (D / 8 + 40)  # a row's sums and a few roundings
    one = torch.ones(rows, 1, dtype=D64, device=x.device)
    mean1, rstd1, n, n_err = 0 * one, one, x, torch.zeros_like(x)
    m1_tol = r1_tol = 0 * one
    if g_post is not None:
        mean1, rstd1 = _stats(x, layer, eps)
        hat = (x - mean1) * rstd1
        size = x.abs().mean(-1, keepdim=True)
        m1_tol, r1_tol = k * size, rstd1 * k * (1 + (size * rstd1) * k)
        n = hat * g_post + (b_post if b_post is not None else 0.0)
        n_err = g_post.abs() * k * (hat.abs() + size * rstd1) + 4 * U * n.abs()
        if b_post is not None:
            n_err = n_err + 2 * U * (hat * g_post).abs()
    gr = gate.repeat_interleave(rows // gate.shape[0], 0) if gate is not None else 1.0
    h = a * r + gr * n
    h_err = (gr.abs() if gate is not None else 1.0) * n_err + 4 * U * ((a * r).abs() + (gr * n).abs())
    mean2, rstd2 = 0 * one, one
    m2_tol = r2_tol = 0 * one
    y = None
    if g_pre is not None:
        mean2, rstd2 = _stats(h, layer, eps)
        hat = (h - mean2) * rstd2
        size = h.abs().mean(-1, keepdim=True)
        moved = h_err.mean(-1, keepdim=True)
        m2_tol = k * size + moved
        r2_rel = k * (1 + size * rstd2 * k) + rstd2 * (h_err * hat.abs()).mean(-1, keepdim=True)
        r2_tol = 1.01 * r2_rel * rstd2
        hat_err = rstd2 * (h_err + moved) + hat.abs() * r2_rel + k * (hat.abs() + size * rstd2)
        y = hat * g_pre + (b_pre if b_pre is not None else 0.0)
        tol = hs * y.abs() + 1.01 * g_pre.abs() * hat_err + 6 * U * ((hat * g_pre).abs() + y.abs())
        y = (y, tol + tiny(dtype))
    stats = torch.cat((mean1, rstd1, mean2, rstd2), 1).T
    tol = torch.cat((m1_tol, r1_tol, m2_tol, r2_tol), 1).T + tiny(torch.float32)
    return (h, hs * h.abs() + 1.01 * h_err + tiny(dtype)), y, (stats, tol)


def block_bw(dy, dh, x, h, stats, g_pre, g_post, b_post, gate, a, layer):
    """{name: (value, tol)} of dx, dr and the parameters, from given fp32 statistics"""
    rows, D = x.shape
    dtype = x.dtype
    hs, k = half_step(dtype), U * (D / 8 + 40)
    chain = U * (rows / 300 + 80)  # a worker's rows, the block's workers, the blocks
    dy, dh, x, h, g_pre, g_post, b_post, gate = wide(dy, dh, x, h, g_pre, g_post, b_post, gate)
    mean1, rstd1, mean2, rstd2 = (s.to(D64)[:, None] for s in stats)
    out = {}

    def column(v, err):
        return v.sum(0), err.sum(0) + chain * v.abs().sum(0) + 1e-30

    def back(g, g_err, v, mean, rstd):
        """input gradient of a norm for g = dy * gamma, its error, the hats and theirs"""
        hat = (v - mean) * rstd
        hat_err = 3 * U * (v.abs() + mean.abs()) * rstd
        s2 = (g * hat).mean(-1, keepdim=True)
        s2_err = k * (g * hat).abs().mean(-1, keepdim=True) + \
            (g.abs() * hat_err + g_err * hat.abs()).mean(-1, keepdim=True)
        inner, err = g - hat * s2, g_err + hat.abs() * s2_err + hat_err * s2.abs()
        size = g.abs() + (hat * s2).abs()
        if layer:
            s1 = g.mean(-1, keepdim=True)
            inner = inner - s1
            err = err + k * g.abs().mean(-1, keepdim=True) + g_err.mean(-1, keepdim=True)
            size = size + s1.abs()
        return rstd * inner, rstd * (err + 5 * U * size), hat, hat_err

    up, up_err = (dh, torch.zeros_like(x)) if dh is not None else (torch.zeros_like(x),) * 2
    if g_pre is not None:
        g = dy * g_pre
        b, b_err, hat, hat_err = back(g, U * g.abs(), h, mean2, rstd2)
        up, up_err = up + b, up_err + b_err + 2 * U * (up.abs() + b.abs())
        out["dg_pre"] = column(dy * hat, dy.abs() * hat_err + 2 * U * (dy * hat).abs())
        if layer:
            out["db_pre"] = column(dy, 0 * dy)
    dr = a * up
    out["dr"] = (dr, hs * dr.abs() + 1.01 * abs(a) * up_err + 2 * U * dr.abs() + tiny(dtype))
    gr = gate.repeat_interleave(rows // gate.shape[0], 0) if gate is not None else \
        torch.ones_like(x)
    dn, dn_err = gr * up, gr.abs() * up_err + 2 * U * (gr * up).abs()
    dx, dx_err, n, n_err = dn, dn_err, x, torch.zeros_like(x)
    if g_post is not None:
        dx, dx_err, hat, hat_err = back(dn * g_post, g_post.abs() * dn_err + 2 * U * (dn * g_post).abs(),
                                        x, mean1, rstd1)
        n = hat * g_post + (b_post if b_post is not None else 0.0)
        n_err = g_post.abs() * hat_err + 3 * U * ((hat * g_post).abs() + n.abs())
        out["dg_post"] = column(dn * hat, dn_err * hat.abs() + dn.abs() * hat_err)
        if layer:
            out["db_post"] = column(dn, dn_err)
    if gate is not None:
        G = gate.shape[0]

        def by_gate(v):
            return v.view(G, -1, D).sum(1)

        # gamma_post sum(up xhat) + beta_post sum(up)
        parts = (up * n).abs()
        if b_post is not None:
            parts = (up * hat * g_post).abs() + (up * b_post).abs()
        out["dgate"] = (by_gate(up * n), by_gate(up_err * n.abs() + up.abs() * n_err) +
                        (chain + 4 * U) * by_gate(parts) + 1e-30)
    out["dx"] = (dx, hs * dx.abs() + 1.01 * dx_err + tiny(dtype))
    return out


# -- cross entropy from hidden states ---------------------------------------------
def _steps(n, dtype):
    """Additions into an accumulator of a sum over n: of fp32, six products of planes
    per 256 elements, then FP32 sums of those."""
    if dtype == torch.float32:
        return 2 * 6 * (min(n, 256) / 16 + 1) + n / 256 + 6  # (and the planes left out)
    return 2 * (n / 16 + 1)


def loss_logits(x, w):
    """(z, bound of its error)"""
    z = x.to(D64) @ w.to(D64).T
    return z, U * _steps(x.shape[1], x.dtype) * (x.to(D64).abs() @ w.to(D64).abs().T)


def loss_fw(x, w, target):
    """((loss, tol), (lse, tol))"""
    V = w.shape[0]
    t = target.long()
    dead, bad = t < 0, t >= V
    x = torch.where((dead | bad)[:, None], 0.0, x.to(D64)).to(x.dtype)
    z, z_err = loss_logits(x, w)
    lse = torch.logsumexp(z, -1)
    err = z_err.amax(-1) + U * (60 + V / 4096 + 8 * z.abs().amax(-1)) + 4 * U * lse.abs()
    at = t.clamp(0, V - 1)[:, None]
    loss = lse - z.gather(1, at)[:, 0]
    loss_err = err + z_err.gather(1, at)[:, 0] + 2 * U * (lse.abs() + z.gather(1, at)[:, 0].abs())
    out = []
    for v, e in ((loss, loss_err), (lse, err)):
        v = torch.where(bad, torch.nan, torch.where(dead, 0.0, v))
        out.append((v, e + 1e-30))
    return tuple(out)


def loss_bw(x, w, target, lse, dloss):
    """((dx, tol), (dw, tol))"""
    V, D = w.shape
    N = x.shape[0]
    dtype = x.dtype
    h = half_step(dtype) if dtype != torch.float32 else 2 * U
    t = target.long()
    dead, bad = t < 0, t >= V
    x = torch.where(dead[:, None], 0.0, x.to(D64)).to(dtype)
    z, z_err = loss_logits(x, w)
    l = torch.where(dead, 0.0, lse.to(D64))[:, None]
    up = torch.where(dead, 0.0, dloss.to(D64))[:, None]
    p = torch.exp(z - l)
    hot = torch.zeros_like(z)
    hot[torch.arange(N, device=x.device), t.clamp(0, V - 1)] = 1.0
    hot[dead | bad] = 0.0
    q = up * (p - hot)
    q[bad] = torch.nan
    top = up.abs().amax() if up.numel() else up.sum()
    q_err = up.abs() * p * (1.01 * z_err + U * (6 * l.abs() + 6 * z.abs() + 16)) + \
        up.abs() * 4 * U * (p + hot) + h * q.abs()
    if dtype == torch.float16:  # subnormals of q scaled by 2^14
        q_err = q_err + top * 2.0 ** -38
    out = []
    for val, mag, err, n in ((q @ w.to(D64), q.abs() @ w.to(D64).abs(), q_err @ w.to(D64).abs(), V),
                             (q.T @ x.to(D64), q.T.abs() @ x.to(D64).abs(),
                              q_err.T @ x.to(D64).abs(), N)):
        tol = half_step(dtype) * val.abs() + 1.01 * err + U * (_steps(n, dtype) + 40) * mag + tiny(dtype)
        out.append((val, tol))
    return tuple(out)
