"""The difference of two softmax maps on rows whose largest z lies beyond 64:
z is rounded before the row's largest is taken off, in every kernel, so that no
exponent leaves its range and the backward meets the forward's weights whichever
kernel made the statistics.

Bound, u = 2^-24.  z = fl(scale * x) is formed here as the kernels form it (the
product of two fp32 numbers is exact in 64 bits; the masks are 0 or -inf).  What
is left are the weights w_j = e^(z_j - m): z_j - m, its product with log2 e and
the constant are off by u each relative to the exponent, ex2.approx and
rcp.approx by 4 u each, the sum by the mean of its weights' errors and by one u
per term of its chain, six in an online pass: of Tk / 32 + 10 terms at most.
Beyond z_j - m = -110 a weight is below 2^-149."""
import math

import pytest
import torch

import _decoder_ref as R

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from transformer_reduce_gb300 import build
    build.build()
    import transformer_reduce_gb300 as L
    L.load()
    return L


def _map(x, mask, causal, scale):
    """(p, its relative error) [B,H,Tq,Tk]"""
    vis = R.visible(x.shape, mask, causal, x.device)
    z = (x.double() * torch.tensor(scale, dtype=torch.float32).double().item()).float().double()
    z = torch.where(vis, z, -math.inf)
    m = z.amax(-1, keepdim=True)
    gap = torch.where(vis, m - z, math.inf)
    e = torch.where(vis, torch.exp(-gap), 0.0)
    s = e.sum(-1, keepdim=True)
    p = torch.where(s == 0, 0.0, e / s)
    gap = gap.clamp(max=110.0)
    mean = (p * gap).sum(-1, keepdim=True)
    return p, R.U * (3 * gap + 3 * mean + 6 * (x.shape[-1] / 32) + 70)


def _check(L, x1, x2, mask, causal, scale, seed, outs):
    B, H, Tq, Tk = x1.shape
    dtype = x1.dtype
    h = R.half_step(dtype)
    g_ = torch.Generator(device=DEV).manual_seed(seed)
    lam = torch.rand(H, generator=g_, device=DEV) + 0.2
    dout = torch.randn(x1.shape, generator=g_, device=DEV).to(dtype)
    lam_h = lam.double()[None, :, None, None]
    (p1, r1), (p2, r2) = (_map(x, mask, causal, scale) for x in (x1, x2))
    y = p1 - lam_h * p2
    tol = h * y.abs() + p1 * r1 + lam_h * p2 * r2 + 3 * R.U * (p1 + lam_h * p2) + 2 * R.tiny(dtype)
    got, stats = L.softmax_fw_diff(x1, x2, lam, mask, causal=causal, scale=scale)
    R.check(got, y, tol, "fw")
    assert stats.isfinite().all()
    g = torch.where(R.visible(x1.shape, mask, causal, DEV), dout.double(), 0.0)
    want = []
    for p, r, f in ((p1, r1, 1.0), (p2, r2, -lam_h)):
        D = (p * g).sum(-1, keepdim=True)
        # the weights' errors, the saved inverse among them, and the sum's chain
        D_err = (p * r * g.abs()).sum(-1, keepdim=True) + \
            R.U * (Tk / 32 + 14) * (p * g).abs().sum(-1, keepdim=True)
        dx = scale * f * p * (g - D)
        size = g.abs() + D.abs()
        err = scale * abs(f) * (p * r * size + p * (D_err + 6 * R.U * size))
        want.append((dx, h * dx.abs() + 1.01 * err + R.tiny(dtype)))
    dlam = -D.sum((0, 2, 3))
    lam_tol = (D_err + 12 * R.U * D.abs()).sum((0, 2, 3)) + 2 * R.U * dlam.abs() + 1e-30
    for out in outs:
        d1, d2, dl = L.softmax_bw_diff(dout, x1, x2, lam, stats, mask, causal=causal, scale=scale,
                                       **out)
        R.check(d1, *want[0], "dx1")
        R.check(d2, *want[1], "dx2")
        R.check(dl, dlam, lam_tol, "dlam")


def _off(t, by):
    return torch.empty(t.numel() + 16, dtype=t.dtype, device=DEV)[by:by + t.numel()].view(t.shape)


BASES = [100.0, -3e4, 1e6, 1e8, 3e9, 1e20, -1e30, "lowest"]


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("scale", [0.125, 0.3, 0.7])
@pytest.mark.parametrize("base", BASES)
def test_diff_rows_of_far_scores(lib, dt, scale, base):
    dtype = DT[dt]
    low = torch.finfo(dtype).min
    if base != "lowest" and abs(base) > -low:
        pytest.skip("beyond the type")
    for Tq, Tk in ((9, 64), (9, 77), (1, 40), (3, 300)):
        gen = torch.Generator(device=DEV).manual_seed(Tk)
        shape, x = (2, 2, Tq, Tk), []
        for far in (base, base if base == "lowest" else -base):
            if far == "lowest":  # a row whose every score was hidden by hand
                x.append(torch.full(shape, low, dtype=dtype, device=DEV))
            else:  # neighbours of a few steps of the type, or of a few units
                step = max(1.0, abs(far) * torch.finfo(dtype).eps)
                v = torch.randn(shape, generator=gen, device=DEV) * 2 * step + 1.2 * far / scale
                x.append(v.clamp(min=low, max=-low).to(dtype))
        pad = torch.zeros(2, Tk, dtype=dtype, device=DEV)
        pad[1, Tk // 2:] = -math.inf
        holes = pad.clone()
        holes[0, 3:5] = -math.inf
        for mask in (None, pad, holes):
            for causal in (False, True):
                _check(lib, *x, mask, causal, scale, Tk,
                       ({}, {"dscores1": _off(x[0], 1), "dscores2": _off(x[1], 3)}))


@pytest.mark.parametrize("dt", list(DT))
def test_diff_far_scores_of_very_long_rows(lib, dt):
    """Rows beyond the register kernels."""
    for base in (1e3, 2e4):
        gen = torch.Generator(device=DEV).manual_seed(3)
        x = [(torch.randn((1, 2, 2, 20000), generator=gen, device=DEV) * 3 + s * base).to(DT[dt])
             for s in (1, -1)]
        _check(lib, *x, None, False, 0.7, 5, ({},))
