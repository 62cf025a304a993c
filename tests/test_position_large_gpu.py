"""The position operators and the clipping past 32-bit offsets: tensors of more
than 2^31 (and 2^32) elements, on sampled rows and on the full sums."""
import pytest
import torch

import _position_ref as R

pytestmark = [pytest.mark.gpu, pytest.mark.slow]

DEV = "cuda:0"


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from transformer_reduce_gb300 import build
    build.build()
    import transformer_reduce_gb300 as L
    L.load()
    torch.cuda.empty_cache()
    yield L
    torch.cuda.empty_cache()


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _need(nbytes):
    free, _ = torch.cuda.mem_get_info(0)
    if free < nbytes:
        pytest.skip(f"needs {nbytes / 1e9:.0f} GB free on the device, {free / 1e9:.0f} GB are")


@pytest.mark.parametrize("Tk", [8192, 8191, 20011])  # whole vectors, odd rows, the looped path
def test_relpos_past_2_pow_31_elements(lib, Tk):
    L = lib
    B, H = 3, 17
    Tq = (1 << 31) // (B * H * Tk) + 60
    _need(40 << 30)
    shape = (B, H, Tq, Tk)
    assert B * H * Tq * Tk > 1 << 31
    dt, nb = torch.bfloat16, 32
    causal = Tq <= Tk
    buckets = L.relpos_buckets(nb, 200, device=DEV)
    table = torch.randn(nb, H, generator=_gen(1), device=DEV).to(dt)
    x = torch.randn(shape, generator=_gen(2), device=DEV, dtype=dt).mul_(3.0)
    mask = torch.zeros(B, Tk, device=DEV, dtype=dt)
    mask[1, Tk - 1000:] = -float("inf")
    y = L.softmax_fw_relpos(x, table, buckets, mask, causal=causal, scale=0.5)
    for b in range(B):
        for h in (0, 7, H - 1):
            want, tol = R.relpos_fw(x[b:b + 1, h:h + 1], table[:, h:h + 1], buckets,
                                    mask[b:b + 1], causal, 0.5)
            R.check(y[b:b + 1, h:h + 1], want, tol, f"fw {b} {h}")
            del want, tol
    dout = x.normal_(generator=_gen(3))
    dx, dtable = L.softmax_bw_relpos(dout, y, buckets, nb, mask, causal=causal, scale=0.5)
    for h in range(H):
        total = torch.zeros(nb, 1, dtype=torch.float64, device=DEV)
        allowed = torch.zeros_like(total)
        for b in range(B):
            (wx, tx), (wt, tt) = R.relpos_bw(dout[b:b + 1, h:h + 1], y[b:b + 1, h:h + 1], buckets,
                                             nb, mask[b:b + 1], causal, 0.5)
            if h in (0, 7, H - 1):
                R.check(dx[b:b + 1, h:h + 1], wx, tx, f"dx {b} {h}")
            total += wt
            allowed += tt
            del wx, tx
        # (each part's bound counts a chain at least as long as its share)
        R.check(dtable[:, h:h + 1], total, B * allowed, f"dtable {h}")


def test_qk_past_2_pow_31_elements(lib):
    L = lib
    T, Hq, Hk, D = 140001, 64, 64, 128
    _need(60 << 30)
    dt = torch.bfloat16
    qkv = torch.randn(T, (Hq + 2 * Hk) * D, generator=_gen(4), device=DEV, dtype=dt)
    assert qkv.numel() > 1 << 31
    q = qkv[:, :Hq * D].view(T, Hq, D)
    k = qkv[:, Hq * D:(Hq + Hk) * D].view(T, Hk, D)
    g = (1 + 0.2 * torch.randn(2, D, generator=_gen(5), device=DEV)).to(dt)
    cos, sin = L.rope_tables(5000, D, device=DEV)
    pos = (torch.arange(T, device=DEV) % 5000).to(torch.int32)
    y, ky, r, kr = L.qk_norm_rope_fw(q, k, g[0], g[1], cos, sin, pos)
    # in place, gradients into a packed buffer, both past 2^31 elements
    dqkv = torch.randn(qkv.shape, generator=_gen(6), device=DEV, dtype=dt)
    dq = dqkv[:, :Hq * D].view(T, Hq, D)
    dk = dqkv[:, Hq * D:(Hq + Hk) * D].view(T, Hk, D)
    rest = dqkv[:, (Hq + Hk) * D:].clone()
    step = 7000
    rows = [slice(0, step), slice(66000, 66000 + step), slice(T - step, T)]
    keep = [(dq[s].clone(), dk[s].clone()) for s in rows]
    sums = [torch.zeros(2, D, dtype=torch.float64, device=DEV) for _ in range(2)]
    for at in range(0, T, step):
        s = slice(at, min(T, at + step))
        for i, (d, x, rs) in enumerate(((dq, q, r), (dk, k, kr))):
            (_, _), (w, t) = R.qk_bw(d[s], x[s], g[i], rs[s], cos, sin, pos[s], False)
            sums[i][0] += w
            sums[i][1] += t
    _, _, dgq, dgk = L.qk_norm_rope_bw(dq, dk, q, k, g[0], g[1], r, kr, cos, sin, pos, dq=dq,
                                       dk=dk)
    for s, (d0, d1) in zip(rows, keep):
        for x, gamma, out, rs, d, dx in ((q, g[0], y, r, d0, dq), (k, g[1], ky, kr, d1, dk)):
            (wy, ty), (wr, tr) = R.qk_fw(x[s], gamma, cos, sin, pos[s], False, 1e-6)
            R.check(out[s], wy, ty, "y")
            R.check(rs[s], wr, tr, "rstd")
            (wx, tx), _ = R.qk_bw(d, x[s], gamma, rs[s], cos, sin, pos[s], False)
            R.check(dx[s], wx, tx, "dx")
    assert torch.equal(dqkv[:, (Hq + Hk) * D:], rest)
    parts = -(-T // step)
    for got, acc in zip((dgq, dgk), sums):
        R.check(got, acc[0], parts * acc[1], "dgamma")


def test_clip_past_2_pow_32_elements(lib):
    L = lib
    n = (1 << 32) + 5
    _need(40 << 30)
    g = [torch.empty(n, device=DEV, dtype=torch.float16).normal_(generator=_gen(7)),
         torch.randn(1001, generator=_gen(8), device=DEV)]
    sq = g[1].double().square().sum()
    step = 1 << 28
    for at in range(0, n, step):
        sq += g[0][at:at + step].double().square().sum()
    ends = [slice(0, 1000), slice((1 << 31) - 500, (1 << 31) + 500), slice(n - 1000, n)]
    keep = [g[0][s].clone() for s in ends]
    _, norm = L.grad_clip(g, 100.0)
    want = float(sq) ** 0.5
    assert abs(float(norm) / want - 1) <= 24 * R.U
    coef = 100.0 / (want + 1e-6)
    for s, k in zip(ends, keep):
        w = k.double() * coef
        R.check(g[0][s], w, w.abs() * (R.half_step(torch.float16) + 30 * R.U) + R.tiny(torch.float16),
                "clipped")
    again = float(L.grad_norm(g))
    assert abs(again / 100.0 - 1) <= 1e-3  # of rounded fp16 values: half a step of 2^-11 each
