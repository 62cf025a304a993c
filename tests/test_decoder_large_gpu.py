"""The difference of two softmax maps, the norms around a block and the cross
entropy from hidden states past 32-bit offsets, on sampled rows against their
64-bit references."""
import pytest
import torch

import _decoder_ref as R

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


def _need(nbytes):
    free, _ = torch.cuda.mem_get_info(0)
    if free < nbytes:
        pytest.skip(f"needs {nbytes / 1e9:.0f} GB free on the device, {free / 1e9:.0f} GB are")


def _fill(t, seed, std=1.0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    for part in t.view(-1).split(1 << 28):
        part.copy_(torch.randn(part.shape, generator=g, device=DEV) * std)
    return t


def test_diff_past_2_pow_31_elements(lib):
    """Two maps in one tensor of 4.3e9 elements."""
    L = lib
    B, H, T = 2, 4, 16384
    _need(60 << 30)
    s = _fill(torch.empty(B, 2 * H, T, T, dtype=torch.bfloat16, device=DEV), 1, 2.0)
    lam = torch.linspace(0.2, 0.8, H, device=DEV)
    y, st = L.softmax_fw_diff(s[:, :H], s[:, H:], lam)
    picks = [(0, 0, 0), (1, 0, 5), (1, H - 1, T - 1), (0, H - 1, 7777)]
    dout = _fill(torch.empty_like(y), 2)
    d1, d2, _ = L.softmax_bw_diff(dout, s[:, :H], s[:, H:], lam, st)
    for b, h, i in picks:
        rows = [t[b:b + 1, h:h + 1, i:i + 1].contiguous()
                for t in (s[:, :H], s[:, H:], y, st, dout, d1, d2)]
        (want, tol), (sw, stol) = R.diff_fw(rows[0], rows[1], lam[h:h + 1], None, False, 1.0)
        R.check(rows[2], want, tol, f"fw {b, h, i}")
        R.check(rows[3], sw, stol, f"stats {b, h, i}")
        a, c, _ = R.diff_bw(rows[4], rows[0], rows[1], lam[h:h + 1], rows[3], None, False, 1.0)
        R.check(rows[5], *a, f"dx1 {b, h, i}")
        R.check(rows[6], *c, f"dx2 {b, h, i}")


def test_block_past_2_pow_31_elements(lib):
    L = lib
    rows, D = 540000, 4096
    _need(60 << 30)
    x = _fill(torch.empty(rows, D, dtype=torch.bfloat16, device=DEV), 1)
    r = _fill(torch.empty_like(x), 2)
    g = torch.full((D,), 1.25, dtype=torch.bfloat16, device=DEV)
    h, y, st = L.block_norm_fw(x, r, g, gamma_post=g)
    dx, dr, dg, _, _, _, _ = L.block_norm_bw(y, r, x, h, st, g, g)
    for i in (0, 262143, 262144, 524289, rows - 1):
        sl = slice(i, i + 1)
        fw = R.block_fw(x[sl], r[sl], g, None, g, None, None, 1.0, False, 1e-6)
        R.check(h[sl], *fw[0], f"h {i}")
        R.check(y[sl], *fw[1], f"y {i}")
        bw = R.block_bw(y[sl], r[sl], x[sl], h[sl], st[:, sl].contiguous(), g, g, None, None, 1.0,
                        False)
        R.check(dx[sl], *bw["dx"], f"dx {i}")
        R.check(dr[sl], *bw["dr"], f"dr {i}")
    want = sum((y[p].double()[:, :64] * (h[p].double()[:, :64] * st[3, p].double()[:, None])).sum(0)
               for p in torch.arange(rows, device=DEV).split(60000))
    # 445 rows of a worker, 8 workers, 304 blocks, of products of a few in magnitude
    mag = sum((y[p].double()[:, :64] * (h[p].double()[:, :64] * st[3, p].double()[:, None])).abs().sum(0)
              for p in torch.arange(rows, device=DEV).split(60000))
    R.check(dg[:64], want, R.U * (rows / 300 + 90) * mag, "dgamma")


def test_linear_ce_past_2_pow_31_elements(lib):
    """A vocabulary matrix of 2.2e9 elements, and gradients written beyond them."""
    L = lib
    rows, D, V = 5, 1024, 2150003
    _need(60 << 30)
    w = _fill(torch.empty(V, D, dtype=torch.bfloat16, device=DEV), 1, 0.05)
    x = _fill(torch.empty(rows, D, dtype=torch.bfloat16, device=DEV), 2)
    t = torch.tensor([0, V - 1, -1, 2097152, 2097151], dtype=torch.int32, device=DEV)
    loss, lse = L.linear_cross_entropy_fw(x, w, t)
    z = torch.cat([x.double() @ p.double().T for p in w.split(100000)], 1)
    want = torch.logsumexp(z, -1)
    live = t >= 0
    # 64 steps of 16 of an accumulator, values up to sum |x w| of about 40
    assert (lse[live].double() - want[live]).abs().max() < 2 * R.U * 70 * 50 + R.U * 700
    hit = z[torch.arange(rows), t.clamp(min=0).long()]
    assert (loss[live].double() - (want - hit)[live]).abs().max() < 4 * R.U * 70 * 50 + R.U * 800
    up = torch.full((rows,), 1.0, device=DEV)
    dx, dw = L.linear_cross_entropy_bw(x, w, t, lse, up)
    q = torch.exp(z - lse.double()[:, None])
    q[torch.arange(rows), t.clamp(min=0).long()] -= 1
    q[~live] = 0
    for v in (0, 1, 2097151, 2097152, V - 1):
        want_v = q[:, v] @ x.double()
        mag = q[:, v].abs() @ x.double().abs()
        assert ((dw[v].double() - want_v).abs() <= 2.0 ** -8 * (want_v.abs() + 1.1 * mag) + 1e-30).all()
    ref = sum(q[:, i:i + 100000] @ w[i:i + 100000].double() for i in range(0, V, 100000))
    mag = sum(q[:, i:i + 100000].abs() @ w[i:i + 100000].double().abs()
              for i in range(0, V, 100000))
    assert ((dx.double() - ref).abs() <= 2.0 ** -8 * (ref.abs() + 1.5 * mag) + 1e-30).all()
    assert (dx[~live] == 0).all()
