"""GPU parity of the softmax with a relative position bias, the per-head norm
with rotation and the gradient clipping with their 64-bit references, at the
sizes, masks, alignments and call forms where they can go wrong."""
import math

import pytest
import torch

import _position_ref as R

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
INF = math.inf


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from transformer_reduce_gb300 import build
    build.build()
    import transformer_reduce_gb300 as L
    L.load()
    return L


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _randn(shape, dtype, seed, std=1.0):
    return (torch.randn(shape, generator=_gen(seed), device=DEV) * std).to(dtype)


# ---------------------------------------------------------------------------
# softmax with a relative position bias
# ---------------------------------------------------------------------------
def _mask(kind, B, Tk, dtype, seed=0):
    """none | pad (batch entry 0 keeps nothing when B > 1) | holes | lowest | mixed"""
    if kind == "none":
        return None
    g = torch.Generator().manual_seed(seed + 17)
    n = torch.randint(1, Tk + 1, (B,), generator=g)
    if B > 1:
        n[0] = 0
        n[1] = Tk
    m = torch.zeros(B, Tk)
    fill = torch.finfo(dtype).min if kind == "lowest" else -INF
    for b in range(B):
        m[b, int(n[b]):] = fill
    if kind in ("holes", "mixed"):
        m = torch.where(torch.rand(B, Tk, generator=g) < 0.3, torch.tensor(-INF), m)
    if kind == "mixed":
        m = m + torch.randn(B, Tk, generator=g)
        if B > 1:
            m[0] = torch.finfo(dtype).min
    return m.to(dtype).to(DEV)


def _relpos(L, shape, dt, nb=32, dist=128, mask="none", causal=False, scale=1.0, seed=1,
            both=True):
    B, H, Tq, Tk = shape
    dtype = DT[dt]
    buckets = L.relpos_buckets(nb, dist, both, device=DEV)
    table = _randn((nb, H), dtype, seed + 1, 0.8)
    x = _randn(shape, dtype, seed, 2.0 / scale)
    m = _mask(mask, B, Tk, dtype, seed)
    return x, table, buckets, m


def _check_relpos(L, shape, dt, nb=32, dist=128, mask="none", causal=False, scale=1.0, seed=1,
                  both=True):
    x, table, buckets, m = _relpos(L, shape, dt, nb, dist, mask, causal, scale, seed, both)
    y = L.softmax_fw_relpos(x, table, buckets, m, causal=causal, scale=scale)
    want, tol = R.relpos_fw(x, table, buckets, m, causal, scale)
    R.check(y, want, tol, f"fw {shape} {dt} {mask}")
    y_in = want.to(DT[dt])
    dout = _randn(shape, DT[dt], seed + 2)
    dx, dtab = L.softmax_bw_relpos(dout, y_in, buckets, nb, m, causal=causal, scale=scale)
    (wx, tx), (wt, tt) = R.relpos_bw(dout, y_in, buckets, nb, m, causal, scale)
    R.check(dx, wx, tx, f"bw {shape} {dt} {mask}")
    R.check(dtab, wt, tt, f"table {shape} {dt} {mask}")


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("Tk", [1, 2, 3, 7, 8, 9, 31, 32, 33, 64, 100, 127, 128, 129, 255, 256,
                                257, 300, 384, 511, 512, 513])
def test_relpos_lengths(lib, dt, Tk):
    _check_relpos(lib, (2, 3, Tk, Tk), dt, mask="pad", scale=0.5, seed=Tk)
    _check_relpos(lib, (1, 2, min(Tk, 5), Tk), dt, causal=True, seed=Tk + 1)


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("Tk", [768, 1000, 1001, 1024, 1030, 2040, 2048, 2049, 4000, 4096, 4101,
                                8192, 16384, 16390, 20000])
def test_relpos_long_rows(lib, dt, Tk):
    _check_relpos(lib, (2, 2, 3, Tk), dt, mask="pad", causal=True, scale=0.125, seed=Tk)
    _check_relpos(lib, (3, 2, 1, Tk), dt, mask="lowest", seed=Tk + 1)


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("mask", ["none", "pad", "holes", "lowest", "mixed"])
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("shape", [(3, 2, 40, 40), (3, 5, 17, 264), (2, 3, 77, 203)])
def test_relpos_masks(lib, dt, mask, causal, shape):
    _check_relpos(lib, shape, dt, nb=16, dist=24, mask=mask, causal=causal, scale=0.7)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("nb,dist,both", [(4, 2, True), (2, 5, False), (8, 1000, True),
                                          (512, 300, True), (64, 2048, True), (7, 33, False)])
def test_relpos_bucket_maps(lib, dt, nb, dist, both):
    _check_relpos(lib, (2, 2, 130, 130), dt, nb=nb, dist=dist, both=both)
    _check_relpos(lib, (1, 2, 3, 2100), dt, nb=nb, dist=dist, both=both, causal=True)


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("shape", [(2, 3, 50, 8), (2, 2, 300, 33), (1, 2, 1000, 264)])
def test_relpos_more_queries_than_keys(lib, dt, shape):
    _check_relpos(lib, shape, dt, mask="pad", nb=32, dist=200)


@pytest.mark.parametrize("shape", [(1, 1, 1, 1), (700, 1, 1, 64), (70, 3, 2, 16), (2, 150, 3, 40),
                                   (33, 20, 1, 1001), (1, 1, 5000, 16)])
def test_relpos_batch_and_head_counts(lib, shape):
    """Blocks that span many batch entries or many heads."""
    for mask in ("pad", "mixed"):
        _check_relpos(lib, shape, "bf16", mask=mask, seed=3)


def test_relpos_one_bucket_per_distance_and_ids_outside(lib):
    L = lib
    dist, nb = 9, 19
    buckets = torch.arange(2 * dist + 1, dtype=torch.int32, device=DEV)
    buckets[3], buckets[12], buckets[18] = -1, nb, 2 ** 31 - 1
    shape = (2, 3, 21, 48)
    x, table = _randn(shape, torch.float32, 5, 2.0), _randn((nb, 3), torch.float32, 6)
    y = L.softmax_fw_relpos(x, table, buckets)
    want, tol = R.relpos_fw(x, table, buckets, None, False, 1.0)
    R.check(y, want, tol, "fw")
    dout = _randn(shape, torch.float32, 7)
    dx, dt = L.softmax_bw_relpos(dout, y, buckets, nb)
    (wx, tx), (wt, tt) = R.relpos_bw(dout, y, buckets, nb, None, False, 1.0)
    R.check(dx, wx, tx, "dx")
    R.check(dt, wt, tt, "dtable")
    assert torch.all(dt[[3, 12, 18]] == 0)


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("Tk", [40, 45, 512, 2049, 17000])
def test_relpos_infinities_and_nan(lib, dt, Tk):
    """NaN and infinities at invisible keys never matter; at visible ones the
    row follows the formula: +inf or NaN make it NaN, -inf gets weight 0, a
    row of -inf alone is zeros."""
    L, dtype = lib, DT[dt]
    shape = (2, 2, 40, Tk)
    x, table, buckets, _ = _relpos(L, shape, dt, nb=8, dist=16)
    mask = torch.zeros(2, Tk, device=DEV)
    mask[:, Tk // 2:] = -INF
    mask[:, 3] = -INF
    mask = mask.to(dtype)
    clean = L.softmax_fw_relpos(x, table, buckets, mask)
    bad = x.clone()
    bad[..., Tk // 2::2] = float("nan")
    bad[..., Tk // 2 + 1::2] = INF
    bad[..., 3] = float("nan")
    assert torch.equal(L.softmax_fw_relpos(bad, table, buckets, mask), clean)
    dout = _randn(shape, dtype, 9)
    gx, gt = L.softmax_bw_relpos(dout, clean, buckets, 8, mask)
    bad_d, bad_y = dout.clone(), clean.clone()
    for t in (bad_d, bad_y):
        t[..., Tk // 2::2] = float("nan")
        t[..., Tk // 2 + 1::2] = INF
        t[..., 3] = -INF
    bx, bt = L.softmax_bw_relpos(bad_d, bad_y, buckets, 8, mask)
    assert torch.equal(bx, gx) and torch.equal(bt, gt)
    # future keys
    tri = torch.ones(40, Tk, device=DEV).triu(Tk - 40 + 1).bool()
    f = x.masked_fill(tri, float("nan"))
    y = L.softmax_fw_relpos(x, table, buckets, causal=True)
    assert torch.equal(L.softmax_fw_relpos(f, table, buckets, causal=True), y)
    hx, ht = L.softmax_bw_relpos(dout, y, buckets, 8, causal=True)
    fx, ft = L.softmax_bw_relpos(dout.masked_fill(tri, float("nan")), y, buckets, 8, causal=True)
    assert torch.equal(fx, hx) and torch.equal(ft, ht)
    # visible keys
    v = x.clone()
    v[0, 0, 0, 1] = float("nan")
    v[0, 0, 1, 2] = INF
    v[0, 0, 2, :] = -INF
    v[0, 0, 3, ::2] = -INF
    y = L.softmax_fw_relpos(v, table, buckets, mask)
    seen = mask[0] != -INF
    assert torch.all(y[0, 0, 0][seen].isnan()) and torch.all(y[0, 0, 1][seen].isnan())
    assert torch.all(y[0, 0, :, :][:, ~seen] == 0)
    assert torch.all(y[0, 0, 2] == 0) and torch.all(y[0, 0, 3, ::2] == 0)
    want, tol = R.relpos_fw(v, table, buckets, mask, False, 1.0)
    R.check(y[0, 0, 3:], want[0, 0, 3:], tol[0, 0, 3:], "rows after")
    R.check(y[1], want[1], tol[1], "other batch entry")


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("Tk", [24, 100, 512, 1001, 5000, 20000])
def test_relpos_lowest_value_everywhere(lib, dt, Tk):
    """A row whose every key carries the type's lowest value is still a softmax."""
    L, dtype = lib, DT[dt]
    shape = (2, 2, 3, Tk)
    x, table, buckets, _ = _relpos(L, shape, dt)
    mask = torch.full((2, Tk), torch.finfo(dtype).min, device=DEV, dtype=dtype)
    y = L.softmax_fw_relpos(x, table, buckets, mask)
    want, tol = R.relpos_fw(x, table, buckets, mask, False, 1.0)
    R.check(y, want, tol, "lowest")
    assert torch.allclose(y.float().sum(-1), torch.ones(2, 2, 3, device=DEV), atol=2e-2)


def _shifted(t, k):
    """A dense copy of t that starts k elements into its storage."""
    buf = torch.empty(t.numel() + k + 64, dtype=t.dtype, device=DEV)
    v = buf[k:k + t.numel()].view(t.shape)
    return v.copy_(t)


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("Tk", [16, 45, 512, 1001])
@pytest.mark.parametrize("shifts", [(1, 1), (3, 0), (0, 5), (8, 8)])
def test_relpos_in_place_and_misaligned(lib, dt, Tk, shifts):
    L = lib
    shape = (2, 2, 9, Tk)
    x, table, buckets, m = _relpos(L, shape, dt, mask="pad")
    want, tol = R.relpos_fw(x, table, buckets, m, False, 1.0)
    a, b = _shifted(x, shifts[0]), _shifted(torch.zeros_like(x), shifts[1])
    mm = _shifted(m, 1)
    L.softmax_fw_relpos(a, _shifted(table, 1), buckets, mm, out=b)
    R.check(b, want, tol, "shifted")
    L.softmax_fw_relpos(a, table, buckets, m, out=a)
    R.check(a, want, tol, "in place")
    y, dout = b, _randn(shape, DT[dt], 4)
    (wx, tx), (wt, tt) = R.relpos_bw(dout, y, buckets, 32, m, False, 1.0)
    g = _shifted(dout, shifts[0])
    dx, dtab = L.softmax_bw_relpos(g, y, buckets, 32, mm, dinp=_shifted(dout, shifts[1] + 2))
    R.check(dx, wx, tx, "dx shifted")
    R.check(dtab, wt, tt, "table shifted")
    dx, dtab = L.softmax_bw_relpos(g, y, buckets, 32, m, dinp=g)
    R.check(g, wx, tx, "dx in place")
    R.check(dtab, wt, tt, "table in place")


@pytest.mark.parametrize("Tk", [45, 2100])
def test_relpos_looped_path_infinities_and_nan(lib, Tk):
    """The looped kernels (tensors at different offsets within 16 bytes)."""
    L = lib
    shape = (2, 2, 12, Tk)
    x, table, buckets, _ = _relpos(L, shape, "f16", nb=8, dist=16)
    mask = torch.zeros(2, Tk, device=DEV, dtype=torch.float16)
    mask[:, Tk // 2:] = -INF
    x[0, 0, 0, 1] = float("nan")
    x[0, 0, 1, 2] = INF
    x[0, 0, 2, :] = -INF
    x[0, 0, 3, ::2] = -INF
    x[..., Tk // 2:] = float("nan")
    out = _shifted(torch.zeros_like(x), 1)
    y = L.softmax_fw_relpos(x, table, buckets, mask, out=out)
    seen = mask[0] == 0
    assert torch.all(y[0, 0, 0][seen].isnan()) and torch.all(y[0, 0, 1][seen].isnan())
    assert torch.all(y[..., ~seen] == 0) and torch.all(y[0, 0, 2] == 0)
    want, tol = R.relpos_fw(x, table, buckets, mask, False, 1.0)
    R.check(y[0, 0, 3:], want[0, 0, 3:], tol[0, 0, 3:], "rows after")
    dout = _randn(shape, torch.float16, 9)
    good = y.nan_to_num()
    d1, t1 = L.softmax_bw_relpos(_shifted(dout, 1), good, buckets, 8, mask)
    bad = dout.clone()
    bad[..., Tk // 2:] = float("nan")
    d2, t2 = L.softmax_bw_relpos(_shifted(bad, 1), good, buckets, 8, mask)
    assert torch.equal(d1, d2) and torch.equal(t1, t2) and torch.all(d1[..., ~seen] == 0)


def test_relpos_bw_many_rows_per_block_and_few_buckets(lib):
    """Long runs of rows of every alignment, whose phases change with the batch entry."""
    for shape, causal in (((7, 3, 701, 40), False), ((9, 2, 333, 130), False),
                          ((5, 4, 257, 257), True), ((40, 3, 17, 66), False)):
        for dt in ("bf16", "f32"):
            _check_relpos(lib, shape, dt, nb=8, dist=60, mask="pad", causal=causal)


def test_relpos_empty_problems(lib):
    L = lib
    buckets = L.relpos_buckets(8, 5, device=DEV)
    for shape in ((0, 2, 3, 4), (2, 2, 0, 4), (2, 2, 3, 0)):
        x = torch.empty(shape, device=DEV)
        assert L.softmax_fw_relpos(x, torch.ones(8, 2, device=DEV), buckets).shape == shape
        dt = torch.full((8, 2), 7.0, device=DEV)
        L.softmax_bw_relpos(x, x, buckets, 8, dtable=dt)
        assert torch.all(dt == 0)
    x = torch.empty(2, 0, 3, 4, device=DEV)
    assert L.softmax_bw_relpos(x, x, buckets, 8)[1].shape == (8, 0)


@pytest.mark.parametrize("dt,shape", [("bf16", (2, 3, 9, 264)), ("f16", (2, 3, 9, 261)),
                                      ("f32", (1, 2, 3, 5001)), ("bf16", (4, 3, 5, 16))])
def test_relpos_stays_inside_its_buffers(lib, dt, shape):
    L, dtype = lib, DT[dt]
    x, table, buckets, m = _relpos(L, shape, dt, mask="pad")
    n = x.numel()

    def framed(numel, dtp):
        buf = torch.full((numel + 128,), 77.0, dtype=dtp, device=DEV)
        return buf, buf[64:64 + numel]

    def intact(buf, numel):
        return bool(torch.all(buf[:64] == 77.0) and torch.all(buf[64 + numel:] == 77.0))

    ob, o = framed(n, dtype)
    y = L.softmax_fw_relpos(x, table, buckets, m, out=o.view(shape))
    gb, g = framed(n, dtype)
    tb, t = framed(32 * shape[1], torch.float32)
    need = L.ls_softmax_bw_relpos_workspace_size(shape[1], 128) // 4
    wb, w = framed(need, torch.float32)
    L.softmax_bw_relpos(_randn(shape, dtype, 3), y, buckets, 32, m, dinp=g.view(shape),
                        dtable=t.view(32, shape[1]), workspace=w)
    torch.cuda.synchronize()
    assert intact(ob, n) and intact(gb, n) and intact(tb, 32 * shape[1]) and intact(wb, need)


# ---------------------------------------------------------------------------
# per-head norm with rotation
# ---------------------------------------------------------------------------
def _qk(L, tokens, Hq, Hk, D, rot, dt, packed=False, seed=1, max_pos=50):
    dtype = DT[dt]
    if packed:
        qkv = _randn((tokens, (Hq + 2 * Hk) * D), dtype, seed, 1.5)
        q = qkv[:, :Hq * D].view(tokens, Hq, D)
        k = qkv[:, Hq * D:(Hq + Hk) * D].view(tokens, Hk, D)
    else:
        q, k = _randn((tokens, Hq, D), dtype, seed, 1.5), _randn((tokens, Hk, D), dtype, seed + 1, 0.4)
    gq = (1 + 0.3 * torch.randn(D, generator=_gen(seed + 2), device=DEV)).to(dtype)
    gk = (1 + 0.3 * torch.randn(D, generator=_gen(seed + 3), device=DEV)).to(dtype)
    cos = sin = pos = None
    if rot:
        cos, sin = L.rope_tables(max_pos, rot, device=DEV)
        pos = torch.randint(0, max_pos, (tokens,), generator=_gen(seed + 4), device=DEV,
                            dtype=torch.int32)
    return q, k, gq, gk, cos, sin, pos


def _check_qk(L, tokens, Hq, Hk, D, rot, dt, interleaved=False, packed=False, seed=1, eps=1e-6):
    q, k, gq, gk, cos, sin, pos = _qk(L, tokens, Hq, Hk, D, rot, dt, packed, seed)
    what = f"{tokens}x({Hq},{Hk})x{D} rot {rot} {dt} il {interleaved} packed {packed}"
    out = L.qk_norm_rope_fw(q, k, gq, gk, cos, sin, pos, interleaved=interleaved, eps=eps)
    rs = []
    for x, g, y, r in ((q, gq, out[0], out[2]), (k, gk, out[1], out[3])):
        (wy, ty), (wr, tr) = R.qk_fw(x, g, cos, sin, pos, interleaved, eps)
        R.check(y, wy, ty, "y " + what)
        R.check(r, wr, tr, "rstd " + what)
        rs.append(wr.float())
    dqo, dko, *_ = _qk(L, tokens, Hq, Hk, D, 0, dt, packed, seed + 10)
    got = L.qk_norm_rope_bw(dqo, dko, q, k, gq, gk, *rs, cos, sin, pos, interleaved=interleaved)
    for x, g, d, r, dx, dg in ((q, gq, dqo, rs[0], got[0], got[2]),
                               (k, gk, dko, rs[1], got[1], got[3])):
        (wx, tx), (wg, tg) = R.qk_bw(d, x, g, r, cos, sin, pos, interleaved)
        R.check(dx, wx, tx, "dx " + what)
        R.check(dg, wg, tg, "dgamma " + what)


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("D,rot", [(64, 64), (128, 128), (128, 64), (256, 256), (80, 80), (96, 48),
                                   (32, 32), (16, 16), (8, 8), (64, 0), (72, 36), (160, 160),
                                   (512, 512), (1024, 1024), (1000, 500), (128, 16), (64, 8)])
def test_qk_head_sizes(lib, dt, interleaved, D, rot):
    _check_qk(lib, 37, 6, 2, D, rot, dt, interleaved, packed=True)


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("D,rot", [(1, 0), (2, 2), (3, 2), (5, 4), (7, 0), (33, 32), (63, 62),
                                   (101, 50), (255, 254), (66, 66)])
def test_qk_odd_head_sizes(lib, dt, D, rot):
    _check_qk(lib, 23, 3, 2, D, rot, dt, interleaved=bool(D % 2))
    _check_qk(lib, 5, 2, 3, D, rot, dt, interleaved=not D % 2, packed=True)


@pytest.mark.parametrize("tokens", [1, 2, 3, 8, 31, 64, 129, 1000, 3001])
@pytest.mark.parametrize("Hq,Hk", [(1, 1), (8, 8), (9, 3), (32, 8), (7, 1), (40, 8)])
def test_qk_counts(lib, tokens, Hq, Hk):
    _check_qk(lib, tokens, Hq, Hk, 64, 64, "bf16", packed=True, seed=tokens)


@pytest.mark.parametrize("dt", list(DT))
def test_qk_many_heads_and_one_side(lib, dt):
    L = lib
    _check_qk(L, 3, 300, 1, 32, 32, dt)
    _check_qk(L, 3, 1, 300, 32, 32, dt)
    q, k, gq, gk, cos, sin, pos = _qk(L, 11, 4, 0, 32, 32, dt)
    y, ky, r, kr = L.qk_norm_rope_fw(q, k, gq, gk, cos, sin, pos)
    assert ky.shape == (11, 0, 32) and kr.shape == (11, 0)
    (wy, ty), (wr, _) = R.qk_fw(q, gq, cos, sin, pos, False, 1e-6)
    R.check(y, wy, ty, "queries alone")
    d = _randn(q.shape, DT[dt], 8)
    dx, _, dg, dgk = L.qk_norm_rope_bw(d, k, q, k, gq, gk, r, kr, cos, sin, pos)
    (wx, tx), (wg, tg) = R.qk_bw(d, q, gq, r, cos, sin, pos, False)
    R.check(dx, wx, tx, "dq alone")
    R.check(dg, wg, tg, "dgamma alone")
    assert torch.all(dgk == 0)


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("D,rot", [(64, 64), (65, 64), (48, 16)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_qk_in_place_and_misaligned(lib, dt, D, rot, interleaved):
    L, dtype = lib, DT[dt]
    T, Hq, Hk = 19, 4, 2
    q, k, gq, gk, cos, sin, pos = _qk(L, T, Hq, Hk, D, rot, dt)
    width = (Hq + Hk) * D + 3  # tokens off every 16-byte boundary
    buf = torch.full((T * width + 8,), 5.0, device=DEV, dtype=dtype)
    qv = buf[1:1 + T * width].view(T, width)[:, :Hq * D].view(T, Hq, D)
    kv = buf[1:1 + T * width].view(T, width)[:, Hq * D:(Hq + Hk) * D].view(T, Hk, D)
    qv.copy_(q)
    kv.copy_(k)
    want = [R.qk_fw(x, g, cos, sin, pos, interleaved, 1e-6) for x, g in ((q, gq), (k, gk))]
    out = L.qk_norm_rope_fw(qv, kv, _shifted(gq, 1), _shifted(gk, 3), _shifted(cos, 1),
                            _shifted(sin, 1), pos, interleaved=interleaved)
    for y, w in zip(out[:2], want):
        R.check(y, *w[0], "misaligned")
    rq, rk = out[2], out[3]
    L.qk_norm_rope_fw(qv, kv, gq, gk, cos, sin, pos, interleaved=interleaved, q_out=qv, k_out=kv)
    for y, w in zip((qv, kv), want):
        R.check(y, *w[0], "in place")
    dq, dk = _randn(q.shape, dtype, 5), _randn(k.shape, dtype, 6)
    wb = [R.qk_bw(d, x, g, r, cos, sin, pos, interleaved)
          for d, x, g, r in ((dq, q, gq, rq), (dk, k, gk, rk))]
    qv.copy_(dq)
    kv.copy_(dk)
    got = L.qk_norm_rope_bw(qv, kv, q, k, gq, gk, rq, rk, cos, sin, pos, interleaved=interleaved,
                            dq=qv, dk=kv)
    for dx, dg, w in ((qv, got[2], wb[0]), (kv, got[3], wb[1])):
        R.check(dx, *w[0], "dx in place")
        R.check(dg, *w[1], "dgamma in place")
    rest = buf.clone()
    rest[1:1 + T * width].view(T, width)[:, :(Hq + Hk) * D] = 5.0
    assert torch.all(rest == 5.0)  # nothing written between the tokens or around them


def test_qk_positions_outside_the_table(lib):
    L = lib
    q, k, gq, gk, cos, sin, pos = _qk(L, 6, 2, 1, 64, 32, "f32")
    pos[1], pos[3], pos[4] = -1, 50, 2 ** 31 - 1
    out = L.qk_norm_rope_fw(q, k, gq, gk, cos, sin, pos)
    for x, g, y, r in ((q, gq, out[0], out[2]), (k, gk, out[1], out[3])):
        (wy, ty), (wr, tr) = R.qk_fw(x, g, cos, sin, pos, False, 1e-6)
        R.check(y, wy, ty, "y")
        R.check(r, wr, tr, "rstd")
        assert torch.all(y[1, :, :32].isnan()) and not torch.any(y[1, :, 32:].isnan())
    d = _randn(q.shape, torch.float32, 7)
    dx, _, dg, _ = L.qk_norm_rope_bw(d, _randn(k.shape, torch.float32, 8), q, k, gq, gk, out[2],
                                     out[3], cos, sin, pos)
    assert torch.all(dx[[1, 3, 4]].isnan()) and torch.all(dx[[0, 2, 5]].isfinite())
    assert torch.all(dg[:32].isnan()) and torch.all(dg[32:].isfinite())


def test_qk_zero_rows_nan_rows_and_no_tokens(lib):
    L = lib
    q, k, gq, gk, cos, sin, pos = _qk(L, 4, 2, 2, 64, 64, "bf16")
    q[1] = 0
    k[2, 1, 5] = float("nan")
    y, ky, r, kr = L.qk_norm_rope_fw(q, k, gq, gk, cos, sin, pos)
    assert torch.all(y[1] == 0) and torch.allclose(r[1], torch.full((2,), 1e3, device=DEV))
    assert torch.all(ky[2, 1].isnan()) and torch.all(ky[2, 0].isfinite())
    e = torch.empty(0, 2, 64, device=DEV, dtype=torch.bfloat16)
    p0 = pos[:0]
    out = L.qk_norm_rope_fw(e, e, gq, gk, cos, sin, p0)
    assert out[0].shape == (0, 2, 64)
    g1, g2 = torch.full((64,), 3.0, device=DEV), torch.full((64,), 3.0, device=DEV)
    L.qk_norm_rope_bw(e, e, e, e, gq, gk, out[2], out[3], cos, sin, p0, dgamma_q=g1, dgamma_k=g2)
    assert torch.all(g1 == 0) and torch.all(g2 == 0)


# ---------------------------------------------------------------------------
# gradient norm and clipping
# ---------------------------------------------------------------------------
def _check_clip(L, grads, max_norm, eps=1e-6):
    (wn, tn), outs = R.clip(grads, max_norm, eps)
    R.check(L.grad_norm(grads), wn, tn, "norm")
    out = [torch.full_like(g, 9.0) for g in grads]
    got, norm = L.grad_clip(grads, max_norm, out=out, eps=eps)
    R.check(norm, wn, tn, "clip norm")
    for i, (o, (w, t)) in enumerate(zip(got, outs)):
        R.check(o, w, t, f"out[{i}]")
    inp = [g.clone() for g in grads]
    same, norm2 = L.grad_clip(inp, max_norm, eps=eps)
    assert all(a is b for a, b in zip(same, inp)) and torch.equal(norm, norm2)
    assert all(torch.equal(a, b) for a, b in zip(inp, out))


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("n", [1, 2, 7, 8, 9, 1023, 16383, 16384, 16385, 40000, 1000003])
@pytest.mark.parametrize("max_norm", [0.5, 1e6])
def test_clip_one_tensor(lib, dt, n, max_norm):
    _check_clip(lib, [_randn((n,), DT[dt], n)], max_norm)


@pytest.mark.parametrize("count", [2, 47, 48, 49, 300, 511, 512, 513, 1100])
def test_clip_many_mixed_tensors(lib, count):
    g = torch.Generator().manual_seed(count)
    sizes = torch.randint(0, 3000, (count,), generator=g).tolist()
    sizes[0] = 0
    sizes[-1] = 70000
    kinds = list(DT.values())
    grads = [_randn((n,), kinds[i % 3], i, 0.1 * (1 + i % 5)) for i, n in enumerate(sizes)]
    _check_clip(lib, grads, 2.0)


def test_clip_views_of_one_buffer_at_every_alignment(lib):
    for dt in DT.values():
        sizes = [1, 2, 3, 5, 16, 31, 32, 33, 100, 4099, 2, 1, 20000, 7]
        buf = _randn((sum(sizes) + 3,), dt, 3)
        grads = list(buf[3:].split(sizes))
        _check_clip(lib, grads, 1.0)
        # outputs at another alignment than their gradients; nothing around them is written
        out = torch.full((sum(sizes) + 9,), 9.0, device=DEV, dtype=dt)
        outs = list(out[4:4 + sum(sizes)].split(sizes))
        lib.grad_clip(grads, 1.0, out=outs)
        (_, _), want = R.clip(grads, 1.0, 1e-6)
        for o, (w, t) in zip(outs, want):
            R.check(o, w, t, "other alignment")
        assert torch.all(out[:4] == 9.0) and torch.all(out[4 + sum(sizes):] == 9.0)
        # in place, between neighbours that are not in the list
        keep = buf.clone()
        lib.grad_clip(grads[1::2], 1.0)
        for i, (a, b) in enumerate(zip(grads, keep[3:].split(sizes))):
            assert i % 2 == 1 or torch.equal(a, b)


def test_clip_extreme_values(lib):
    L = lib
    f32, bf = torch.float32, torch.bfloat16
    _check_clip(L, [torch.full((1000,), 1e30, device=DEV), _randn((77,), bf, 1)], 1.0)
    _check_clip(L, [torch.full((1000,), 1e-30, device=DEV, dtype=f32)], 1e-31, eps=0.0)
    _check_clip(L, [torch.full((999,), 2e38, device=DEV, dtype=bf)[:2]], 1.0)
    _check_clip(L, [torch.full((3,), 1e-45, device=DEV)], 1.0, eps=0.0)
    _check_clip(L, [torch.zeros(5000, device=DEV), torch.zeros(3, device=DEV, dtype=bf)], 1.0)
    _check_clip(L, [torch.zeros(5000, device=DEV)], 1.0, eps=0.0)
    # past fp32: the norm is inf, finite gradients become 0
    g = [torch.full((1000,), 3e38, device=DEV)]
    out, norm = L.grad_clip(g, 1.0)
    assert torch.isposinf(norm).all() and torch.all(out[0] == 0)
    g = [torch.ones(10, device=DEV), torch.tensor([1.0, INF], device=DEV)]
    out, norm = L.grad_clip(g, 1.0)
    assert torch.isposinf(norm).all() and torch.all(out[0] == 0) and bool(out[1][1].isnan())
    g = [torch.ones(10, device=DEV), torch.tensor([1.0, float("nan")], device=DEV)]
    out, norm = L.grad_clip(g, 1.0)
    assert norm.isnan().all() and out[0].isnan().all() and out[1].isnan().all()


def test_clip_leaves_what_needs_no_clipping(lib):
    g = [_randn((5000,), dt, i) for i, dt in enumerate(DT.values())]
    keep = [t.clone() for t in g]
    lib.grad_clip(g, 1e4)
    assert all(torch.equal(a, b) for a, b in zip(g, keep))
    # no gradient at all
    e = [torch.empty(0, device=DEV), torch.empty(0, 3, device=DEV, dtype=torch.float16)]
    out, norm = lib.grad_clip(e, 1.0)
    assert float(norm) == 0.0 and float(lib.grad_norm(e)) == 0.0


# ---------------------------------------------------------------------------
# together, reproducibility, streams and graphs
# ---------------------------------------------------------------------------
def _layer(L, dt, seed=1, T=48, B=3, H=4, D=32, rot=16):
    """Inputs of one attention layer's training step."""
    dtype = DT[dt]
    q, k, gq, gk, cos, sin, _ = _qk(L, B * T, H, H, D, rot, dt, packed=True, seed=seed, max_pos=T)
    pos = torch.arange(T, dtype=torch.int32, device=DEV).repeat(B)
    mask = _mask("pad", B, T, dtype, seed)
    mask[0] = 0
    return dict(q=q, k=k, gq=gq, gk=gk, cos=cos, sin=sin, pos=pos, mask=mask, B=B, T=T, H=H, D=D,
                table=_randn((32, H), dtype, seed + 5, 0.5), buckets=L.relpos_buckets(device=DEV),
                dy=_randn((B, H, T, T), dtype, seed + 6))


def _step(L, s, ws=None):
    """Norm and rotation, scores, softmax, and back to the clipped gradients."""
    B, T, H, D = s["B"], s["T"], s["H"], s["D"]
    ws = ws or {}

    def split(t):  # [B*T, H, D] -> [B, H, T, D]
        return t.view(B, T, H, D).transpose(1, 2)

    def join(t):
        return t.transpose(1, 2).reshape(B * T, H, D)

    qn, kn, rq, rk = L.qk_norm_rope_fw(s["q"], s["k"], s["gq"], s["gk"], s["cos"], s["sin"],
                                       s["pos"])
    scores = split(qn) @ split(kn).transpose(-1, -2)
    y = L.softmax_fw_relpos(scores, s["table"], s["buckets"], s["mask"], causal=True,
                            scale=D ** -0.5)
    ds, dtable = L.softmax_bw_relpos(s["dy"], y, s["buckets"], 32, s["mask"], causal=True,
                                     scale=D ** -0.5, workspace=ws.get("soft"))
    dqn, dkn = join(ds @ split(kn)), join(ds.transpose(-1, -2) @ split(qn))
    dq, dk, dgq, dgk = L.qk_norm_rope_bw(dqn, dkn, s["q"], s["k"], s["gq"], s["gk"], rq, rk,
                                         s["cos"], s["sin"], s["pos"], workspace=ws.get("qk"))
    grads = [dq, dk, dgq, dgk, dtable]
    clipped, norm = L.grad_clip(grads, 0.5, out=[torch.empty_like(g) for g in grads],
                                workspace=ws.get("clip"))
    return [y, ds, *grads, *clipped, norm]


def test_layer_step_against_autograd(lib):
    """The operators as a training step uses them, against torch's autograd of
    the whole step in 64 bits (storage fp32: only fp32 roundings remain)."""
    L = lib
    s = _layer(L, "f32")
    got = _step(L, s)
    B, T, H, D = s["B"], s["T"], s["H"], s["D"]
    leaf = {n: s[n].double().detach().contiguous().requires_grad_()
            for n in ("q", "k", "gq", "gk", "table")}

    def norm(x, g):
        n = x * (x.square().mean(-1, keepdim=True) + 1e-6).rsqrt() * g
        return R.rotate(n, s["cos"], s["sin"], s["pos"], False).view(B, T, H, D).transpose(1, 2)

    ids, seen = R.relpos_pairs(T, T, s["buckets"], 32, True, DEV)
    z = norm(leaf["q"], leaf["gq"]) @ norm(leaf["k"], leaf["gk"]).transpose(-1, -2) * D ** -0.5
    z = z + leaf["table"][ids].permute(2, 0, 1) + s["mask"].double()[:, None, None, :]
    z = z.masked_fill(~seen, -1e30).clamp(min=-1e30)
    vis = R.relpos_visible(z.shape, s["mask"], seen)
    y = torch.softmax(z, -1) * vis
    (y * s["dy"].double()).sum().backward()
    want = [leaf[n].grad for n in ("q", "k", "gq", "gk", "table")]
    total = sum((g * g).sum() for g in want) ** 0.5
    # fp32 through four kernels and products of 32 to 48 terms: 1e-5 of the largest value is
    # over 100 u, where each stage gives at most some tens
    assert float((got[0].double() - y.detach()).abs().max()) <= 1e-5
    for g, w in zip(got[2:7], want):
        assert float((g.double() - w).abs().max()) <= 1e-5 * max(1.0, float(w.abs().max()))
    assert abs(float(got[-1]) / float(total) - 1) <= 1e-5
    for c, w in zip(got[7:12], want):
        w = w * min(1.0, 0.5 / float(total))
        assert float((c.double() - w).abs().max()) <= 1e-5 * max(1.0, float(w.abs().max()))


@pytest.mark.parametrize("dt", ["f16", "bf16"])
def test_layer_step_is_reproducible_on_any_stream(lib, dt):
    L = lib
    s = _layer(L, dt, T=101)
    torch.cuda.synchronize()
    want = _step(L, s)
    again = _step(L, s)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = _step(L, s)
    torch.cuda.synchronize()
    for w, a, o in zip(want, again, other):
        assert torch.equal(w, a) and torch.equal(w, o)


def test_two_steps_at_once_with_their_own_workspaces(lib):
    L = lib
    states = [_layer(L, "bf16", seed=20 * i + 1, T=64 + 8 * i) for i in range(2)]
    want = [_step(L, s) for s in states]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in states]
    got = [None, None]
    for _ in range(3):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                got[i] = _step(L, states[i])
    torch.cuda.synchronize()
    for w, g in zip(want, got):
        assert all(torch.equal(a, b) for a, b in zip(w, g))


def test_layer_step_captured_and_replayed(lib):
    """Two graphs of the step, each with its own workspaces, replayed in turn on
    new inputs: the eager step's results, bit for bit."""
    L = lib
    states, graphs, outs, held = [], [], [], []
    for i in range(2):
        s = _layer(L, "bf16", seed=40 + i, T=64)
        ws = {"soft": L.softmax_relpos_workspace(s["H"], 128, DEV),
              "qk": L.qk_norm_rope_workspace(s["B"] * s["T"], s["H"], s["H"], s["D"], DEV),
              "clip": L.grad_norm_workspace(5, DEV)}
        held.append(ws)  # a captured graph goes on writing to its workspaces
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            _step(L, s, ws)
        torch.cuda.current_stream().wait_stream(side)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(_step(L, s, ws))
        states.append(s)
        graphs.append(g)
    for turn in range(2):
        for i in (1, 0):
            new = _layer(L, "bf16", seed=70 + 10 * turn + i, T=64)
            for n, t in new.items():
                if torch.is_tensor(t):
                    states[i][n].copy_(t)
            graphs[i].replay()
            torch.cuda.synchronize()
            want = _step(L, new)
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(outs[i], want))
