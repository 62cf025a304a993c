"""GPU parity of the difference of two softmax maps, the norms around a block and
the cross entropy from hidden states with their 64-bit references, at the
sizes, masks, layouts, alignments and call forms where they can go wrong."""
import math

import pytest
import torch

import _decoder_ref as R

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


def _randn(shape, dtype, seed, std=1.0, mean=0.0):
    return (torch.randn(shape, generator=_gen(seed), device=DEV) * std + mean).to(dtype)


def _shifted(t, by=1):
    """A copy of t that starts `by` elements past a 16-byte address."""
    flat = torch.empty(t.numel() + 16, dtype=t.dtype, device=t.device)
    out = flat[by:by + t.numel()].view(t.shape)
    out.copy_(t)
    return out


# ---------------------------------------------------------------------------
# difference of two softmax maps
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


def _maps(shape, dtype, layout, seed, std):
    B, H, Tq, Tk = shape
    if layout == "apart":
        return _randn(shape, dtype, seed, std), _randn(shape, dtype, seed + 1, std)
    s = _randn((B, 2 * H, Tq, Tk), dtype, seed, std)
    return (s[:, 0::2], s[:, 1::2]) if layout == "pairs" else (s[:, :H], s[:, H:])


def _check_diff(L, shape, dt, mask="none", causal=False, scale=1.0, layout="halves", shared=False,
                seed=1, shift=0, packed=False):
    B, H, Tq, Tk = shape
    dtype = DT[dt]
    x1, x2 = _maps(shape, dtype, layout, seed, 2.0 / scale)
    m = _mask(mask, B, Tk, dtype, seed)
    lam = torch.rand(1 if shared else H, generator=_gen(seed + 2), device=DEV) * 1.5 - 0.3
    dout = _randn(shape, dtype, seed + 3)
    if shift:
        x1, x2, dout = _shifted(x1, shift), _shifted(x2, 3), _shifted(dout, shift)
    what = f"{shape} {dt} {mask} {layout}"
    (y, ytol), (st, stol) = R.diff_fw(x1, x2, lam, m, causal, scale)
    got, stats = L.softmax_fw_diff(x1, x2, lam, m, causal=causal, scale=scale)
    R.check(got, y, ytol, "fw " + what)
    R.check(stats, st, stol, "stats " + what)
    given = st.float().contiguous()
    a, b, l = R.diff_bw(dout, x1, x2, lam, given, m, causal, scale)
    outs = {}
    if packed:  # the gradients of both maps in one tensor, as the scores lie
        d = torch.full((B, 2 * H, Tq, Tk), 7.0, dtype=dtype, device=DEV)
        outs = {"dscores1": d[:, 0::2], "dscores2": d[:, 1::2]}
    elif shift:
        outs = {"dscores1": _shifted(torch.zeros_like(x1), shift),
                "dscores2": _shifted(torch.zeros_like(x1), shift)}
    d1, d2, dl = L.softmax_bw_diff(dout, x1, x2, lam, given, m, causal=causal, scale=scale, **outs)
    R.check(d1, *a, "dx1 " + what)
    R.check(d2, *b, "dx2 " + what)
    R.check(dl, *l, "dlam " + what)


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("Tk", [1, 2, 3, 7, 8, 9, 31, 32, 33, 64, 100, 127, 128, 129, 255, 256, 257,
                                300, 384, 511, 512, 513])
def test_diff_lengths(lib, dt, Tk):
    _check_diff(lib, (2, 3, Tk, Tk), dt, mask="pad", scale=0.5, seed=Tk)
    _check_diff(lib, (1, 2, min(Tk, 5), Tk), dt, causal=True, seed=Tk + 1, layout="pairs")


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("Tk", [768, 1000, 1001, 1024, 2040, 2048, 2049, 4096, 4101, 8192, 16384,
                                16390, 20000])
def test_diff_long_rows(lib, dt, Tk):
    _check_diff(lib, (2, 2, 3, Tk), dt, mask="pad", causal=True, scale=0.125, seed=Tk)
    _check_diff(lib, (3, 2, 1, Tk), dt, mask="lowest", seed=Tk + 1, shared=True)


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("mask", ["none", "pad", "holes", "lowest", "mixed"])
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("shape", [(3, 2, 40, 40), (3, 5, 17, 264), (2, 3, 77, 203)])
def test_diff_masks(lib, dt, mask, causal, shape):
    _check_diff(lib, shape, dt, mask=mask, causal=causal, scale=0.7, layout="pairs")


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("layout", ["apart", "halves", "pairs"])
@pytest.mark.parametrize("Tk", [64, 101])
def test_diff_layouts_and_offsets(lib, dt, layout, Tk):
    _check_diff(lib, (2, 3, 20, Tk), dt, mask="pad", layout=layout, seed=3)
    for shift in (1, 2, 5):
        _check_diff(lib, (2, 3, 20, Tk), dt, mask="pad", layout=layout, seed=4, shift=shift)
    _check_diff(lib, (2, 3, 20, Tk), dt, layout=layout, seed=5, packed=True)


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("shape", [(80, 16, 5, 128), (200, 1, 9, 72), (3, 8, 300, 200),
                                   (4, 700, 2, 40), (2000, 1, 1, 33)])
def test_diff_many_rows(lib, shape, causal):
    """Runs of rows over many heads and batch entries, more of these than a block
    keeps windows for."""
    if causal and shape[2] > shape[3]:  # more queries than keys have no causal order
        with pytest.raises(lib.LsError):
            _check_diff(lib, shape, "bf16", causal=True)
        return
    _check_diff(lib, shape, "bf16", mask="pad", causal=causal, seed=7)
    _check_diff(lib, shape, "f32", causal=causal, seed=8, shared=True)


def test_diff_invisible_scores_and_gradients_do_not_matter(lib):
    L = lib
    for dt in DT:
        for Tk in (64, 77):
            shape = (2, 2, 9, Tk)
            x1, x2 = _maps(shape, DT[dt], "halves", 1, 2.0)
            m = _mask("holes", 2, Tk, DT[dt], 3)
            dout = _randn(shape, DT[dt], 5)
            lam = torch.tensor([0.3, 0.8], device=DEV)
            want = L.softmax_fw_diff(x1, x2, lam, m, causal=True)
            grads = L.softmax_bw_diff(dout, x1, x2, lam, want[1], m, causal=True)
            hid = ~R.visible(shape, m, True, DEV)
            for bad in (INF, -INF, math.nan):
                a, b, g = (t.clone().masked_fill_(hid, bad) for t in (x1, x2, dout))
                got = L.softmax_fw_diff(a, b, lam, m, causal=True)
                assert all(torch.equal(p, q) for p, q in zip(want, got))
                again = L.softmax_bw_diff(g, a, b, lam, want[1], m, causal=True)
                assert all(torch.equal(p, q) for p, q in zip(grads, again))
            assert (got[0][hid] == 0).all() and (grads[0][hid] == 0).all()
            assert (grads[1][hid] == 0).all()


def test_diff_nan_and_infinite_scores_stay_in_their_row(lib):
    L = lib
    for dt in DT:
        x1, x2 = (_randn((1, 2, 6, 40), DT[dt], s) for s in (1, 2))
        m = _mask("none", 1, 40, DT[dt])
        lam = torch.tensor([0.5, 0.25], device=DEV)
        clean, stats = L.softmax_fw_diff(x1, x2, lam, m, causal=True)
        a, b = x1.clone(), x2.clone()
        a[0, 0, 1, 3] = math.nan
        a[0, 1, 2, 0] = INF
        b[0, 0, 3, 5] = math.nan
        b[0, 1, 4, 7] = -INF  # an ordinary score of weight 0
        got, st = L.softmax_fw_diff(a, b, lam, m, causal=True)
        vis = R.visible(x1.shape, m, True, DEV)
        for h, i in ((0, 1), (1, 2), (0, 3)):
            row = vis[0, h, i]
            assert got[0, h, i][row].isnan().all() and (got[0, h, i][~row] == 0).all()
        touched = torch.zeros(1, 2, 6, dtype=torch.bool, device=DEV)
        for h, i in ((0, 1), (1, 2), (0, 3), (1, 4)):
            touched[0, h, i] = True
        assert torch.equal(got[~touched], clean[~touched])
        assert got[0, 1, 4].isfinite().all()
        g = _randn(x1.shape, DT[dt], 9)
        want = L.softmax_bw_diff(g, x1, x2, lam, stats, m, causal=True)
        d1, d2, _ = L.softmax_bw_diff(g, a, b, lam, st, m, causal=True)
        assert torch.equal(d1[~touched], want[0][~touched])
        assert torch.equal(d2[~touched], want[1][~touched])
        assert d1[0, 0, 1][vis[0, 0, 1]].isnan().all() and (d1[0, 0, 1][~vis[0, 0, 1]] == 0).all()


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("big", [63.0, 65.0, 3e4, 1e30])
def test_diff_far_scores(lib, dt, big):
    """Rows whose largest z lies beyond the bound of the fused exponent."""
    L = lib
    x1, x2 = (_randn((1, 2, 5, 96), DT[dt], s) for s in (1, 2))
    x1 = (x1.float() + big).to(DT[dt])
    lam = torch.tensor([0.5], device=DEV)
    (y, tol), (st, stol) = R.diff_fw(x1, x2, lam, None, False, 1.0)
    got, stats = L.softmax_fw_diff(x1, x2, lam)
    R.check(got, y, tol, f"{big}")
    R.check(stats, st, stol, f"{big}")
    g = _randn(x1.shape, DT[dt], 3)
    given = st.float()
    for (want, t), d in zip(R.diff_bw(g, x1, x2, lam, given, None, False, 1.0),
                            L.softmax_bw_diff(g, x1, x2, lam, given)):
        R.check(d, want, t, f"bw {big}")


def test_diff_rows_without_a_finite_score(lib):
    L = lib
    x1, x2 = (_randn((1, 1, 4, 48), torch.float16, s) for s in (1, 2))
    x1[0, 0, 2] = -INF
    lam = torch.tensor([0.5], device=DEV)
    got, stats = L.softmax_fw_diff(x1, x2, lam)
    p2 = torch.softmax(x2[0, 0, 2].double(), -1)
    assert torch.allclose(got[0, 0, 2].double(), -0.5 * p2, atol=1e-4)
    assert stats[0, 0, 2, :2].tolist() == [0.0, 0.0]
    d1, d2, _ = L.softmax_bw_diff(torch.ones_like(x1), x1, x2, lam, stats)
    assert (d1[0, 0, 2] == 0).all() and d2.isfinite().all()


@pytest.mark.parametrize("Tk", [64, 101, 17000])
def test_diff_in_place(lib, Tk):
    L = lib
    for dt in DT:
        shape = (2, 2, 6, Tk)
        x1, x2 = _maps(shape, DT[dt], "apart", 1, 2.0)
        lam = torch.tensor([0.3, 0.8], device=DEV)
        m = _mask("pad", 2, Tk, DT[dt], 3)
        want, stats = L.softmax_fw_diff(x1, x2, lam, m)
        got = x1.clone()
        L.softmax_fw_diff(got, x2, lam, m, out=got)
        assert torch.equal(got, want)
        g = _randn(shape, DT[dt], 4)
        d1, d2, dl = L.softmax_bw_diff(g, x1, x2, lam, stats, m)
        e1, e2, el = L.softmax_bw_diff(g, x1, x2, lam, stats, m, dscores1=x1, dscores2=x2)
        assert e1 is x1 and torch.equal(e1, d1) and torch.equal(e2, d2) and torch.equal(el, dl)


def test_diff_without_statistics(lib):
    """Through the C entry point: NULL statistics are not written."""
    L = lib
    for Tk in (64, 77, 20000):
        x1, x2 = (_randn((1, 2, 3, Tk), torch.bfloat16, s) for s in (1, 2))
        lam = torch.tensor([0.3, 0.8], device=DEV)
        want, _ = L.softmax_fw_diff(x1, x2, lam, causal=True)
        got = torch.empty_like(want)
        s = L.ls_softmax_fw_diff(got.data_ptr(), None, x1.data_ptr(), x2.data_ptr(), lam.data_ptr(),
                                 None, 1, 2, 3, Tk, 6 * Tk, 3 * Tk, 6 * Tk, 3 * Tk, 2, 1, 1.0, 2,
                                 torch.cuda.current_stream().cuda_stream)
        torch.cuda.synchronize()
        assert s == 0 and torch.equal(got, want)


def test_diff_one_map_for_both(lib):
    """The same scores twice, and strides of 0: one head's scores for every head."""
    L = lib
    x = _randn((2, 1, 5, 48), torch.float32, 1)
    lam = torch.tensor([1.0, 0.25, 0.0], device=DEV)
    e = x.expand(2, 3, 5, 48)
    got, _ = L.softmax_fw_diff(e, e, lam)
    p = torch.softmax(x.double(), -1)
    # round(e i) - e i, of which the second product is not rounded (fused): half a step of p,
    # which is itself off by a few steps
    assert (got[:, 0].abs().double() <= R.U * 1.001 * p[:, 0]).all()
    assert torch.allclose(got.double(), (1 - lam.double())[None, :, None, None] * p, atol=1e-6)


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("Tk", [1, 2, 3, 8, 64, 100, 257, 1001, 1024, 2049, 5000, 20000])
def test_diff_rows_with_one_visible_key(lib, dt, Tk):
    """All weight is on one key whatever its score: p (g - sum p g) is 0 but for the
    roundings of p = e i.  scale * x less the row's saved maximum is not 0 where their
    product is rounded, so that neither is p exactly 1; in steps of 2^-24: e in either
    direction 4 (2^-22 of ex2), the reciprocal 2, its correction, e g and (e g) i 1 each."""
    B, H, Tq = 2, 2, 3
    x1, x2 = _maps((B, H, Tq, Tk), DT[dt], "halves", Tk, 3.0)
    lam = torch.rand(H, generator=_gen(Tk + 2), device=DEV)
    dout = _randn((B, H, Tq, Tk), DT[dt], Tk + 3)
    m = torch.full((B, Tk), -INF, dtype=DT[dt], device=DEV)
    for b in range(B):
        m[b, (b * 7 + 3) % Tk] = 0
    _, stats = lib.softmax_fw_diff(x1, x2, lam, m, scale=0.3)
    d1, d2, _ = lib.softmax_bw_diff(dout, x1, x2, lam, stats, m, scale=0.3)

    def check(got, g, factor):  # 13 steps; the output's own rounding, of fp16 down to 2^-24
        lim = 14 * 2.0 ** -24 * factor * g.double().abs()
        assert (got.double().abs() <= lim + (2.0 ** -25 if dt == "f16" else 0)).all()

    lam_h = lam.double().abs()[None, :, None, None]
    hidden = (m == -INF)[:, None, None, :].expand_as(d1)
    assert not d1[hidden].any() and not d2[hidden].any()
    check(d1, dout, 0.3)
    check(d2, dout, 0.3 * lam_h)
    shape = (B, H, Tk if Tk < 300 else 1, Tk)  # causal: the first query sees one key
    y1, y2 = _maps(shape, DT[dt], "halves", Tk + 5, 3.0)
    g = _randn(shape, DT[dt], Tk + 8)
    if shape[2] == Tk:
        _, stats = lib.softmax_fw_diff(y1, y2, lam, causal=True)
        d1, d2, _ = lib.softmax_bw_diff(g, y1, y2, lam, stats, causal=True)
        assert not d1[:, :, 0, 1:].any() and not d2[:, :, 0, 1:].any()
        check(d1[:, :, :1], g[:, :, :1], 1.0)
        check(d2[:, :, :1], g[:, :, :1], lam_h)


def test_diff_empty(lib):
    L = lib
    lam = torch.ones(2, device=DEV)
    for shape in ((0, 2, 3, 4), (2, 2, 0, 4), (2, 2, 3, 0)):
        x = torch.zeros(shape, device=DEV)
        y, st = L.softmax_fw_diff(x, x.clone(), lam)
        assert y.shape == shape and st.shape == shape[:3] + (4,)
        _, _, dl = L.softmax_bw_diff(x.clone(), x, x.clone(), lam, st)
        assert dl.tolist() == [0.0, 0.0]


# ---------------------------------------------------------------------------
# norms around a block
# ---------------------------------------------------------------------------
def _block(rows, D, dtype, kind, post, pre, gates, seed):
    layer = kind == "layer"
    v = {"x": _randn((rows, D), dtype, seed, 1.5, 0.4), "r": _randn((rows, D), dtype, seed + 1, 2.0)}
    for k, on, s in (("pre", pre, 2), ("post", post, 4)):
        v["g_" + k] = _randn((D,), dtype, seed + s, 0.2, 1.0) if on else None
        v["b_" + k] = _randn((D,), dtype, seed + s + 1, 0.1) if on and layer else None
    v["gate"] = _randn((gates, D), dtype, seed + 6, 0.5, 0.5) if gates else None
    return v


NAMES = ("dx", "dr", "dg_pre", "db_pre", "dg_post", "db_post", "dgate")


def _check_block(L, rows, D, dt, kind="rms", post=True, pre=True, gates=0, a=1.0, with_dh=True,
                 seed=1, shift=0):
    dtype, layer = DT[dt], kind == "layer"
    v = _block(rows, D, dtype, kind, post, pre, gates, seed)
    if shift:
        v = {k: None if t is None else _shifted(t, shift) for k, t in v.items()}
    what = f"[{rows},{D}] {dt} {kind} post={post} pre={pre} gates={gates}"
    fw = R.block_fw(v["x"], v["r"], v["g_pre"], v["b_pre"], v["g_post"], v["b_post"], v["gate"], a,
                    layer, 1e-6)
    h, y, stats = L.block_norm_fw(v["x"], v["r"], v["g_pre"], v["b_pre"], v["g_post"], v["b_post"],
                                  v["gate"], a, kind)
    R.check(h, *fw[0], "h " + what)
    assert (y is None) == (not pre)
    if pre:
        R.check(y, *fw[1], "y " + what)
    R.check(stats, *fw[2], "stats " + what)
    h_in, st = fw[0][0].to(dtype), fw[2][0].float().contiguous()
    dy = _randn((rows, D), dtype, seed + 8) if pre else None
    dh = _randn((rows, D), dtype, seed + 9) if with_dh or not pre else None
    if shift:
        h_in = _shifted(h_in, shift)
    want = R.block_bw(dy, dh, v["x"], h_in, st, v["g_pre"], v["g_post"], v["b_post"], v["gate"], a,
                      layer)
    got = dict(zip(NAMES, L.block_norm_bw(dy, dh, v["x"], h_in, st, v["g_pre"], v["g_post"],
                                          v["b_post"], v["gate"], a, kind)))
    for k in NAMES:
        assert (got[k] is None) == (k not in want), k
        if k in want:
            R.check(got[k], *want[k], f"{k} {what}")


FORMS = [(True, True, 0), (True, True, 1), (True, True, "rows"), (False, True, 0), (False, True, 1),
         (True, False, 1), (False, False, "rows"), (True, False, 0)]


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("rows,D", [(1, 2), (3, 7), (5, 8), (16, 64), (33, 100), (700, 128),
                                    (17, 256), (64, 333), (2000, 512), (9, 768), (1300, 1024),
                                    (700, 1000), (40, 2048), (11, 4096)])
def test_block_sizes_and_forms(lib, dt, kind, rows, D):
    for i, (post, pre, g) in enumerate(FORMS):
        _check_block(lib, rows, D, dt, kind, post, pre, rows if g == "rows" else g,
                     a=1.5 if post else 1.0, with_dh=i % 2 == 0, seed=D + i)


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("rows,D", [(700, 4096), (5, 5000), (3, 8192), (700, 8192), (4, 10000),
                                    (3, 16384), (6, 16383)])
def test_block_wide_rows(lib, dt, kind, rows, D):
    _check_block(lib, rows, D, dt, kind, True, True, 1, seed=D)
    _check_block(lib, rows, D, dt, kind, True, True, rows, seed=D + 1)
    _check_block(lib, rows, D, dt, kind, False, True, 0, seed=D + 2)


@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("rows,gates", [(4095, 9), (3000, 1000), (2048, 128), (2400, 600),
                                        (5000, 2500), (1217, 1), (2432, 1216), (1220, 610)])
def test_block_gates(lib, kind, rows, gates):
    """Gates that span several runs of rows, one, and parts of one."""
    _check_block(lib, rows, 96, "bf16", kind, True, True, gates, seed=rows)
    _check_block(lib, rows, 96, "f32", kind, False, True, gates, seed=rows + 1)


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("shift", [1, 3])
def test_block_offsets(lib, dt, shift):
    _check_block(lib, 50, 128, dt, "layer", True, True, 5, shift=shift)
    _check_block(lib, 50, 128, dt, "rms", True, True, 1, shift=shift)


def test_block_large_means(lib):
    """A mean a thousand times the deviation costs the statistics no digits."""
    L = lib
    x = _randn((64, 512), torch.float32, 1, 1.0, 1000.0)
    r = torch.zeros_like(x)
    g = torch.ones(512, device=DEV)
    _, y, stats = L.block_norm_fw(x, r, g, kind="layer", eps=0.0)
    d = x.double()
    mean, var = d.mean(-1), d.var(-1, unbiased=False)
    assert ((stats[2] - mean).abs() / mean).max() < 1e-6
    # the mean's rounding moves the variance by its square, and each difference by half a
    # step of 1000 (3e-5)
    assert ((stats[3] - var ** -0.5).abs() * var.sqrt()).max() < 1e-4
    assert (y - (d - mean[:, None]) * (var ** -0.5)[:, None]).abs().max() < 5e-4


def test_block_in_place(lib):
    L = lib
    for dt in DT:
        for D in (128, 77, 12000):
            for kind in ("rms", "layer"):
                v = _block(30, D, DT[dt], kind, True, True, 3, 5)
                args = (v["g_pre"], v["b_pre"], v["g_post"], v["b_post"], v["gate"], 1.0, kind)
                h, y, st = L.block_norm_fw(v["x"], v["r"], *args)
                for a, b in (("r", "x"), ("x", "r")):
                    c = {k: v[k].clone() for k in "xr"}
                    h2, y2, st2 = L.block_norm_fw(c["x"], c["r"], *args, h=c[a], y=c[b])
                    assert h2 is c[a]
                    assert torch.equal(h2, h) and torch.equal(y2, y) and torch.equal(st2, st)
                dy, dh = _randn(h.shape, DT[dt], 7), _randn(h.shape, DT[dt], 8)
                bargs = (v["g_pre"], v["g_post"], v["b_post"], v["gate"], 1.0, kind)
                want = L.block_norm_bw(dy, dh, v["x"], h, st, *bargs)
                for i, j in ((0, 1), (2, 1), (3, 0), (1, 0), (0, 3)):  # dx, dr among dy, dh, x, h
                    c = [t.clone() for t in (dy, dh, v["x"], h)]
                    got = L.block_norm_bw(c[0], c[1], c[2], c[3], st, *bargs, dx=c[i], dr=c[j])
                    for p, q in zip(want, got):
                        assert (p is None and q is None) or torch.equal(p, q)


def test_block_without_rows(lib):
    L = lib
    x = torch.zeros(0, 24, device=DEV)
    g, gate = torch.ones(24, device=DEV), torch.ones(5, 24, device=DEV)
    h, y, st = L.block_norm_fw(x, x, g, g, g, g, gate, kind="layer")
    assert h.shape == y.shape == (0, 24) and st.shape == (4, 0)
    out = L.block_norm_bw(x, x, x, h, st, g, g, g, gate, kind="layer")
    assert all((t == 0).all() for t in out[2:]) and out[6].shape == (5, 24)
    out = L.block_norm_bw(x, x, x, h, st, g, g)
    assert all(t is None or (t == 0).all() for t in out[2:])


def test_block_nan_rows_stay_their_own(lib):
    L = lib
    for D in (256, 99):
        v = _block(40, D, torch.float32, "layer", True, True, 0, 3)
        h, y, st = L.block_norm_fw(v["x"], v["r"], v["g_pre"], v["b_pre"], v["g_post"], v["b_post"],
                                   kind="layer")
        x = v["x"].clone()
        x[7, 5] = math.nan
        h2, y2, _ = L.block_norm_fw(x, v["r"], v["g_pre"], v["b_pre"], v["g_post"], v["b_post"],
                                    kind="layer")
        keep = torch.arange(40, device=DEV) != 7
        assert torch.equal(h[keep], h2[keep]) and torch.equal(y[keep], y2[keep])
        assert h2[7].isnan().all() and y2[7].isnan().all()


# ---------------------------------------------------------------------------
# cross entropy from hidden states
# ---------------------------------------------------------------------------
def _loss(rows, D, V, dtype, ignored, seed):
    x = _randn((rows, D), dtype, seed)
    w = _randn((V, D), dtype, seed + 1, 2.5 / D ** 0.5)
    t = torch.randint(0, V, (rows,), generator=_gen(seed + 2), device=DEV)
    skip = torch.rand(rows, generator=_gen(seed + 3), device=DEV) < ignored
    if ignored == "prefix":
        skip = torch.arange(rows, device=DEV) < rows // 2
    return x, w, t.masked_fill(skip, -1 - seed % 3).to(torch.int32)


def _check_loss(L, rows, D, V, dt, ignored=0.0, seed=1, shift=0, up=None):
    dtype = DT[dt]
    x, w, t = _loss(rows, D, V, dtype, 0.0 if ignored == "prefix" else ignored, seed)
    if ignored == "prefix":
        t = t.masked_fill(torch.arange(rows, device=DEV) < rows // 2, -1)
    if shift:
        x = _shifted(x, shift)
    what = f"[{rows},{D}]x{V} {dt} ignored={ignored}"
    fw = R.loss_fw(x, w, t)
    loss, lse = L.linear_cross_entropy_fw(x, w, t)
    R.check(loss, *fw[0], "loss " + what)
    R.check(lse, *fw[1], "lse " + what)
    given = fw[1][0].float()
    if up is None:
        up = torch.rand(rows, generator=_gen(seed + 4), device=DEV) / rows
    outs = {}
    if shift:
        outs = {"dhidden": _shifted(torch.zeros_like(x), shift),
                "dweight": _shifted(torch.zeros_like(w), shift)}
    a, b = R.loss_bw(x, w, t, given, up)
    dx, dw = L.linear_cross_entropy_bw(x, w, t, given, up, **outs)
    R.check(dx, *a, "dx " + what)
    R.check(dw, *b, "dw " + what)
    only, none = L.linear_cross_entropy_bw(x, w, t, given, up, weight_grad=False)
    assert none is None
    R.check(only, *a, "dx alone " + what)


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("rows,D,V", [(1, 1, 1), (1, 8, 5), (3, 7, 65), (127, 64, 255),
                                      (128, 64, 256), (129, 72, 257), (255, 128, 511),
                                      (256, 120, 512), (257, 100, 777), (300, 1024, 1000),
                                      (33, 768, 3200), (513, 333, 1025), (700, 257, 130),
                                      (2049, 40, 300)])
def test_linear_ce_sizes(lib, dt, rows, D, V):
    _check_loss(lib, rows, D, V, dt, seed=rows)
    _check_loss(lib, rows, D, V, dt, ignored=0.4, seed=rows + 1)


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("ignored", [0.97, 1.0, "prefix"])
def test_linear_ce_ignored_rows(lib, dt, ignored):
    _check_loss(lib, 600, 96, 500, dt, ignored=ignored, seed=5)
    _check_loss(lib, 5000, 24, 70, dt, ignored=ignored, seed=6)  # counted in a launch of its own


@pytest.mark.parametrize("dt", list(DT))
def test_linear_ce_offsets(lib, dt):
    _check_loss(lib, 70, 64, 200, dt, shift=1)
    _check_loss(lib, 70, 61, 200, dt, shift=3)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_linear_ce_in_pieces_of_the_vocabulary(lib, dt):
    """Enough rows that the vocabulary is cut into pieces, against chunks of rows."""
    L = lib
    rows, D, V = (70000, 24, 9001) if dt == "bf16" else (23000, 16, 8300)
    x, w, t = _loss(rows, D, V, DT[dt], 0.2, 3)
    loss, lse = L.linear_cross_entropy_fw(x, w, t)
    up = (t >= 0).float() / rows
    parts = list(torch.arange(rows, device=DEV).split(10000))
    given = torch.empty(rows, device=DEV)
    dw = dw_tol = 0
    for p in parts:
        (v, tol), (s, stol) = R.loss_fw(x[p], w, t[p])
        R.check(loss[p], v, tol, "loss")
        R.check(lse[p], s, stol, "lse")
        given[p] = s.float()
    dx, got = L.linear_cross_entropy_bw(x, w, t, given, up)
    for p in parts:
        a, b = R.loss_bw(x[p], w, t[p], given[p], up[p])
        R.check(dx[p], *a, "dx")
        # one sum over all rows: the chunks' bounds add up, its chain is longer
        dw, dw_tol = dw + b[0], dw_tol + b[1]
    mag = sum(R.loss_bw(x[p].abs(), w, t[p], given[p], up[p])[1][0].abs() for p in parts[:1])
    assert mag.isfinite().all()
    R.check(got, dw, dw_tol * (rows / 10000), "dw")


@pytest.mark.parametrize("dt", list(DT))
def test_linear_ce_what_ignored_rows_hold_does_not_matter(lib, dt):
    L = lib
    for D in (64, 37):
        x, w, t = _loss(300, D, 400, DT[dt], 0.5, 9)
        up = torch.rand(300, device=DEV)
        loss, lse = L.linear_cross_entropy_fw(x, w, t)
        want = L.linear_cross_entropy_bw(x, w, t, lse, up)
        dead = t < 0
        assert (loss[dead] == 0).all() and (lse[dead] == 0).all() and (want[0][dead] == 0).all()
        for bad in (math.nan, INF, -INF):
            y = x.clone().masked_fill_(dead[:, None], bad)
            got = L.linear_cross_entropy_fw(y, w, t)
            assert torch.equal(got[0], loss) and torch.equal(got[1], lse)
            dx, dw = L.linear_cross_entropy_bw(y, w, t, lse.masked_fill(dead, bad),
                                               up.masked_fill(dead, bad))
            assert torch.equal(dx, want[0]) and torch.equal(dw, want[1])


@pytest.mark.parametrize("dt", list(DT))
def test_linear_ce_classes_beyond_the_vocabulary(lib, dt):
    L = lib
    x, w, t = _loss(200, 48, 100, DT[dt], 0.3, 4)
    up = torch.rand(200, device=DEV)
    clean, lse0 = L.linear_cross_entropy_fw(x, w, t)
    dx0, _ = L.linear_cross_entropy_bw(x, w, t, lse0, up)
    t2 = t.clone()
    t2[17], t2[150] = 100, 2 ** 31 - 1
    loss, lse = L.linear_cross_entropy_fw(x, w, t2)
    keep = torch.ones(200, dtype=torch.bool, device=DEV)
    keep[17] = keep[150] = False
    assert loss[~keep].isnan().all() and lse[~keep].isnan().all()
    assert torch.equal(loss[keep], clean[keep]) and torch.equal(lse[keep], lse0[keep])
    dx, dw = L.linear_cross_entropy_bw(x, w, t2, lse, up)
    assert dx[~keep].isnan().all() and dx[keep].isfinite().all() and dw.isnan().all()


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("kind", ["zeros", "equal", "signs", "tiny", "spread"])
def test_linear_ce_upstream_gradients(lib, dt, kind):
    g = torch.rand(300, generator=_gen(8), device=DEV)
    up = {"zeros": torch.zeros(300, device=DEV), "equal": torch.full((300,), 1 / 7373, device=DEV),
          "signs": g - 0.5, "tiny": g * 1e-30, "spread": torch.exp2(-24 * g)}[kind]
    if dt == "f16" and kind == "tiny":
        up = g * 1e-6  # (below that fp16 cannot hold the gradients)
    _check_loss(lib, 300, 72, 333, dt, ignored=0.1, up=up)


def test_linear_ce_gradient_that_is_not_finite(lib):
    L = lib
    x, w, t = _loss(60, 32, 50, torch.bfloat16, 0.0, 2)
    _, lse = L.linear_cross_entropy_fw(x, w, t)
    up = torch.full((60,), 0.01, device=DEV)
    want, _ = L.linear_cross_entropy_bw(x, w, t, lse, up)
    up[5] = math.nan
    dx, dw = L.linear_cross_entropy_bw(x, w, t, lse, up)
    keep = torch.arange(60, device=DEV) != 5
    assert dx[5].isnan().all() and dw.isnan().all()
    # (without a common scale the gradients are rounded elsewhere)
    assert torch.allclose(dx[keep].float(), want[keep].float(), rtol=0.02, atol=1e-4)


def test_linear_ce_far_logits(lib):
    """Logits of hundreds: the largest one decides, and nothing overflows."""
    L = lib
    x, w, t = _loss(130, 64, 300, torch.float32, 0.0, 6)
    x = x * 300
    (loss, ltol), (lse, stol) = R.loss_fw(x, w, t)
    got, s = L.linear_cross_entropy_fw(x, w, t)
    R.check(got, loss, ltol, "loss")
    R.check(s, lse, stol, "lse")


def test_linear_ce_without_rows(lib):
    L = lib
    x, w = torch.zeros(0, 16, device=DEV), torch.ones(9, 16, device=DEV)
    t = torch.zeros(0, dtype=torch.int32, device=DEV)
    loss, lse = L.linear_cross_entropy_fw(x, w, t)
    dx, dw = L.linear_cross_entropy_bw(x, w, t, lse, loss)
    assert loss.shape == (0,) and dx.shape == (0, 16) and (dw == 0).all()


def test_linear_ce_agrees_with_the_cross_entropy_of_its_logits(lib):
    L = lib
    x, w, t = _loss(500, 128, 1000, torch.float32, 0.2, 7)
    z = (x.double() @ w.double().T).float()
    loss, lse = L.cross_entropy_fw(z, t)
    got, s = L.linear_cross_entropy_fw(x, w, t)
    assert torch.allclose(got, loss, atol=2e-5) and torch.allclose(s, lse, atol=2e-5)


# ---------------------------------------------------------------------------
# together: a differential decoder layer and its loss
# ---------------------------------------------------------------------------
def _layer_parameters(dtype, D, H, V, seed):
    hd = D // H  # a head's values; a map's queries and keys have half
    p = {"qk": _randn((D, 2 * D), dtype, seed, D ** -0.5), "v": _randn((D, D), dtype, seed + 1, D ** -0.5),
         "o": _randn((D, D), dtype, seed + 2, D ** -0.5), "emb": _randn((V, D), dtype, seed + 3, D ** -0.5),
         "lam": torch.rand(H, generator=_gen(seed + 4), device=DEV) * 0.5 + 0.2,
         "gate": _randn((1, D), dtype, seed + 5, 0.2, 0.8)}
    for k in ("g_post", "g_pre"):
        p[k] = _randn((D,), dtype, seed + 6, 0.1, 1.0)
    return p, hd


def _heads(t, B, T, n):
    return t.view(B, T, n, -1).transpose(1, 2)


def _layer_step(L, p, x, target, mask, B, T, H):
    """Loss, and gradients of every parameter and of x, by the framework's operators and
    torch's matrix products."""
    D = x.shape[1]
    hd = D // H
    scale = (hd // 2) ** -0.5
    qk, v = x @ p["qk"], x @ p["v"]
    q, k = _heads(qk[:, :D].contiguous(), B, T, 2 * H), _heads(qk[:, D:].contiguous(), B, T, 2 * H)
    s = (q @ k.transpose(2, 3)).contiguous()
    y, st = L.softmax_fw_diff(s[:, :H], s[:, H:], p["lam"], mask, causal=True, scale=scale)
    vh = _heads(v, B, T, H)
    att = (y @ vh).transpose(1, 2).reshape(B * T, D)
    out = att @ p["o"]
    h, n, bst = L.block_norm_fw(out, x, gamma_pre=p["g_pre"], gamma_post=p["g_post"], gate=p["gate"])
    loss, lse = L.linear_cross_entropy_fw(n, p["emb"], target)
    count = (target >= 0).sum().clamp(min=1)
    up = (target >= 0).float() / count
    g = {}
    dn, g["emb"] = L.linear_cross_entropy_bw(n, p["emb"], target, lse, up)
    dout, dx, g["g_pre"], _, g["g_post"], _, g["gate"] = L.block_norm_bw(
        dn, None, out, h, bst, gamma_pre=p["g_pre"], gamma_post=p["g_post"], gate=p["gate"])
    g["o"] = att.T @ dout
    datt = _heads(dout @ p["o"].T, B, T, H)
    dy = (datt @ vh.transpose(2, 3)).contiguous()
    dv = (y.transpose(2, 3) @ datt).transpose(1, 2).reshape(B * T, D)
    ds = torch.empty_like(s)
    _, _, g["lam"] = L.softmax_bw_diff(dy, s[:, :H], s[:, H:], p["lam"], st, mask, causal=True,
                                       scale=scale, dscores1=ds[:, :H], dscores2=ds[:, H:])
    dq = (ds @ k).transpose(1, 2).reshape(B * T, D)
    dk = (ds.transpose(2, 3) @ q).transpose(1, 2).reshape(B * T, D)
    dqk = torch.cat((dq, dk), 1)
    g["qk"], g["v"] = x.T @ dqk, x.T @ dv
    g["x"] = dx + dqk @ p["qk"].T + dv @ p["v"].T
    clipped, norm = L.grad_clip([g[k].contiguous() for k in sorted(g)], 0.1,
                                out=[torch.empty_like(g[k], memory_format=torch.contiguous_format)
                                     for k in sorted(g)])
    return [loss, *(g[k] for k in sorted(g)), *clipped, norm], sorted(g)


def _layer_inputs(dtype, B, T, D, H, V, seed=1):
    p, _ = _layer_parameters(dtype, D, H, V, seed)
    x = _randn((B * T, D), dtype, seed + 20)
    t = torch.randint(0, V, (B * T,), generator=_gen(seed + 21), device=DEV).to(torch.int32)
    n = torch.randint(T // 2, T + 1, (B,), generator=torch.Generator().manual_seed(seed))
    mask = torch.zeros(B, T)
    for b in range(B):
        mask[b, int(n[b]):] = -INF
    pad = (mask.view(-1) == -INF).to(DEV)
    return p, x, t.masked_fill(pad, -1), mask.to(dtype).to(DEV)


@pytest.mark.parametrize("T", [24, 37])
def test_decoder_layer_gradients(lib, T):
    """All operators of a differential layer and its loss, forward and backward, in fp32
    against automatic differentiation in 64 bits."""
    L = lib
    B, D, H, V = 2, 64, 4, 301
    p, x, t, mask = _layer_inputs(torch.float32, B, T, D, H, V)
    got, names = _layer_step(L, p, x, t, mask, B, T, H)
    q64 = {k: v.double().requires_grad_() for k, v in {**p, "x": x}.items()}
    X = q64["x"]
    qk = X @ q64["qk"]
    q, k = _heads(qk[:, :D], B, T, 2 * H), _heads(qk[:, D:], B, T, 2 * H)
    z = q @ k.transpose(2, 3) * (D // H // 2) ** -0.5 + mask.double()[:, None, None, :]
    z = z.masked_fill(~torch.ones(T, T, dtype=torch.bool, device=DEV).tril(), -INF)
    a = torch.softmax(z, -1)
    y = a[:, :H] - q64["lam"][None, :, None, None] * a[:, H:]
    out = (y @ _heads(X @ q64["v"], B, T, H)).transpose(1, 2).reshape(B * T, D) @ q64["o"]
    rms = lambda v, g: v * (v.square().mean(-1, keepdim=True) + 1e-6) ** -0.5 * g  # noqa: E731
    h = X + q64["gate"] * rms(out, q64["g_post"])
    logits = rms(h, q64["g_pre"]) @ q64["emb"].T
    live = t >= 0
    each = torch.nn.functional.cross_entropy(logits[live], t[live].long(), reduction="none")
    each.mean().backward()
    # a dozen operators in a row, each off by some tens of steps of fp32 (sums of up to 64
    # terms and exponentials), of values whose parts nearly cancel by at most a factor of
    # ten: 12 * 100 * 2^-24 = 7e-5, a third more for torch's own products
    tol = 1e-4
    assert torch.allclose(got[0][live].double(), each.detach(), rtol=tol, atol=tol)
    grads = [q64[k].grad for k in names]
    for name, w, a in zip(names, grads, got[1:]):
        far = float((a.double() - w).abs().max() / w.abs().max())
        assert far < tol, (name, far)
    norm = math.sqrt(sum(float(w.square().sum()) for w in grads))
    assert abs(float(got[-1]) - norm) < tol * norm


def _equal(a, b):
    return all(torch.equal(p, q) for p, q in zip(a, b))


@pytest.mark.parametrize("dt", list(DT))
def test_operators_are_reproducible_on_any_stream(lib, dt):
    L = lib
    B, T, D, H, V = 3, 40, 128, 4, 700
    p, x, t, mask = _layer_inputs(DT[dt], B, T, D, H, V)
    torch.cuda.synchronize()

    def ops():
        s = _randn((B, 2 * H, T, T), DT[dt], 5)
        y, st = L.softmax_fw_diff(s[:, 0::2], s[:, 1::2], p["lam"], mask, causal=True)
        d = L.softmax_bw_diff(y, s[:, 0::2], s[:, 1::2], p["lam"], st, mask, causal=True)
        h, n, bst = L.block_norm_fw(x, x, p["g_pre"], gamma_post=p["g_post"], gate=p["gate"])
        g = L.block_norm_bw(n, h, x, h, bst, p["g_pre"], p["g_post"], gate=p["gate"])
        loss, lse = L.linear_cross_entropy_fw(n, p["emb"], t)
        e = L.linear_cross_entropy_bw(n, p["emb"], t, lse, (t >= 0).float())
        return [v for v in (y, st, *d, h, n, *g, loss, lse, *e) if v is not None]

    want = ops()
    again = ops()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = ops()
    torch.cuda.synchronize()
    assert _equal(want, again) and _equal(want, other)


def test_operators_in_a_graph(lib):
    """A captured step, replayed on new inputs, gives what the calls give."""
    L = lib
    B, T, D, H, V = 2, 33, 64, 2, 130
    dtype = torch.bfloat16
    p, x, t, mask = _layer_inputs(dtype, B, T, D, H, V)
    s = _randn((B, 2 * H, T, T), dtype, 5)
    ws = L.linear_cross_entropy_workspace(B * T, D, V, dtype, DEV, backward=True)
    ws_fw = L.linear_cross_entropy_workspace(B * T, D, V, dtype, DEV)
    ws_diff = L.softmax_diff_workspace(B, H, T, DEV)
    ws_block = L.block_norm_workspace(B * T, D, 1, "rms", dtype, DEV)

    def ops():
        y, st = L.softmax_fw_diff(s[:, :H], s[:, H:], p["lam"], mask, causal=True)
        d = L.softmax_bw_diff(y, s[:, :H], s[:, H:], p["lam"], st, mask, causal=True,
                              workspace=ws_diff)
        h, n, bst = L.block_norm_fw(x, x, p["g_pre"], gamma_post=p["g_post"], gate=p["gate"])
        g = L.block_norm_bw(n, h, x, h, bst, p["g_pre"], p["g_post"], gate=p["gate"],
                            workspace=ws_block)
        loss, lse = L.linear_cross_entropy_fw(n, p["emb"], t, workspace=ws_fw)
        e = L.linear_cross_entropy_bw(n, p["emb"], t, lse, (t >= 0).float(), workspace=ws)
        return [v for v in (y, st, *d, h, n, *g, loss, lse, *e) if v is not None]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        ops()
        graph = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph, stream=side):
            held = ops()
    for seed in (50, 60):
        _, x2, t2, _ = _layer_inputs(dtype, B, T, D, H, V, seed)
        x.copy_(x2)
        t.copy_(t2)
        s.copy_(_randn(s.shape, dtype, seed))
        graph.replay()
        torch.cuda.synchronize()
        got = [v.clone() for v in held]
        assert _equal(got, ops())


def test_two_calls_at_once_with_their_own_workspaces(lib):
    L = lib
    states = [_layer_inputs(torch.bfloat16, 2, 60 + 9 * i, 128, 4, 900, seed=30 * i + 1)
              for i in range(2)]

    def step(v):
        p, x, t, _ = v
        loss, lse = L.linear_cross_entropy_fw(x, p["emb"], t)
        return [loss, lse, *L.linear_cross_entropy_bw(x, p["emb"], t, lse, (t >= 0).float())]

    want = [step(v) for v in states]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in states]
    got = [None, None]
    for _ in range(4):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                got[i] = step(states[i])
    torch.cuda.synchronize()
    for w, g in zip(want, got):
        assert _equal(w, g)
