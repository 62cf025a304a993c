"""Host-side refusals of the difference of two softmax maps, the norms around a
block and the cross entropy from hidden states: through the C ABI and through
the PyTorch layer.  No kernel is launched here."""
import math

import pytest
import torch

import transformer_reduce_gb300 as L

FAKE = 0x10000  # never dereferenced: every call below returns on the host
STEP = 1 << 24  # far enough apart for every tensor below


@pytest.fixture(scope="module")
def abi():
    from transformer_reduce_gb300 import build as b
    b.build()
    from transformer_reduce_gb300 import _lib
    _lib.load()
    return _lib


def _at(i):
    return FAKE + i * STEP


# -- difference of two softmax maps ------------------------------------------------
def _diff_fw(abi, out=_at(1), stats=_at(2), x1=_at(3), x2=_at(4), lam=_at(5), mask=None, B=2, H=3,
             Tq=4, Tk=8, s1=(96, 32), s2=(96, 32), n=3, causal=0, scale=1.0, dt=None):
    return abi.ls_softmax_fw_diff(out, stats, x1, x2, lam, mask, B, H, Tq, Tk, *s1, *s2, n, causal,
                                  scale, abi.LS_F32 if dt is None else dt)


def _diff_bw(abi, dx1=_at(1), dx2=_at(2), dlam=_at(3), dout=_at(4), x1=_at(5), x2=_at(6),
             lam=_at(7), stats=_at(8), mask=None, B=2, H=3, Tq=4, Tk=8, d1=(96, 32), d2=(96, 32),
             s1=(96, 32), s2=(96, 32), n=3, causal=0, scale=1.0, ws=_at(9), wsb=1 << 40, dt=None):
    return abi.ls_softmax_bw_diff(dx1, dx2, dlam, dout, x1, x2, lam, stats, mask, B, H, Tq, Tk, *d1,
                                  *d2, *s1, *s2, n, causal, scale, ws, wsb,
                                  abi.LS_F32 if dt is None else dt)


def test_diff_rejections(abi):
    bad, un, mis = abi.LS_ERR_INVALID_ARG, abi.LS_ERR_UNSUPPORTED, abi.LS_ERR_MISALIGNED
    for call in (_diff_fw, _diff_bw):
        assert call(abi, dt=7) == un
        for k in ("B", "H", "Tq", "Tk"):
            assert call(abi, **{k: -1}) == bad
        assert call(abi, Tk=(1 << 30) + 1) == un and call(abi, Tq=(1 << 30) + 1) == un
        assert call(abi, B=1 << 29, H=3, Tq=1 << 29) == un
        assert call(abi, Tq=9, causal=1) == bad
        for scale in (0.0, -1.0, math.inf, math.nan):
            assert call(abi, scale=scale) == bad
        assert call(abi, n=2) == bad and call(abi, n=0) == bad
        assert call(abi, s1=(-1, 32)) == bad and call(abi, s2=(96, -32)) == bad
        assert call(abi, s1=(1 << 60, 32)) == un
        assert call(abi, lam=None) == bad and call(abi, lam=FAKE + 2) == mis
        assert call(abi, x1=None) == bad and call(abi, x2=FAKE + 1) == mis
        assert call(abi, mask=FAKE + 2) == mis and call(abi, stats=FAKE + 8) == mis
    assert _diff_fw(abi, out=None) == bad and _diff_fw(abi, out=FAKE + 2) == mis
    for k in ("dx1", "dx2", "dlam", "dout", "stats"):
        assert _diff_bw(abi, **{k: None}) == bad
    for k in ("dx1", "dx2", "dlam", "dout"):
        assert _diff_bw(abi, **{k: FAKE + 2}) == mis
    need = abi.ls_softmax_bw_diff_workspace_size(2, 3, 4)
    assert need == 2 * 3 * 4 * 4
    assert _diff_bw(abi, ws=None) == abi.LS_ERR_WORKSPACE
    assert _diff_bw(abi, ws=_at(9) + 8) == abi.LS_ERR_WORKSPACE
    assert _diff_bw(abi, wsb=need - 1) == abi.LS_ERR_WORKSPACE
    assert abi.ls_softmax_bw_diff_workspace_size(-1, 3, 4) == 0
    assert abi.ls_softmax_bw_diff_workspace_size(2, 0, 4) == 0
    # nothing to do
    for k in ("B", "Tq", "Tk"):
        assert _diff_fw(abi, out=None, x1=None, x2=None, lam=None, **{k: 0}) == abi.LS_OK
    assert _diff_fw(abi, out=None, x1=None, x2=None, lam=None, H=0, n=1) == abi.LS_OK
    assert _diff_bw(abi, H=0, n=0, dlam=None) == abi.LS_OK


def test_diff_overlaps(abi):
    bad = abi.LS_ERR_INVALID_ARG
    row = 4 * 32  # bytes of a head
    # outputs that meet an input or each other
    assert _diff_fw(abi, out=_at(4)) == bad                      # x2 in place
    assert _diff_fw(abi, out=_at(3) + 16) == bad                 # x1, shifted
    assert _diff_fw(abi, out=_at(3), s1=(192, 64)) == bad        # x1 in place, other strides
    assert _diff_fw(abi, out=_at(2)) == bad and _diff_fw(abi, stats=_at(3)) == bad
    assert _diff_fw(abi, out=_at(5)) == bad
    for k in ("dx1", "dx2"):
        for other in (4, 8, 9, 3, 7):
            assert _diff_bw(abi, **{k: _at(other)}) == bad, (k, other)
    assert _diff_bw(abi, dx1=_at(6)) == bad and _diff_bw(abi, dx2=_at(5)) == bad
    assert _diff_bw(abi, dx1=_at(2)) == bad                      # both the same
    assert _diff_bw(abi, dx1=_at(5) + 16) == bad
    # interleaved heads: apart by a head, or not quite
    inter = dict(d1=(192, 64), d2=(192, 64))
    assert _diff_bw(abi, dx2=_at(1) + row - 4, **inter) == bad
    assert _diff_bw(abi, dx2=_at(1) + 2 * row, **inter) == bad
    assert _diff_bw(abi, dx2=_at(1) + 3 * row + 4, **inter) == bad
    # a gradient that overlaps itself
    assert _diff_bw(abi, d1=(96, 31)) == bad and _diff_bw(abi, d1=(95, 32)) == bad
    assert _diff_bw(abi, d2=(0, 32)) == bad and _diff_bw(abi, d2=(32, 32)) == bad


def _raises(match, fn, *a, **k):
    with pytest.raises(ValueError, match=match):
        fn(*a, **k)


def test_diff_arguments_are_checked():
    bf16, f32 = torch.bfloat16, torch.float32
    s = torch.zeros(2, 6, 4, 8, dtype=bf16)
    a, b = s[:, :3], s[:, 3:]
    lam = torch.zeros(3)
    _raises("scores1 must be", L.softmax_fw_diff, s[0], s[0], lam)
    _raises("scores2 must be", L.softmax_fw_diff, a, s, lam)
    _raises("scores2 must be", L.softmax_fw_diff, a, b.float(), lam)
    _raises("dense rows", L.softmax_fw_diff, a.transpose(2, 3), b.transpose(2, 3), lam)
    _raises("lam must be", L.softmax_fw_diff, a, b, lam[:2])
    _raises("lam must be", L.softmax_fw_diff, a, b, lam.to(bf16))
    _raises("lam must be", L.softmax_fw_diff, a, b, torch.zeros(1, dtype=bf16))
    _raises("mask must be", L.softmax_fw_diff, a, b, lam, torch.zeros(2, 7, dtype=bf16))
    _raises("out must be", L.softmax_fw_diff, a, b, lam, out=torch.zeros(2, 3, 4, 7, dtype=bf16))
    _raises("stats must be", L.softmax_fw_diff, a, b, lam, stats=torch.zeros(2, 3, 4, 2))
    _raises("CUDA device", L.softmax_fw_diff, a, b, lam)
    g, st = torch.zeros(2, 3, 4, 8, dtype=bf16), torch.zeros(2, 3, 4, 4)
    _raises("dout must be", L.softmax_bw_diff, g[:1], a, b, lam, st)
    _raises("stats must be", L.softmax_bw_diff, g, a, b, lam, st.to(bf16))
    _raises("dscores1 must be", L.softmax_bw_diff, g, a, b, lam, st, dscores1=s)
    _raises("dlam must be", L.softmax_bw_diff, g, a, b, lam, st, dlam=torch.zeros(1))
    _raises("workspace must be", L.softmax_bw_diff, g, a, b, lam, st,
            workspace=torch.zeros(64, dtype=bf16))
    _raises("CUDA device", L.softmax_bw_diff, g, a, b, lam, st)
    assert f32  # (lam and stats are fp32 whatever the scores)


# -- norms around a block ------------------------------------------------------------
def _bn_fw(abi, h=_at(1), y=_at(2), stats=_at(3), x=_at(4), r=_at(5), gate=None, g_post=_at(6),
           b_post=None, g_pre=_at(7), b_pre=None, rows=6, hidden=8, gates=0, a=1.0, eps=1e-6,
           layer=1, dt=None):
    return abi.ls_block_norm_fw(h, y, stats, x, r, gate, g_post, b_post, g_pre, b_pre, rows, hidden,
                                gates, a, eps, layer, abi.LS_F32 if dt is None else dt)


def _bn_bw(abi, dx=_at(1), dr=_at(2), dgate=None, dg_post=_at(3), db_post=None, dg_pre=_at(4),
           db_pre=None, dy=_at(5), dh=_at(6), x=_at(7), h=_at(8), stats=_at(9), gate=None,
           g_post=_at(10), b_post=None, g_pre=_at(11), rows=6, hidden=8, gates=0, a=1.0, layer=1,
           ws=_at(12), wsb=1 << 40, dt=None):
    return abi.ls_block_norm_bw(dx, dr, dgate, dg_post, db_post, dg_pre, db_pre, dy, dh, x, h, stats,
                                gate, g_post, b_post, g_pre, rows, hidden, gates, a, layer, ws, wsb,
                                abi.LS_F32 if dt is None else dt)


def test_block_norm_rejections(abi):
    bad, un, mis = abi.LS_ERR_INVALID_ARG, abi.LS_ERR_UNSUPPORTED, abi.LS_ERR_MISALIGNED
    gate = _at(20)
    for call in (_bn_fw, _bn_bw):
        assert call(abi, dt=9) == un
        assert call(abi, rows=-1) == bad and call(abi, hidden=0) == bad
        assert call(abi, hidden=16385) == un and call(abi, rows=(1 << 40) + 1) == un
        for a in (math.inf, math.nan):
            assert call(abi, a=a) == bad
        for gates in (0, -1, 4, 7):
            assert call(abi, gate=gate, gates=gates) == bad
        assert call(abi, x=FAKE + 2) == mis and call(abi, stats=FAKE + 2) == mis
        assert call(abi, b_post=_at(21), layer=0) == bad
        assert call(abi, b_post=_at(21), g_post=None) == bad
        for k in ("x", "stats"):
            assert call(abi, **{k: None}) == bad
    for eps in (-1.0, math.inf, math.nan):
        assert _bn_fw(abi, eps=eps) == bad
    assert _bn_fw(abi, b_pre=_at(21), layer=0) == bad and _bn_fw(abi, b_pre=_at(21), g_pre=None) == bad
    for k in ("h", "y", "r"):
        assert _bn_fw(abi, **{k: None}) == bad
    assert _bn_fw(abi, rows=0, h=None, y=None, stats=None, x=None, r=None) == abi.LS_OK
    for k in ("dx", "dr", "dy", "h", "dg_post", "dg_pre"):
        assert _bn_bw(abi, **{k: None}) == bad
    assert _bn_bw(abi, g_pre=None, dg_pre=None, dy=None, h=None, dh=None) == bad
    assert _bn_bw(abi, gate=gate, gates=2) == bad                 # no dgate
    assert _bn_bw(abi, db_post=_at(22), layer=0) == bad and _bn_bw(abi, db_pre=_at(22), layer=0) == bad
    assert _bn_bw(abi, dg_pre=FAKE + 2) == mis
    need = abi.ls_block_norm_bw_workspace_size(6, 8, 0, 1, abi.LS_F32)
    assert need > 0 and need % 32 == 0
    assert _bn_bw(abi, ws=None) == abi.LS_ERR_WORKSPACE
    assert _bn_bw(abi, ws=_at(12) + 4) == abi.LS_ERR_WORKSPACE
    assert _bn_bw(abi, wsb=need - 1) == abi.LS_ERR_WORKSPACE
    for bad_size in ((0, 8, 0), (6, 0, 0), (6, 8, 4), (6, 16385, 0), (6, 8, -1)):
        assert abi.ls_block_norm_bw_workspace_size(*bad_size, 1, abi.LS_F32) == 0
    assert abi.ls_block_norm_bw_workspace_size(6, 8, 0, 1, 9) == 0


def test_block_norm_overlaps(abi):
    bad = abi.LS_ERR_INVALID_ARG
    assert _bn_fw(abi, h=_at(2)) == bad and _bn_fw(abi, h=_at(4) + 32) == bad
    assert _bn_fw(abi, y=_at(5) + 4) == bad and _bn_fw(abi, stats=_at(4)) == bad
    assert _bn_fw(abi, h=_at(6)) == bad and _bn_fw(abi, y=_at(7)) == bad
    assert _bn_bw(abi, dx=_at(2)) == bad and _bn_bw(abi, dr=_at(7)) == bad
    assert _bn_bw(abi, dx=_at(5) + 4) == bad and _bn_bw(abi, dr=_at(6) + 32) == bad
    for k in ("dg_post", "dg_pre"):
        for other in (1, 2, 5, 6, 7, 8, 9, 10, 11, 12):
            assert _bn_bw(abi, **{k: _at(other)}) == bad, (k, other)
    assert _bn_bw(abi, dg_post=_at(4)) == bad


def test_block_norm_arguments_are_checked():
    x = torch.zeros(6, 8, dtype=torch.float16)
    g = torch.ones(8, dtype=torch.float16)
    _raises("kind must be", L.block_norm_fw, x, x, g, kind="batch")
    _raises("residual must be", L.block_norm_fw, x, x[:5], g)
    _raises("gamma_pre must be", L.block_norm_fw, x, x, g[:7])
    _raises("gamma_post must be", L.block_norm_fw, x, x, g, gamma_post=g.float())
    _raises("beta_pre wants", L.block_norm_fw, x, x, g, beta_pre=g)
    _raises("beta_post wants", L.block_norm_fw, x, x, g, beta_post=g, kind="layer")
    _raises("gate must be", L.block_norm_fw, x, x, g, gate=g)
    _raises("gate must be", L.block_norm_fw, x, x, g, gate=x[:4])
    _raises("gate must be", L.block_norm_fw, x, x, g, gate=x[:2, :4])
    _raises("y is not computed", L.block_norm_fw, x, x, y=x)
    _raises("h must be", L.block_norm_fw, x, x, g, h=x[:3])
    _raises("stats must be", L.block_norm_fw, x, x, g, stats=torch.zeros(6, 4))
    _raises(r"\[rows, hidden\]", L.block_norm_fw, x.view(2, 3, 8), x, g)
    _raises("CUDA device", L.block_norm_fw, x, x, g)
    st = torch.zeros(4, 6)
    _raises("no y, and no dy", L.block_norm_bw, x, x, x, x, st)
    _raises("dh is needed", L.block_norm_bw, None, None, x, x, st)
    _raises("dy and h are needed", L.block_norm_bw, None, x, x, x, st, gamma_pre=g)
    _raises("dy and h are needed", L.block_norm_bw, x, x, x, None, st, gamma_pre=g)
    _raises("dh must be", L.block_norm_bw, x, x[:2], x, x, st, gamma_pre=g)
    _raises("stats must be", L.block_norm_bw, x, x, x, x, st[:3], gamma_pre=g)
    _raises("workspace must be", L.block_norm_bw, x, x, x, x, st, gamma_pre=g,
            workspace=torch.zeros(8, dtype=torch.int32))
    _raises("CUDA device", L.block_norm_bw, x, x, x, x, st, gamma_pre=g)


# -- cross entropy from hidden states ------------------------------------------------
def _ce_fw(abi, loss=_at(1), lse=_at(2), x=_at(3), w=_at(4), target=_at(5), rows=4, hidden=16,
           vocab=9, ws=_at(6), wsb=1 << 40, dt=None):
    return abi.ls_linear_cross_entropy_fw(loss, lse, x, w, target, rows, hidden, vocab, ws, wsb,
                                          abi.LS_BF16 if dt is None else dt)


def _ce_bw(abi, dx=_at(1), dw=_at(2), x=_at(3), w=_at(4), target=_at(5), lse=_at(7), dloss=_at(8),
           rows=4, hidden=16, vocab=9, ws=_at(9), wsb=1 << 40, dt=None):
    return abi.ls_linear_cross_entropy_bw(dx, dw, x, w, target, lse, dloss, rows, hidden, vocab, ws,
                                          wsb, abi.LS_BF16 if dt is None else dt)


def test_linear_cross_entropy_rejections(abi):
    bad, un, mis = abi.LS_ERR_INVALID_ARG, abi.LS_ERR_UNSUPPORTED, abi.LS_ERR_MISALIGNED
    for call, size in ((_ce_fw, abi.ls_linear_cross_entropy_fw_workspace_size),
                       (_ce_bw, abi.ls_linear_cross_entropy_bw_workspace_size)):
        assert call(abi, dt=5) == un
        assert call(abi, rows=-1) == bad and call(abi, hidden=0) == bad and call(abi, vocab=0) == bad
        assert call(abi, rows=(1 << 26) + 1) == un and call(abi, hidden=(1 << 16) + 1) == un
        assert call(abi, vocab=(1 << 28) + 1) == un
        assert call(abi, vocab=1 << 27, hidden=1 << 13) == un
        for k in ("x", "w", "target"):
            assert call(abi, **{k: None}) == bad
        assert call(abi, x=FAKE + 1) == mis and call(abi, target=FAKE + 2) == mis
        assert call(abi, w=FAKE + 8) == mis                       # rows read where they lie
        assert call(abi, w=FAKE + 1, hidden=15) == mis
        need = size(4, 16, 9, abi.LS_BF16)
        assert need > 0
        assert call(abi, ws=None) == abi.LS_ERR_WORKSPACE
        assert call(abi, ws=_at(9) + 8) == abi.LS_ERR_WORKSPACE
        assert call(abi, wsb=need - 1) == abi.LS_ERR_WORKSPACE
        for sizes in ((-1, 16, 9), (4, 0, 9), (4, 16, 0), (4, (1 << 16) + 1, 9)):
            assert size(*sizes, abi.LS_BF16) == 0
        assert size(4, 16, 9, 5) == 0
    assert abi.ls_linear_cross_entropy_fw_workspace_size(0, 16, 9, abi.LS_F32) == 0
    for k in ("loss", "lse"):
        assert _ce_fw(abi, **{k: None}) == bad and _ce_fw(abi, **{k: FAKE + 2}) == mis
    for k in ("dx", "lse", "dloss"):
        assert _ce_bw(abi, **{k: None}) == bad
        assert _ce_bw(abi, **{k: FAKE + 1}) == mis
    assert _ce_bw(abi, dw=FAKE + 1) == mis
    assert _ce_fw(abi, rows=0, loss=None, lse=None, x=None, w=None, target=None, ws=None) == abi.LS_OK
    assert _ce_bw(abi, rows=0, dw=None, dx=None, x=None, w=None, target=None, ws=None) == abi.LS_OK


def test_linear_cross_entropy_overlaps(abi):
    bad = abi.LS_ERR_INVALID_ARG
    assert _ce_fw(abi, loss=_at(2)) == bad and _ce_fw(abi, lse=_at(5)) == bad
    assert _ce_fw(abi, loss=_at(3)) == bad and _ce_fw(abi, loss=_at(6)) == bad
    assert _ce_fw(abi, ws=_at(4)) == bad
    for other in (2, 3, 4, 5, 7, 8, 9):
        assert _ce_bw(abi, dx=_at(other)) == bad, other
    for other in (3, 4, 5, 7, 8, 9):
        assert _ce_bw(abi, dw=_at(other)) == bad, other


def test_workspace_of_a_large_vocabulary_stays_below_the_logits(abi):
    """The backward keeps a piece of the logits' gradients, not all of them."""
    rows, hidden, vocab = 65536, 4096, 131072
    size = abi.ls_linear_cross_entropy_bw_workspace_size(rows, hidden, vocab, abi.LS_BF16)
    logits = rows * vocab * 2
    copies = 2 * rows * hidden * 2 + rows * hidden * 4
    assert size < logits // 4 + copies


def test_linear_cross_entropy_arguments_are_checked():
    x, w = torch.zeros(4, 16), torch.zeros(9, 16)
    t = torch.zeros(4, dtype=torch.int32)
    _raises("hidden must be", L.linear_cross_entropy_fw, x[0], w, t)
    _raises("weight must be", L.linear_cross_entropy_fw, x, w[:, :8], t)
    _raises("weight must be", L.linear_cross_entropy_fw, x, w.half(), t)
    _raises("target must be", L.linear_cross_entropy_fw, x, w, t.long())
    _raises("target must be", L.linear_cross_entropy_fw, x, w, t[:3])
    _raises("loss must be", L.linear_cross_entropy_fw, x, w, t, loss=torch.zeros(5))
    _raises("workspace must be", L.linear_cross_entropy_fw, x, w, t, workspace=torch.zeros(4, 4))
    _raises("CUDA device", L.linear_cross_entropy_fw, x, w, t)
    v = torch.zeros(4)
    _raises("lse must be", L.linear_cross_entropy_bw, x, w, t, v[:2], v)
    _raises("dloss must be", L.linear_cross_entropy_bw, x, w, t, v, v.double())
    _raises("dhidden must be", L.linear_cross_entropy_bw, x, w, t, v, v, dhidden=w)
    _raises("dweight must be", L.linear_cross_entropy_bw, x, w, t, v, v, dweight=x)
    _raises("dweight is not computed", L.linear_cross_entropy_bw, x, w, t, v, v, weight_grad=False,
            dweight=w)
    _raises("CUDA device", L.linear_cross_entropy_bw, x, w, t, v, v)
