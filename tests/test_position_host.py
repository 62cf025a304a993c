"""Host-side refusals of the softmax with a relative position bias, the
per-head norm with rotation and the gradient clipping: through the C ABI and
through the PyTorch layer.  No kernel is launched here."""
import ctypes
import math

import pytest
import torch

import transformer_reduce_gb300 as L

FAKE = 0x10000  # never dereferenced: every call below returns on the host


@pytest.fixture(scope="module")
def abi():
    from transformer_reduce_gb300 import build as b
    b.build()
    from transformer_reduce_gb300 import _lib
    _lib.load()
    return _lib


def _fw(abi, out=FAKE, inp=FAKE, mask=None, table=FAKE, bucket=FAKE, B=1, H=2, Tq=4, Tk=4, nb=8,
        R=5, causal=0, scale=1.0, dt=None):
    return abi.ls_softmax_fw_relpos(out, inp, mask, table, bucket, B, H, Tq, Tk, nb, R, causal,
                                    scale, abi.LS_F32 if dt is None else dt)


def _bw(abi, dinp=FAKE, dtable=FAKE, dout=FAKE, y=FAKE, mask=None, bucket=FAKE, B=1, H=2, Tq=4,
        Tk=4, nb=8, R=5, causal=0, scale=1.0, ws=FAKE, wsb=1 << 40, dt=None):
    return abi.ls_softmax_bw_relpos(dinp, dtable, dout, y, mask, bucket, B, H, Tq, Tk, nb, R,
                                    causal, scale, ws, wsb, abi.LS_F32 if dt is None else dt)


def test_relpos_rejections(abi):
    bad, un, mis = abi.LS_ERR_INVALID_ARG, abi.LS_ERR_UNSUPPORTED, abi.LS_ERR_MISALIGNED
    for call in (_fw, _bw):
        assert call(abi, dt=7) == un
        for k in ("B", "H", "Tq", "Tk"):
            assert call(abi, **{k: -1}) == bad
        assert call(abi, nb=0) == bad and call(abi, R=0) == bad
        assert call(abi, R=2049) == un and call(abi, nb=65537) == un
        assert call(abi, Tk=(1 << 30) + 1) == un and call(abi, Tq=(1 << 30) + 1) == un
        assert call(abi, B=1 << 40, H=1 << 20, Tq=1 << 20) == un
        assert call(abi, Tq=5, causal=1) == bad
        for scale in (0.0, -1.0, math.inf, math.nan):
            assert call(abi, scale=scale) == bad
        assert call(abi, bucket=None) == bad and call(abi, bucket=FAKE + 2) == mis
        assert call(abi, mask=FAKE + 2) == mis
    assert _fw(abi, out=None) == bad and _fw(abi, inp=None) == bad and _fw(abi, table=None) == bad
    assert _fw(abi, out=FAKE + 1, dt=abi.LS_BF16) == mis and _fw(abi, table=FAKE + 2) == mis
    for k in ("dinp", "dtable", "dout", "y"):
        assert _bw(abi, **{k: None}) == bad
        assert _bw(abi, **{k: FAKE + 2}) == mis
    need = abi.ls_softmax_bw_relpos_workspace_size(2, 5)
    assert need % (11 * 4) == 0 and need > 0
    assert _bw(abi, ws=None) == abi.LS_ERR_WORKSPACE
    assert _bw(abi, ws=FAKE + 8) == abi.LS_ERR_WORKSPACE
    assert _bw(abi, wsb=need - 1) == abi.LS_ERR_WORKSPACE
    # empty problems: nothing to do, whatever the pointers
    assert _fw(abi, None, None, None, None, None, B=0) == abi.LS_OK
    assert _fw(abi, None, None, None, None, None, Tk=0) == abi.LS_OK
    assert _bw(abi, None, None, None, None, None, None, H=0, ws=None) == abi.LS_OK
    ws = abi.ls_softmax_bw_relpos_workspace_size
    assert ws(0, 5) == ws(2, 0) == ws(2, 2049) == ws(-1, 5) == 0


def _qk(abi, dt=None, **kw):
    a = dict(q_out=FAKE, k_out=FAKE, q_rstd=FAKE, k_rstd=FAKE, q=FAKE, k=FAKE, gq=FAKE, gk=FAKE,
             cos=FAKE, sin=FAKE, pos=FAKE, tokens=4, Hq=4, Hk=2, D=16, rot=16, max_pos=8, qos=64,
             kos=32, qs=64, ks=32, il=0, eps=1e-6)
    assert set(kw) <= set(a)
    a.update(kw)
    return abi.ls_qk_norm_rope_fw(*a.values(), abi.LS_F32 if dt is None else dt)


def _qkb(abi, dt=None, **kw):
    a = dict(dq=FAKE, dk=FAKE, dgq=FAKE, dgk=FAKE, dqo=FAKE, dko=FAKE, q=FAKE, k=FAKE, gq=FAKE,
             gk=FAKE, rq=FAKE, rk=FAKE, cos=FAKE, sin=FAKE, pos=FAKE, tokens=4, Hq=4, Hk=2, D=16,
             rot=16, max_pos=8, dqs=64, dks=32, dqos=64, dkos=32, qs=64, ks=32, il=0, ws=FAKE,
             wsb=1 << 40)
    assert set(kw) <= set(a)
    a.update(kw)
    return abi.ls_qk_norm_rope_bw(*a.values(), abi.LS_F32 if dt is None else dt)


def test_qk_rejections(abi):
    bad, un, mis = abi.LS_ERR_INVALID_ARG, abi.LS_ERR_UNSUPPORTED, abi.LS_ERR_MISALIGNED
    for call in (_qk, _qkb):
        assert call(abi, dt=-1) == un
        for k in ("tokens", "Hq", "Hk", "rot"):
            assert call(abi, **{k: -1}) == bad
        assert call(abi, D=0, rot=0) == bad and call(abi, rot=18) == bad and call(abi, rot=3) == bad
        assert call(abi, D=1025, qs=1 << 20, ks=1 << 20) == un
        for k in ("q", "k", "gq", "gk", "cos", "sin", "pos"):
            assert call(abi, **{k: None}) == bad
            assert call(abi, **{k: FAKE + 2}) == mis
        assert call(abi, max_pos=0) == bad
        assert call(abi, qs=63) == bad and call(abi, ks=31) == bad
        assert call(abi, tokens=1 << 60) == un
        assert call(abi, Hq=(1 << 29) + 1, qs=1 << 40) == un
        assert call(abi, Hk=(1 << 29) + 1, ks=1 << 40) == un
        assert call(abi, tokens=1 << 40, qs=1 << 40) == un
    assert _qk(abi, eps=-1.0) == bad and _qk(abi, eps=math.nan) == bad
    assert _qk(abi, q_out=None) == bad and _qk(abi, qos=63) == bad and _qk(abi, kos=31) == bad
    assert _qk(abi, q_rstd=FAKE + 2) == mis
    for k in ("dq", "dk", "dqo", "dko", "rq", "rk", "dgq", "dgk"):
        assert _qkb(abi, **{k: None}) == bad
        assert _qkb(abi, **{k: FAKE + 2}) == mis
    need = abi.ls_qk_norm_rope_bw_workspace_size(4, 4, 2, 16)
    assert need > 0 and need % 64 == 0
    for kw in (dict(ws=None), dict(ws=FAKE + 4), dict(wsb=need - 1)):
        assert _qkb(abi, **kw) == abi.LS_ERR_WORKSPACE
    assert _qk(abi, tokens=0, q=None, k=None, q_out=None) == abi.LS_OK
    assert _qk(abi, Hq=0, Hk=0, q=None, k=None) == abi.LS_OK
    assert _qkb(abi, Hq=0, Hk=0, q=None, k=None) == abi.LS_OK
    ws = abi.ls_qk_norm_rope_bw_workspace_size
    assert ws(0, 4, 2, 16) == ws(4, 4, 2, 0) == ws(4, -1, 2, 16) == ws(4, 4, 2, 1025) == 0
    assert ws(4, 0, 0, 16) == 0


def _lists(ptrs, sizes, dts):
    n = len(ptrs)
    return ((ctypes.c_void_p * n)(*ptrs), (ctypes.c_int64 * n)(*sizes), (ctypes.c_int32 * n)(*dts))


def test_clip_rejections(abi):
    bad, un, mis = abi.LS_ERR_INVALID_ARG, abi.LS_ERR_UNSUPPORTED, abi.LS_ERR_MISALIGNED
    big = 1 << 40

    def both(ptrs=(FAKE, FAKE), sizes=(3, 4), dts=(0, 1), norm=FAKE, ws=FAKE, wsb=big, count=2):
        p, s, d = _lists(ptrs, sizes, dts)
        r = abi.ls_grad_norm(norm, p, s, d, count, ws, wsb)
        assert abi.ls_grad_clip(norm, p, p, s, d, count, 1.0, 0.0, ws, wsb) == r
        return r

    assert both(norm=None) == bad and both(norm=FAKE + 2) == mis
    assert both(count=-1) == bad
    assert both(ptrs=(None, FAKE)) == bad and both(sizes=(-1, 4)) == bad
    assert both(dts=(0, 5)) == un and both(sizes=(1 << 60, 1 << 60)) == un
    assert both(ptrs=(FAKE + 2, FAKE)) == mis and both(ptrs=(FAKE, FAKE + 1)) == mis
    need = abi.ls_grad_norm_workspace_size(2)
    assert need == abi.ls_grad_norm_workspace_size(1) > 0
    assert abi.ls_grad_norm_workspace_size(0) == abi.ls_grad_norm_workspace_size(-4) == 0
    assert abi.ls_grad_norm_workspace_size(513) == 2 * need
    for kw in (dict(ws=None), dict(ws=FAKE + 8), dict(wsb=need - 1)):
        assert both(**kw) == abi.LS_ERR_WORKSPACE
    p, s, d = _lists((FAKE,), (3,), (0,))
    assert abi.ls_grad_norm(FAKE, None, s, d, 1, FAKE, big) == bad
    assert abi.ls_grad_norm(FAKE, p, None, d, 1, FAKE, big) == bad
    assert abi.ls_grad_norm(FAKE, p, s, None, 1, FAKE, big) == bad
    assert abi.ls_grad_clip(FAKE, None, p, s, d, 1, 1.0, 0.0, FAKE, big) == bad
    for m in (0.0, -1.0, math.inf, math.nan):
        assert abi.ls_grad_clip(FAKE, p, p, s, d, 1, m, 0.0, FAKE, big) == bad
    for e in (-1.0, math.inf, math.nan):
        assert abi.ls_grad_clip(FAKE, p, p, s, d, 1, 1.0, e, FAKE, big) == bad


def _raises(match, fn, *a, **k):
    with pytest.raises((ValueError, TypeError), match=match):
        fn(*a, **k)


def test_binding_checks_relpos():
    s = torch.zeros(2, 3, 4, 8, dtype=torch.bfloat16)
    t = torch.zeros(8, 3, dtype=torch.bfloat16)
    b = L.relpos_buckets(8, 5, device="cpu")
    _raises("scores must be", L.softmax_fw_relpos, s[0], t, b)
    _raises("table must be", L.softmax_fw_relpos, s, t[:, :2], b)
    _raises("table must be", L.softmax_fw_relpos, s, t.float(), b)
    _raises("table must be", L.softmax_fw_relpos, s, t[:, 0], b)
    _raises("buckets must be", L.softmax_fw_relpos, s, t, b.long())
    _raises("buckets must be", L.softmax_fw_relpos, s, t, b[:-1])
    _raises("buckets must be", L.softmax_fw_relpos, s, t, b[None])
    _raises("mask must be", L.softmax_fw_relpos, s, t, b, s[0, 0])
    _raises("out must be", L.softmax_fw_relpos, s, t, b, out=s[:1])
    _raises("CUDA device", L.softmax_fw_relpos, s, t, b)
    _raises("dout must be", L.softmax_bw_relpos, s[0], s, b, 8)
    _raises("out_fw must be", L.softmax_bw_relpos, s, s[:1], b, 8)
    _raises("dinp must be", L.softmax_bw_relpos, s, s, b, 8, dinp=s.float())
    _raises("dtable must be", L.softmax_bw_relpos, s, s, b, 8, dtable=t)
    _raises("workspace must be", L.softmax_bw_relpos, s, s, b, 8, workspace=t)
    _raises("CUDA device", L.softmax_bw_relpos, s, s, b, 8)


def test_binding_checks_qk():
    q, k = torch.zeros(5, 4, 16), torch.zeros(5, 2, 16)
    g = torch.ones(16)
    cos, sin = L.rope_tables(9, 8, device="cpu")
    pos = torch.zeros(5, dtype=torch.int32)
    fw = L.qk_norm_rope_fw
    _raises("q must be", fw, q[0], k, g, g)
    _raises("k must be", fw, q, k[:4], g, g)
    _raises("k must be", fw, q, k[..., :8], g, g)
    _raises("k must be", fw, q, k.half(), g, g)
    _raises("gamma_q must be", fw, q, k, g[:8], g)
    _raises("gamma_k must be", fw, q, k, g, g.half())
    _raises("dense heads", fw, q.transpose(0, 1), q.transpose(0, 1), g, g)
    _raises("dense heads", fw, q[..., ::2], k[..., ::2], g[:8], g[:8])
    _raises("overlap itself", fw, q[:1].expand(5, 4, 16), k, g, g)
    _raises("go together", fw, q, k, g, g, cos, sin)
    _raises("cos must be", fw, q, k, g, g, torch.zeros(9, 9), torch.zeros(9, 9), pos)
    _raises("cos must be", fw, q, k, g, g, cos.double(), sin, pos)
    _raises("sin must be", fw, q, k, g, g, cos, sin[:, :2], pos)
    _raises("positions must be", fw, q, k, g, g, cos, sin, pos.long())
    _raises("positions must be", fw, q, k, g, g, cos, sin, pos[:4])
    _raises("q_out must be", fw, q, k, g, g, q_out=k)
    _raises("k_out must be", fw, q, k, g, g, k_out=k.half())
    _raises("q_rstd must be", fw, q, k, g, g, q_rstd=torch.zeros(5, 3))
    _raises("CUDA device", fw, q, k, g, g, cos, sin, pos)
    bw, rq, rk = L.qk_norm_rope_bw, torch.ones(5, 4), torch.ones(5, 2)
    _raises("dq_out must be", bw, k, k, q, k, g, g, rq, rk)
    _raises("dk_out must be", bw, q, q, q, k, g, g, rq, rk)
    _raises("k_rstd must be", bw, q, k, q, k, g, g, rq, rq)
    _raises("dgamma_q must be", bw, q, k, q, k, g, g, rq, rk, dgamma_q=torch.zeros(15))
    _raises("dk must be", bw, q, k, q, k, g, g, rq, rk, dk=q)
    _raises("workspace must be", bw, q, k, q, k, g, g, rq, rk, workspace=g.half())
    _raises("CUDA device", bw, q, k, q, k, g, g, rq, rk)


def test_binding_checks_clip():
    g = torch.zeros(4, 4)
    _raises("empty list", L.grad_norm, [])
    _raises("CUDA device", L.grad_norm, [g])
    _raises("CUDA device", L.grad_clip, [g], 1.0)
    _raises("contiguous", L.grad_norm, [_Cuda(g.t()[:2])])
    _raises("unsupported", L.ls_dtype, g.double())


class _Cuda:
    """A tensor that says it is on a GPU, for checks that come after that one."""

    def __init__(self, t):
        self._t = t

    is_cuda = True

    def __getattr__(self, name):
        return getattr(self._t, name)


def test_binding_checks_clip_outputs():
    a, b = _Cuda(torch.zeros(4)), _Cuda(torch.zeros(5))
    _raises("out must hold", L.grad_clip, [a, b], 1.0, out=[a])
    _raises(r"out\[1\] must be", L.grad_clip, [a, b], 1.0, out=[a, a])
    _raises("in out twice", L.grad_clip, [a, a], 1.0)
    _raises("unsupported", L.grad_clip, [_Cuda(torch.zeros(4).double())], 1.0)
