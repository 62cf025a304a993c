"""The 64-bit references of the differential decoder's operators against automatic
differentiation and differences (CPU)."""
import pytest
import torch

import _decoder_ref as R

F64 = torch.float64


def _randn(*shape, seed=0, std=1.0):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed), dtype=F64) * std


def _close(a, b, tol=1e-9):
    assert torch.allclose(a, b, rtol=tol, atol=tol), float((a - b).abs().max())


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("lams", [1, 3])
def test_difference_of_maps(causal, lams):
    B, H, Tq, Tk = 2, 3, 4, 6
    x1, x2 = _randn(B, H, Tq, Tk).requires_grad_(), _randn(B, H, Tq, Tk, seed=1).requires_grad_()
    lam = _randn(lams, seed=2).requires_grad_()
    mask = torch.zeros(B, Tk, dtype=F64)
    mask[0, 4:] = -torch.inf
    mask[1] = _randn(Tk, seed=3)
    z = [0.7 * x + mask[:, None, None, :] for x in (x1, x2)]
    if causal:
        see = torch.ones(Tq, Tk, dtype=torch.bool).tril(Tk - Tq)
        z = [v.masked_fill(~see, -torch.inf) for v in z]
    y = torch.softmax(z[0], -1) - lam.expand(H)[None, :, None, None] * torch.softmax(z[1], -1)
    (want, _), (stats, _) = R.diff_fw(x1.detach(), x2.detach(), lam.detach(), mask, causal, 0.7)
    _close(want, y.detach())
    g = _randn(B, H, Tq, Tk, seed=4)
    (y * g).sum().backward()
    a, b, l = R.diff_bw(g, x1.detach(), x2.detach(), lam.detach(), stats, mask, causal, 0.7)
    _close(a[0], x1.grad)
    _close(b[0], x2.grad)
    _close(l[0], lam.grad)


@pytest.mark.parametrize("layer", [False, True])
@pytest.mark.parametrize("post,pre,gates", [(True, True, 1), (True, True, 3), (True, False, 6),
                                            (False, True, 0), (False, True, 2), (False, False, 1)])
def test_norms_around_a_block(layer, post, pre, gates):
    rows, D = 6, 10
    v = {"x": _randn(rows, D), "r": _randn(rows, D, seed=1)}
    if pre:
        v["g_pre"] = 1 + _randn(D, seed=2, std=0.2)
        v["b_pre"] = _randn(D, seed=3) if layer else None
    if post:
        v["g_post"] = 1 + _randn(D, seed=4, std=0.2)
        v["b_post"] = _randn(D, seed=5) if layer else None
    if gates:
        v["gate"] = _randn(gates, D, seed=6)
    v = {k: t.requires_grad_() for k, t in v.items() if t is not None}
    get = v.get
    plain = {k: t.detach() for k, t in v.items()}

    def norm(t, g, b):
        m = t.mean(-1, keepdim=True) if layer else 0.0
        n = (t - m) / ((t - m).square().mean(-1, keepdim=True) + 1e-6).sqrt() * g
        return n if b is None else n + b

    n = norm(v["x"], v["g_post"], get("b_post")) if post else v["x"]
    h = 1.3 * v["r"] + (v["gate"].repeat_interleave(rows // gates, 0) * n if gates else n)
    dy, dh = _randn(rows, D, seed=7), _randn(rows, D, seed=8)
    loss = (h * dh).sum()
    p = plain.get
    fw = R.block_fw(plain["x"], plain["r"], p("g_pre"), p("b_pre"), p("g_post"), p("b_post"),
                    p("gate"), 1.3, layer, 1e-6)
    _close(fw[0][0], h.detach())
    if pre:
        y = norm(h, v["g_pre"], get("b_pre"))
        _close(fw[1][0], y.detach())
        loss = loss + (y * dy).sum()
    loss.backward()
    out = R.block_bw(dy if pre else None, dh, plain["x"], h.detach(), fw[2][0], p("g_pre"),
                     p("g_post"), p("b_post"), p("gate"), 1.3, layer)
    names = {"dx": "x", "dr": "r", "dg_pre": "g_pre", "db_pre": "b_pre", "dg_post": "g_post",
             "db_post": "b_post", "dgate": "gate"}
    for k, (val, _) in out.items():
        _close(val, v[names[k]].grad)
    assert {names[k] for k in out} == set(v)


def test_cross_entropy_from_hidden_states():
    N, D, V = 7, 5, 11
    x, w = _randn(N, D).requires_grad_(), _randn(V, D, seed=1).requires_grad_()
    t = torch.tensor([0, 10, -1, 3, 3, -5, 9], dtype=torch.int32)
    live = t >= 0
    z = x @ w.T
    loss = torch.nn.functional.cross_entropy(z[live], t[live].long(), reduction="none")
    (val, _), (lse, _) = R.loss_fw(x.detach(), w.detach(), t)
    _close(val[live], loss.detach())
    assert (val[~live] == 0).all() and (lse[~live] == 0).all()
    up = _randn(N, seed=2)
    (loss * up[live]).sum().backward()
    (dx, _), (dw, _) = R.loss_bw(x.detach(), w.detach(), t, lse, up)
    _close(dx, x.grad)
    _close(dw, w.grad)
    # and a difference of the loss itself
    step = 1e-6
    e = torch.zeros_like(w)
    e[3, 2] = step
    hi, lo = (float((R.loss_fw(x.detach(), w.detach() + s * e, t)[0][0] * up)[live].sum())
              for s in (1, -1))
    assert abs((hi - lo) / (2 * step) - float(dw[3, 2])) < 1e-6


def test_a_class_beyond_the_vocabulary_is_nan():
    x, w = _randn(3, 4), _randn(5, 4, seed=1)
    t = torch.tensor([1, 5, -1], dtype=torch.int32)
    (val, _), (lse, _) = R.loss_fw(x, w, t)
    assert val.isnan().tolist() == [False, True, False]
    (dx, _), (dw, _) = R.loss_bw(x, w, t, lse, torch.ones(3))
    assert dx.isnan().any(-1).tolist() == [False, True, False] and dw.isnan().all()
