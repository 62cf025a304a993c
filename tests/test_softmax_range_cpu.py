"""The reference of tests/_softmax_range.py: its bound refuses wrong answers for
every kind of mask and type, and its values are torch's softmax of the same z."""
import math

import pytest
import torch

import _position_ref as R
import _softmax_range as S

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
INF = math.inf


def _inputs(dt, kind, B=3, H=2, Tq=5, Tk=40):
    g = torch.Generator().manual_seed(3)
    dtype = DT[dt]
    x = S.grid(torch.randn(B, H, Tq, Tk, generator=g) * 2, 2.0 ** -5).to(dtype)
    table = S.grid(torch.randn(9, H, generator=g), 2.0 ** -5).to(dtype)
    buckets = torch.arange(9, dtype=torch.int32)
    low = torch.finfo(dtype).min
    fill = {"pad": -INF, "lowest": low, "mixed": low, "1e10": max(-1e10, low)}.get(kind)
    m = torch.zeros(B, Tk)
    if fill is not None:
        m[1, Tk // 2:] = fill
        m[2, :] = fill
    if kind == "mixed":
        m += S.grid(torch.randn(B, Tk, generator=g), 2.0 ** -5)
        m = m.clamp(min=low)
    return x, table, buckets, None if kind == "none" else m.to(dtype)


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("kind", ["none", "pad", "lowest", "mixed", "1e10"])
def test_bound_refuses_wrong_answers(dt, kind):
    x, table, buckets, m = _inputs(dt, kind)
    for causal in (False, True):
        y, tol = S.biased_softmax(x, table, buckets, m, causal, 0.5)
        z, vis = S.scores(x, table, buckets, m, causal, 0.5)
        empty = z.amax(-1).isneginf()
        want = torch.where(empty[..., None], 0.0, torch.softmax(z, -1))
        assert float((y - want).abs().max()) < 1e-14
        stored = y.to(DT[dt])
        R.check(stored, y, tol, "the answer itself")
        uniform = vis.double() / vis.double().sum(-1, keepdim=True).clamp(min=1)
        for b in range(x.shape[0]):
            if bool(empty[b].all()):
                continue
            flat = bool((z[b].amax(-1) == z[b].masked_fill(~vis[b], INF).amin(-1)).all())
            for wrong in (torch.zeros_like(y), 2 * y, y * 1.02, uniform):
                if wrong is uniform and flat:
                    continue  # every key of the row at one value: uniform is right
                with pytest.raises(AssertionError):
                    R.check(wrong[b], y[b], tol[b], "wrong")
