"""The 64-bit references of the position operators and of the clipping against
facts that do not come from them: central differences, closed forms, torch's
own softmax and norm."""
import math

import pytest
import torch

import _position_ref as R
import transformer_reduce_gb300 as L

F64 = torch.float64


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _differences(f, x, step=1e-5):
    """Gradient of the scalar f at x by central differences."""
    g = torch.zeros_like(x)
    for i in range(x.numel()):
        keep = float(x.view(-1)[i])
        x.view(-1)[i] = keep + step
        up = float(f())
        x.view(-1)[i] = keep - step
        g.view(-1)[i] = (up - float(f())) / (2 * step)
        x.view(-1)[i] = keep
    return g


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("Tq,Tk", [(4, 7), (7, 7), (1, 6)])
def test_relpos_gradients_against_differences(Tq, Tk, causal):
    B, H, nb = 2, 2, 8
    buckets = L.relpos_buckets(nb, 5, device="cpu")
    x = torch.randn(B, H, Tq, Tk, generator=_gen(1), dtype=F64)
    table = torch.randn(nb, H, generator=_gen(2), dtype=F64)
    dout = torch.randn(B, H, Tq, Tk, generator=_gen(3), dtype=F64)
    mask = torch.zeros(B, Tk, dtype=F64)
    mask[0, Tk - 2:] = -math.inf
    mask[1, 0] = -0.7

    def loss():
        return (R.relpos_fw(x, table, buckets, mask, causal, 0.6)[0] * dout).sum()

    y = R.relpos_fw(x, table, buckets, mask, causal, 0.6)[0]
    (dx, _), (dt, _) = R.relpos_bw(dout, y, buckets, nb, mask, causal, 0.6)
    assert torch.allclose(dx, _differences(loss, x), atol=1e-8)
    assert torch.allclose(dt, _differences(loss, table), atol=1e-8)


def test_relpos_reference_against_torch_softmax():
    B, H, Tq, Tk, nb = 2, 3, 5, 9, 8
    buckets = L.relpos_buckets(nb, 6, device="cpu")
    x = torch.randn(B, H, Tq, Tk, generator=_gen(4), dtype=F64)
    table = torch.randn(nb, H, generator=_gen(5), dtype=F64)
    y, _ = R.relpos_fw(x, table, buckets, None, False, 0.5)
    bias = torch.empty(H, Tq, Tk, dtype=F64)
    for i in range(Tq):
        for j in range(Tk):
            r = max(-6, min(6, j - (i + Tk - Tq)))
            bias[:, i, j] = table[int(buckets[r + 6])]
    assert torch.allclose(y, torch.softmax(x * 0.5 + bias, -1), atol=1e-14)
    # a row without a key is zeros
    mask = torch.zeros(B, Tk, dtype=F64)
    mask[1] = -math.inf
    y, _ = R.relpos_fw(x, table, buckets, mask, False, 0.5)
    assert torch.all(y[1] == 0) and torch.allclose(y[0].sum(-1), torch.ones(H, Tq, dtype=F64))


@pytest.mark.parametrize("nb,dist,both", [(32, 128, True), (32, 128, False), (8, 20, True),
                                          (12, 300, True), (5, 17, False), (64, 2048, True)])
def test_bucket_map(nb, dist, both):
    b = L.relpos_buckets(nb, dist, both, device="cpu")
    assert b.shape == (2 * dist + 1,) and b.dtype == torch.int32
    half = nb // 2 if both else nb
    e = half // 2
    before = b[:dist + 1].flip(0).tolist()  # by growing distance
    assert before[:e] == list(range(e)) and before[dist] == half - 1
    assert all(0 <= v - u <= max(1, half) for u, v in zip(before, before[1:]))
    assert set(before) <= set(range(half))
    after = b[dist:].tolist()
    if both:
        assert after[1:] == [half + v for v in before[1:]]
    else:
        assert set(after) == {0}
    # wide buckets begin where the ratio says, up to a rounding of the logarithm
    for n in range(e, dist):
        t = math.log(n / e) / math.log(dist / e) * (half - e)
        assert before[n] in {min(half - 1, e + int(t - 1e-9)), min(half - 1, e + int(t + 1e-9))}
    with pytest.raises(ValueError):
        L.relpos_buckets(2, 128, True, device="cpu")
    with pytest.raises(ValueError):
        L.relpos_buckets(nb, e, both, device="cpu")


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("D,rot", [(8, 8), (7, 4), (6, 0)])
def test_qk_gradients_against_differences(D, rot, interleaved):
    T, Hn = 3, 2
    x = torch.randn(T, Hn, D, generator=_gen(6), dtype=F64)
    gamma = 1 + 0.3 * torch.randn(D, generator=_gen(7), dtype=F64)
    dout = torch.randn(T, Hn, D, generator=_gen(8), dtype=F64)
    cos = sin = pos = None
    if rot:
        ang = torch.rand(5, rot // 2, generator=_gen(9), dtype=F64) * 6
        cos, sin = ang.cos(), ang.sin()
        pos = torch.tensor([4, 0, 2], dtype=torch.int32)

    def loss():
        return (R.qk_fw(x, gamma, cos, sin, pos, interleaved, 1e-3)[0][0] * dout).sum()

    rstd = R.qk_fw(x, gamma, cos, sin, pos, interleaved, 1e-3)[1][0]
    (dx, _), (dg, _) = R.qk_bw(dout, x, gamma, rstd, cos, sin, pos, interleaved)
    assert torch.allclose(dx, _differences(loss, x), atol=1e-8)
    assert torch.allclose(dg, _differences(loss, gamma), atol=1e-8)


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_keeps_length_and_adds_angles(interleaved):
    cos, sin = (t.double() for t in L.rope_tables(64, 8, device="cpu"))
    x = torch.randn(4, 3, 10, generator=_gen(10), dtype=F64)
    at = lambda p: torch.full((4,), p, dtype=torch.int32)  # noqa: E731
    y = R.rotate(x, cos, sin, at(20), interleaved)
    assert torch.allclose(y.norm(dim=-1), x.norm(dim=-1), atol=1e-6)
    assert torch.equal(y[..., 8:], x[..., 8:])
    both = R.rotate(y, cos, sin, at(11), interleaved)
    assert torch.allclose(both, R.rotate(x, cos, sin, at(31), interleaved), atol=1e-6)
    assert torch.allclose(R.rotate(y, cos, sin, at(20), interleaved, back=True), x, atol=1e-6)
    assert torch.equal(R.rotate(x, cos, sin, at(0), interleaved), x)


def test_rope_tables():
    cos, sin = L.rope_tables(100, 6, base=500.0, device="cpu")
    assert cos.shape == sin.shape == (100, 3) and cos.dtype == torch.float32
    for pos in (0, 1, 57, 99):
        for p in range(3):
            a = pos * 500.0 ** (-2 * p / 6)
            assert abs(float(cos[pos, p]) - math.cos(a)) <= 2.0 ** -24
            assert abs(float(sin[pos, p]) - math.sin(a)) <= 2.0 ** -24
    for rot in (0, 3):
        with pytest.raises(ValueError):
            L.rope_tables(4, rot, device="cpu")


def test_clip_reference():
    grads = [torch.tensor([3.0, 0.0]), torch.tensor([[4.0]])]
    (norm, _), outs = R.clip(grads, 1.0, 0.0)
    assert float(norm) == 5.0
    assert torch.allclose(outs[0][0], torch.tensor([0.6, 0.0], dtype=F64))
    (_, _), outs = R.clip(grads, 6.0, 0.0)
    assert torch.equal(outs[1][0], grads[1].double())
