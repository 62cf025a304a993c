"""GPU parity of the plain and the scaled softmax for rows whose largest score is
far from zero: rows that see only keys hidden by a finite mask, large scores."""
import pytest
import torch

import _position_ref as R
import _softmax_range as S

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


def _check(L, x, mask, causal, scale, what):
    """Both kernels: an output off a 16-byte address takes the looped one.  That
    one forms z log2 e first, so below 2^20, where it does so, its weights are
    off by a few u of |z| and |m| each, not of their difference."""
    H = x.shape[1]
    none = torch.zeros((1, H), dtype=x.dtype, device=DEV)
    buckets = torch.zeros(3, dtype=torch.int32, device=DEV)
    want, tol = S.biased_softmax(x, none, buckets, mask, causal, scale or 1.0)
    z, _ = S.scores(x, none, buckets, mask, causal, scale or 1.0)
    m = z.amax(-1, keepdim=True).abs()
    near = torch.where(z.isneginf(), 0.0, z.abs()).minimum(m + 110) + m
    loose = tol + want * 4 * R.U * torch.where(m < 2.0 ** 20, near, 0.0)
    for out in (None, torch.empty(x.numel() + 1, dtype=x.dtype, device=DEV)[1:].view(x.shape)):
        y = L.softmax_fw(x, mask, causal=causal, scale=scale, out=out)
        R.check(y, want, loose, f"{what}, scale {scale}, {'own' if out is None else 'other'} offset")


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("fill", ["lowest", -1e4, -1e6, -1e9, -3e9, -2.0 ** 32 + 1, -1e10, -1e12,
                                  -1e20, -1e30, 1e10])
def test_rows_that_see_only_keys_hidden_by_a_finite_mask(lib, dt, fill):
    dtype = DT[dt]
    fill = torch.finfo(dtype).min if fill == "lowest" else fill
    step = 2.0 ** -10 if dt == "f32" else 2.0 ** -4
    g = torch.Generator(device=DEV).manual_seed(1)
    for Tk in (8, 45, 64, 512, 1000, 2100, 4096):
        shape = (3, 2, min(Tk, 40), Tk)
        x = S.grid(torch.randn(shape, generator=g, device=DEV) * 3, step).to(dtype)
        mask = torch.zeros(3, Tk, device=DEV)
        mask[0] = fill
        mask[1, Tk // 2:] = fill
        mask[2, :Tk - 3] = fill
        mask = mask.to(dtype)
        for causal in (False, True):
            for scale in (None, 0.5):
                _check(lib, x, mask, causal, scale, f"{Tk} causal {causal}")


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("power", [16, 22, 33, 90])
def test_rows_of_large_scores(lib, dt, power):
    for Tk in (40, 77, 600, 2100):
        whole = torch.randint(-8, 9, (2, 2, 9, Tk), device=DEV,
                              generator=torch.Generator(device=DEV).manual_seed(power))
        x = (whole.double() * 2.0 ** (power - 3)).to(DT[dt])
        mask = torch.zeros(2, Tk, device=DEV, dtype=DT[dt])
        mask[1, Tk // 2:] = -torch.inf
        for scale in (None, 0.5, 2.0):
            _check(lib, x, mask, False, scale, f"{Tk}")
        _check(lib, -x.abs() - x.abs().max(), None, True, None, f"{Tk} negative")


@pytest.mark.parametrize("dt", list(DT))
def test_empty_rows_stay_zero_and_infinities_stay_invisible(lib, dt):
    g = torch.Generator(device=DEV).manual_seed(2)
    for Tk in (64, 77, 2101):
        x = torch.randn(2, 2, 5, Tk, generator=g, device=DEV).to(DT[dt])
        mask = torch.zeros(2, Tk, device=DEV, dtype=DT[dt])
        mask[0] = -torch.inf
        mask[1, ::2] = -torch.inf
        y = lib.softmax_fw(x, mask)
        assert torch.all(y[0] == 0) and torch.all(y[1, ..., ::2] == 0)
        assert torch.allclose(y[1].float().sum(-1), torch.ones((), device=DEV), atol=2e-2)
