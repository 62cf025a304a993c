"""The scaled softmax on rows whose largest scaled score lies far beyond 2^20,
at scales that are no powers of two: the difference to the largest score is
taken before the scale.

Bound, u = 2^-24, of a weight e^(s (x_j - top)): the difference, its products
with the scale and log2 e and the constants are off by u each relative to the
exponent, 4 u |gap| (a row nearer than 2^20 has one product, one constant and
the fused sum); ex2.approx and rcp.approx by 4 u each, the sum by the mean of
its weights' errors and u per term of its chain, Tk / 32 + 10 at most.  Rows that
are no whole number of 16-byte vectors, and very long ones, round the product
s x_j to FP32 first: their weights are those of fl(s x_j), within the same
bound, and a call has to agree with one of the two throughout."""
import math

import pytest
import torch

from _position_ref import U, check, half_step, tiny

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


def _want(x, causal, scale, rounded):
    Tq, Tk = x.shape[-2:]
    z = x.double() * torch.tensor(scale, dtype=torch.float32).double().item()
    if rounded:
        z = z.float().double()
    if causal:
        see = torch.ones(Tq, Tk, dtype=torch.bool, device=DEV).tril(Tk - Tq)
        z = z.masked_fill(~see, -math.inf)
    gap = z.amax(-1, keepdim=True) - z
    y = torch.softmax(z, -1)
    gap = gap.clamp(max=110.0)
    mean = (y * gap).sum(-1, keepdim=True)
    return y, y * (half_step(x.dtype) + U * (4 * gap + 4 * mean + Tk / 32 + 70)) + tiny(x.dtype)


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("scale", [0.3, 0.7, 0.0884])
@pytest.mark.parametrize("Tk", [33, 64, 100, 512, 1000, 2048, 3000])
def test_rows_of_far_scores(lib, dt, scale, Tk):
    dtype = DT[dt]
    low = torch.finfo(dtype).min
    gen = torch.Generator(device=DEV).manual_seed(Tk)
    for base in (low, 3e4, -2e6, 1e9, -3e9, 1e12, -1e30):
        if abs(base) > -low:
            continue
        shape = (2, 2, 5, Tk)
        if base == low:  # every score of the rows was hidden by hand
            x = torch.full(shape, low, device=DEV).to(dtype)
        else:  # neighbours of a few steps of the type, or of a few units
            step = max(1.0, abs(base) * torch.finfo(dtype).eps)
            x = (torch.randn(shape, generator=gen, device=DEV) * 2 * step + base).to(dtype)
        for causal in (False, True):
            got = lib.softmax_fw(x, causal=causal, scale=scale)
            y, tol = _want(x, causal, scale, True)
            if not bool(((got.double() - y).abs() <= tol).all()):
                y, tol = _want(x, causal, scale, False)
            check(got, y, tol, f"{base} {causal}")


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("Tk", [64, 77, 513, 20000])
def test_filled_rows_are_uniform_under_a_padding_mask(lib, dt, Tk):
    """Also where the mask is added element by element, and in very long rows."""
    x = torch.full((2, 2, 5, Tk), torch.finfo(DT[dt]).min, dtype=DT[dt], device=DEV)
    mask = torch.zeros(2, Tk, dtype=DT[dt], device=DEV)
    mask[1, Tk // 2:] = -math.inf
    for holes in (False, True):
        if holes:
            mask[0, 3:6] = -math.inf
        see = ~mask.isneginf()[:, None, None, :].expand(x.shape)
        want = torch.where(see, 1.0 / see.sum(-1, keepdim=True).double(), 0.0)
        got = lib.softmax_fw(x, mask, scale=0.7)
        check(got, want, want * (half_step(x.dtype) + U * (Tk / 32 + 20)) + tiny(x.dtype), "filled")
