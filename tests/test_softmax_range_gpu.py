"""GPU parity of the softmax with a relative position bias where a row's largest
score is far from zero (rows that see only keys hidden by a finite mask, large
scores), and for every kind of mask, within a bound that stays tight there."""
import math

import pytest
import torch

import _position_ref as R
import _softmax_range as S

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
INF = math.inf
# finite masks that programs hide keys with, and the ones around 2^20 and 2^31
FILLS = [-1e4, -2.0 ** 20, -1.5 * 2.0 ** 20, -1e8, -1e9, -2.0 ** 31, -2e9, -3e9, -2.0 ** 32 + 1, -5e9,
         -1e10, -1e12, -1e15, -1e20, -1e29, -1e30, -1e36, 1e10, 1e20]


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from transformer_reduce_gb300 import build
    build.build()
    import transformer_reduce_gb300 as L
    L.load()
    return L


def _randn(shape, seed, std=1.0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return torch.randn(shape, generator=g, device=DEV) * std


def _inputs(L, shape, dtype, scale=0.5, seed=1):
    step = 2.0 ** -10 if dtype == torch.float32 else 2.0 ** -4
    x = S.grid(_randn(shape, seed, 2.0 / scale), step).to(dtype)
    table = S.grid(_randn((16, shape[1]), seed + 1, 0.8), step).to(dtype)
    return x, table, L.relpos_buckets(16, 24, device=DEV)


def _shifted(t, k=1):
    """A dense tensor of t's shape that starts k elements into its storage."""
    return torch.empty(t.numel() + k, dtype=t.dtype, device=DEV)[k:].view(t.shape)


def _check(L, x, table, buckets, mask, causal, scale, what):
    """The register-resident kernel (where the length allows it) and, with an
    output at another offset, the looped one."""
    want, tol = S.biased_softmax(x, table, buckets, mask, causal, scale)
    for out, how in ((None, "same offset"), (_shifted(x), "other offset")):
        y = L.softmax_fw_relpos(x, table, buckets, mask, causal=causal, scale=scale, out=out)
        R.check(y, want, tol, f"{what}, {how}")


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("fill", FILLS)
def test_rows_that_see_only_keys_hidden_by_a_finite_mask(lib, dt, fill):
    """An empty batch entry, and a left-padded sentence under causal."""
    dtype = DT[dt]
    for Tk in (24, 45, 130, 512, 777, 2100):
        shape = (3, 2, min(Tk, 48), Tk)
        x, table, buckets = _inputs(lib, shape, dtype)
        mask = torch.zeros(3, Tk, device=DEV)
        mask[0] = fill
        mask[1, Tk // 2:] = fill
        mask[2, :Tk - 3] = fill
        mask = mask.to(dtype)
        for causal in (False, True):
            _check(lib, x, table, buckets, mask, causal, 0.5, f"{Tk} causal {causal}")


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("Tk", [8192, 16384, 20000])
def test_long_rows_that_see_only_hidden_keys(lib, dt, Tk):
    x, table, buckets = _inputs(lib, (2, 2, 3, Tk), DT[dt])
    for fill in (-1e9, -1e10, -1e20):
        mask = torch.full((2, Tk), fill, device=DEV, dtype=DT[dt])
        mask[1, Tk // 3:] = 0
        _check(lib, x, table, buckets, mask, False, 0.5, f"{Tk} {fill}")


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("power", [16, 20, 24, 31, 33, 50, 90])
def test_rows_of_large_scores(lib, dt, power):
    """Scores around 2^power, some of a row's at its maximum."""
    dtype = DT[dt]
    for Tk in (40, 77, 600):
        shape = (2, 2, 9, Tk)
        _, table, buckets = _inputs(lib, shape, dtype)
        table = torch.zeros_like(table)
        whole = torch.randint(-8, 9, shape, device=DEV,
                              generator=torch.Generator(device=DEV).manual_seed(power))
        scale = 2.0 ** (power - 3)
        if dtype == torch.float16:
            _check(lib, whole.to(dtype), table, buckets, None, False, scale, f"{Tk} by the scale")
        else:
            x = (whole.double() * scale).to(dtype)
            _check(lib, x, table, buckets, None, False, 1.0, f"{Tk}")
            _check(lib, -x.abs() - x.abs().max(), table, buckets, None, True, 1.0, f"{Tk} negative")

def _mask(kind, B, Tk, dtype, seed):
    if kind == "none":
        return None
    g = torch.Generator().manual_seed(seed)
    low = torch.finfo(dtype).min
    n = torch.randint(1, Tk + 1, (B,), generator=g)
    n[0], n[1] = 0, Tk
    m = torch.zeros(B, Tk)
    for b in range(B):
        m[b, int(n[b]):] = low if kind in ("lowest", "mixed") else -INF
    if kind in ("holes", "mixed"):
        m = torch.where(torch.rand(B, Tk, generator=g) < 0.3, torch.tensor(-INF), m)
    if kind == "mixed":
        m = (m + S.grid(torch.randn(B, Tk, generator=g), 2.0 ** -4)).clamp(min=low) + \
            torch.where(m.isneginf(), m, torch.zeros(()))
    return m.to(dtype).to(DEV)


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("kind", ["none", "pad", "holes", "lowest", "mixed"])
@pytest.mark.parametrize("shape", [(3, 2, 40, 40), (3, 5, 17, 264), (3, 3, 77, 203), (3, 2, 1, 1001),
                                   (3, 2, 3, 2049)])
def test_masks_within_a_bound_that_binds(lib, dt, kind, shape):
    x, table, buckets = _inputs(lib, shape, DT[dt], seed=7)
    mask = _mask(kind, shape[0], shape[3], DT[dt], 11)
    for causal in (False, True):
        for scale in (0.5, 1.0):
            _check(lib, x, table, buckets, mask, causal, scale, f"{kind} causal {causal}")
