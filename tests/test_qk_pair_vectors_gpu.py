"""The per-head norm with rotation at 66 to 128 features that are no whole
vectors of four elements, where forward and backward take different kernels."""
import pytest
import torch

import _position_ref as R

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


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("D,rot,shift", [(66, 64, 0), (70, 36, 0), (90, 88, 0), (98, 0, 0),
                                         (100, 96, 2), (126, 124, 0), (128, 128, 2)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_heads_of_element_pairs(lib, dt, D, rot, shift, interleaved):
    L, dtype = lib, DT[dt]
    T, Hq, Hk = 61, 5, 2
    g = torch.Generator(device=DEV).manual_seed(D)
    width = (Hq + Hk) * D + 6

    def packed(std):
        buf = (torch.randn(T * width + shift, generator=g, device=DEV) * std).to(dtype)
        rows = buf[shift:].view(T, width)
        return (rows[:, :Hq * D].view(T, Hq, D),
                rows[:, Hq * D:(Hq + Hk) * D].view(T, Hk, D))

    x, d = packed(1.5), packed(1.0)
    gamma = [(1 + 0.3 * torch.randn(D, generator=g, device=DEV)).to(dtype) for _ in range(2)]
    cos = sin = pos = None
    if rot:
        cos, sin = L.rope_tables(40, rot, device=DEV)
        pos = torch.randint(0, 40, (T,), generator=g, device=DEV, dtype=torch.int32)
    out = L.qk_norm_rope_fw(*x, *gamma, cos, sin, pos, interleaved=interleaved)
    got = L.qk_norm_rope_bw(*d, *x, *gamma, out[2], out[3], cos, sin, pos,
                            interleaved=interleaved)
    for i in range(2):
        (wy, ty), (wr, tr) = R.qk_fw(x[i], gamma[i], cos, sin, pos, interleaved, 1e-6)
        R.check(out[i], wy, ty, "y")
        R.check(out[2 + i], wr, tr, "rstd")
        (wx, tx), (wg, tg) = R.qk_bw(d[i], x[i], gamma[i], out[2 + i], cos, sin, pos, interleaved)
        R.check(got[i], wx, tx, "dx")
        R.check(got[2 + i], wg, tg, "dgamma")
