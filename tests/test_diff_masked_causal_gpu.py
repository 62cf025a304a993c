"""The difference of two softmax maps under a causal mask and a padding mask, for few
and many batch entries of short and long heads: rows dealt over the grid and rows
in runs, windows of the masks kept and too many of them to keep."""
import pytest
import torch

import _decoder_ref as R

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
@pytest.mark.parametrize("shape", [(64, 1, 16, 200), (2, 3, 700, 700), (1, 2, 1030, 1030),
                                   (70, 2, 40, 41), (65, 1, 90, 96), (8, 2, 500, 520),
                                   (300, 1, 5, 33), (3, 1, 2, 64)])
@pytest.mark.parametrize("holes", [False, True])
def test_padded_causal_maps(lib, dt, shape, holes):
    B, H, Tq, Tk = shape
    gen = torch.Generator(device=DEV).manual_seed(B + Tk)
    s = (torch.randn((B, 2 * H, Tq, Tk), generator=gen, device=DEV) * 2).to(DT[dt])
    x1, x2 = s[:, :H], s[:, H:]
    lam = torch.rand(H, generator=gen, device=DEV)
    dout = torch.randn((B, H, Tq, Tk), generator=gen, device=DEV).to(DT[dt])
    n = torch.randint(0, Tk + 1, (B,), generator=gen, device=DEV)  # 0: nothing is left
    hidden = torch.arange(Tk, device=DEV)[None, :] >= n[:, None]
    if holes:
        hidden = hidden | (torch.rand(B, Tk, generator=gen, device=DEV) < 0.2)
    mask = torch.zeros(B, Tk, device=DEV).masked_fill_(hidden, -torch.inf).to(DT[dt])
    (y, ytol), (st, stol) = R.diff_fw(x1, x2, lam, mask, True, 0.7)
    got, stats = lib.softmax_fw_diff(x1, x2, lam, mask, causal=True, scale=0.7)
    R.check(got, y, ytol, "fw")
    R.check(stats, st, stol, "stats")
    given = st.float().contiguous()
    a, b, l = R.diff_bw(dout, x1, x2, lam, given, mask, True, 0.7)
    d1, d2, dl = lib.softmax_bw_diff(dout, x1, x2, lam, given, mask, causal=True, scale=0.7)
    R.check(d1, *a, "dx1")
    R.check(d2, *b, "dx2")
    R.check(dl, *l, "dlam")
