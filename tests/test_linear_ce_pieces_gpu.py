"""The backward of the cross entropy from hidden states where the vocabulary is cut
into pieces: with dx cut along each piece as well, with rows off 16-byte
addresses, and with dW of many rows held to one bound over all of them."""
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
    torch.cuda.empty_cache()
    yield L
    torch.cuda.empty_cache()


def _shifted(t, by):
    return torch.empty(t.numel() + 16, dtype=t.dtype, device=DEV)[by:by + t.numel()].view(t.shape)


def _steps(n, dtype):
    """Cut-offs (at most 2 u of the sum each) and additions to nearest (u each) of a sum
    over n: 4096 elements (fp32: 256, six products of planes) between them."""
    if dtype == torch.float32:
        return 2 * 6 * (min(n, 256) / 16 + 1) + n / 256 + 6
    return 2 * (min(n, 4096) / 16 + 1) + n / 4096 + 32  # (and the joins of cuts and pieces)


def _pieces(rows, V, dtype):
    bytes_ = 2 * (3 if dtype == torch.float32 else 1) * -(-rows // 256) * 256
    most = max((512 << 20) // bytes_ // 256 * 256, 4096)
    return -(-V // most)


@pytest.mark.parametrize("dt,rows,D,V,shift", [
    ("bf16", 10000, 256, 50257, 0), ("bf16", 10000, 250, 50257, 0), ("f16", 10000, 256, 50257, 1),
    ("f16", 9000, 77, 50304, 3), ("f32", 10000, 77, 30011, 0), ("f32", 6000, 64, 40000, 1),
    ("bf16", 70000, 24, 9001, 0), ("f16", 70000, 33, 9001, 1)])
def test_pieces(lib, monkeypatch, dt, rows, D, V, shift):
    dtype = DT[dt]
    assert _pieces(rows, V, dtype) > 1
    monkeypatch.setattr(R, "_steps", _steps)
    g = torch.Generator(device=DEV).manual_seed(rows + D)
    x = torch.randn((rows, D), generator=g, device=DEV).to(dtype)
    w = (torch.randn((V, D), generator=g, device=DEV) * 2.5 / D ** 0.5).to(dtype)
    t = torch.randint(-V // 4, V, (rows,), generator=g, device=DEV).to(torch.int32)
    (loss, ltol), (lse, stol) = R.loss_fw(x, w, t)
    got = lib.linear_cross_entropy_fw(x, w, t)
    R.check(got[0], loss, ltol, "loss")
    R.check(got[1], lse, stol, "lse")
    lse = lse.float()
    up = torch.rand(rows, generator=g, device=DEV) / rows
    outs = {"dhidden": _shifted(x, shift), "dweight": _shifted(w, shift)} if shift else {}
    dx, dw = lib.linear_cross_entropy_bw(x, w, t, lse, up, **outs)
    only, _ = lib.linear_cross_entropy_bw(x, w, t, lse, up, weight_grad=False)
    a, b = R.loss_bw(x, w, t, lse, up)
    R.check(dx, *a, "dx")
    R.check(dw, *b, "dw")
    R.check(only, *a, "dx alone")
