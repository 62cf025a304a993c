"""Clipping with outputs that share memory: refused through the PyTorch layer,
with nothing written; neighbours, in-place lists and gradients given twice are
not overlaps."""
import pytest
import torch

import _position_ref as R

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from transformer_reduce_gb300 import build
    build.build()
    import transformer_reduce_gb300 as L
    L.load()
    return L


@pytest.mark.parametrize("count", [2, 700])
def test_overlaps_are_refused_and_nothing_is_written(lib, count):
    L = lib
    g = torch.Generator(device=DEV).manual_seed(1)
    buf = torch.randn(count * 100 + 50, generator=g, device=DEV)
    parts = list(buf[:count * 100].split(100))
    keep = buf.clone()
    with pytest.raises(ValueError, match="overlaps"):
        L.grad_clip(parts, 1.0, out=parts[::-1])
    with pytest.raises(ValueError, match="overlaps"):
        L.grad_clip(parts, 1.0, out=[buf[100 * i + 1:100 * i + 101] for i in range(count)])
    with pytest.raises(ValueError, match="overlaps"):
        L.grad_clip([buf[99 * i:99 * i + 100] for i in range(count)], 1.0)
    with pytest.raises(ValueError, match="overlaps"):
        L.grad_clip([parts[0], parts[0]], 1.0, out=[parts[0], parts[1]])
    torch.cuda.synchronize()
    assert torch.equal(buf, keep)


@pytest.mark.parametrize("count", [3, 150, 700, 1300])
def test_what_does_not_overlap_is_clipped(lib, count):
    L = lib
    g = torch.Generator(device=DEV).manual_seed(2)
    buf = torch.randn(count * 7, generator=g, device=DEV, dtype=torch.bfloat16)
    parts = list(buf.split(7))
    order = torch.randperm(count, generator=torch.Generator().manual_seed(3)).tolist()
    mixed = [parts[i] for i in order]
    # elsewhere, the first gradient given twice; then half of the list in place
    twice = mixed + mixed[:1]
    to = torch.empty(len(twice) * 7, device=DEV, dtype=torch.bfloat16).split(7)
    (wn, tn), want = R.clip(twice, 2.0, 1e-6)
    out, norm = L.grad_clip(twice, 2.0, out=list(to))
    R.check(norm, wn, tn, "norm")
    for o, (w, t) in zip(out, want):
        R.check(o, w, t, "elsewhere")
    (wn, tn), want = R.clip(mixed, 2.0, 1e-6)
    half = [m if i % 2 else to[i] for i, m in enumerate(mixed)]
    out, norm = L.grad_clip(mixed, 2.0, out=half)
    R.check(norm, wn, tn, "norm")
    for o, (w, t) in zip(out, want):
        R.check(o, w, t, "half in place")
