"""Long sums of one sign in the cross entropy from hidden states: over the rows in
dW, over the hidden elements in the logits.  The tensor cores cut their
accumulator off where a step of 16 is added, at most 2 u of the sum (u = 2^-24);
of 16-bit operands 64 steps of 64 elements (logits: 16) are summed that way, 256
(64) cut-offs, and FP32 additions rounded to nearest join the parts, u each."""
import math

import pytest
import torch

import _decoder_ref as R

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
U = R.U


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from transformer_reduce_gb300 import build
    build.build()
    import transformer_reduce_gb300 as L
    L.load()
    return L


def _positive(shape, dtype, seed, scale=1.0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return ((torch.rand(shape, generator=g, device=DEV) + 0.5) * scale).to(dtype)


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("rows", [4096, 4097, 65536, 1 << 18, (1 << 20) + 5])
def test_gradient_of_the_vocabulary_over_many_rows(lib, dt, rows):
    """Equal logits: every weight is 1 / 32, which the 16-bit types hold exactly, as they
    do 1 / 32 - 1; what is off is the sum over the rows and the output's rounding."""
    D, V = 8, 32
    x = _positive((rows, D), DT[dt], rows)
    w = torch.zeros(V, D, dtype=DT[dt], device=DEV)
    t = torch.zeros(rows, dtype=torch.int32, device=DEV)
    lse = torch.full((rows,), math.log(V), device=DEV)
    up = torch.full((rows,), 1.0, device=DEV) / rows
    dx, dw = lib.linear_cross_entropy_bw(x, w, t, lse, up)
    total = (x.double() * up.double()[:, None]).sum(0)
    want = (torch.full((V, 1), 1 / V, dtype=torch.float64, device=DEV) -
            (torch.arange(V, device=DEV) == 0).double()[:, None]) * total
    tol = want.abs() * (R.half_step(DT[dt]) + U * (2 * 256 + rows / 4096 + 40)) + R.tiny(DT[dt])
    R.check(dw, want, tol, f"dw {rows}")
    assert not dx.any()


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("D", [1024, 1025, 4096, 16384, 65536])
def test_logits_over_many_hidden_elements(lib, dt, D):
    x, w = _positive((70, D), DT[dt], D), _positive((300, D), DT[dt], D + 1, 20 / D)
    t = torch.arange(70, device=DEV, dtype=torch.int32)
    loss, lse = lib.linear_cross_entropy_fw(x, w, t)
    z = x.double() @ w.double().T
    want = torch.logsumexp(z, -1)
    top = z.amax(-1)
    # the logit's sum; the exponent's product and difference, the parts' joins
    tol = U * (2 * 64 + D / 1024 + 8) * top + U * (60 + 12 * top)
    R.check(lse, want, tol, f"lse {D}")
    R.check(loss, want - z[torch.arange(70), t.long()], 2 * tol, f"loss {D}")


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("rows,D,V", [(33, 1025, 300), (300, 2049, 515), (17, 65536, 40),
                                      (5, 3001, 1000), (4200, 1100, 270)])
def test_hidden_sizes_of_several_parts(lib, dt, rows, D, V):
    dtype = DT[dt]
    g = torch.Generator(device=DEV).manual_seed(D)
    x = torch.randn((rows, D), generator=g, device=DEV).to(dtype)
    w = (torch.randn((V, D), generator=g, device=DEV) * 2.5 / D ** 0.5).to(dtype)
    t = torch.randint(-V // 3, V, (rows,), generator=g, device=DEV).to(torch.int32)
    (loss, ltol), (lse, stol) = R.loss_fw(x, w, t)
    got = lib.linear_cross_entropy_fw(x, w, t)
    R.check(got[0], loss, ltol, "loss")
    R.check(got[1], lse, stol, "lse")
    up = torch.rand(rows, generator=g, device=DEV) / rows
    a, b = R.loss_bw(x, w, t, lse.float(), up)
    dx, dw = lib.linear_cross_entropy_bw(x, w, t, lse.float(), up)
    R.check(dx, *a, "dx")
    R.check(dw, *b, "dw")
