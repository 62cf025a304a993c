"""fp32 gradients of the cross entropy from hidden states where nearly all of a
row's weight lies on its target: q = p - 1 cancels and carries the absolute error
of the logit.

A plain FP32 sum of 1024 products rounds to nearest at each: about sqrt(1024) / 2
= 16 steps u = 2^-24 of a typical partial sum.  The kernel's sixteen parts of 64
elements are cut off four times each at full size, by u in the mean and to one
side: 4 u of a part, whose signs vary, 4 sqrt(16) = 16 u.  So both are equally
far from 64 bits; a factor of two is left for the exponential (4 u) and for the
order of the plain form's sums."""
import math

import pytest
import torch

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


def _far(got, want):
    return max(float((a.double() - b).norm() / b.norm()) for a, b in zip(got, want))


@pytest.mark.parametrize("rows,D,V,gain", [(14, 1024, 65, 6.0), (14, 1024, 65, 14.0),
                                           (200, 512, 65, 14.0), (64, 2048, 300, 16.0)])
def test_as_near_to_64_bits_as_a_plain_form(lib, rows, D, V, gain):
    assert not torch.backends.cuda.matmul.allow_tf32
    own, plain = [], []
    for seed in range(16):
        g = torch.Generator(device=DEV).manual_seed(seed)
        std = 2.5 / math.sqrt(D)
        w = torch.randn(V, D, device=DEV, generator=g) * std
        t = torch.randint(0, V, (rows,), device=DEV, generator=g)
        x = torch.randn(rows, D, device=DEV, generator=g) + w[t] * (gain / (std * std * D))
        up = torch.full((rows,), 1 / rows, device=DEV)
        lse = torch.logsumexp(x.double() @ w.double().T, -1).float()

        def grads(dt):
            q = torch.exp(x.to(dt) @ w.to(dt).T - lse.to(dt)[:, None])
            q[torch.arange(rows), t] -= 1
            q = q * up.to(dt)[:, None]
            return q @ w.to(dt), q.T @ x.to(dt)

        want = grads(torch.float64)
        plain.append(_far(grads(torch.float32), want))
        own.append(_far(lib.linear_cross_entropy_bw(x, w, t.to(torch.int32), lse, up), want))
    own.sort()
    plain.sort()
    assert own[8] <= 2 * plain[8], (own, plain)
    assert own[-1] <= 3 * plain[-1], (own, plain)
