"""LayerNorm around a block with gammas and a gate but no betas."""
import pytest
import torch

import _decoder_ref as R

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


@pytest.mark.parametrize("rows,D,gates", [(60, 96, 5), (7, 33, 7), (50, 1000, 1)])
def test_norms_around_a_block_without_betas(lib, rows, D, gates):
    """dgate is that of a forward without beta_post."""
    g = torch.Generator(device=DEV).manual_seed(1)

    def rand(*shape, std=1.0, mean=0.0):
        return torch.randn(shape, generator=g, device=DEV) * std + mean

    x, r, dy, dh = (rand(rows, D) for _ in range(4))
    gp, gq, gate = rand(D, std=0.2, mean=1.0), rand(D, std=0.2, mean=1.0), rand(gates, D)
    fw = R.block_fw(x, r, gp, None, gq, None, gate, 1.0, True, 1e-6)
    h, y, st = lib.block_norm_fw(x, r, gamma_pre=gp, gamma_post=gq, gate=gate, kind="layer")
    R.check(h, *fw[0], "h")
    R.check(y, *fw[1], "y")
    given = fw[2][0].float().contiguous()
    want = R.block_bw(dy, dh, x, h, given, gp, gq, None, gate, 1.0, True)
    out = lib.block_norm_bw(dy, dh, x, h, given, gamma_pre=gp, gamma_post=gq, gate=gate,
                            kind="layer")
    for name, v in zip(("dx", "dr", "dg_pre", "db_pre", "dg_post", "db_post", "dgate"), out):
        R.check(v, *want[name], name)
