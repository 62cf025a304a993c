"""The workspace sizes of the cross entropy from hidden states are what
ls_reduce.h says that they hold."""
import pytest

CODES = {"f32": 0, "f16": 1, "bf16": 2}
SIZES = [(1, 1, 1), (1, 4096, 128256), (5, 24, 300), (33, 768, 32000), (257, 100, 777),
         (1001, 333, 10007), (8192, 1024, 50257), (2049, 40, 300), (10000, 250, 50257),
         (65536, 4096, 131072), (1 << 20, 64, 32000)]


@pytest.fixture(scope="module")
def abi():
    from transformer_reduce_gb300 import build as b
    b.build()
    from transformer_reduce_gb300 import _lib
    _lib.load()
    assert (_lib.LS_F32, _lib.LS_F16, _lib.LS_BF16) == (0, 1, 2)
    return _lib


def _up(v, to):
    return -(-v // to) * to


def _common(rows, hidden, vocab, dt):
    R, D = _up(rows, 256), _up(hidden, 8)
    es = 6 if dt == "f32" else 2
    copies = es * R * D
    if dt == "f32" or hidden % 8:
        copies += es * vocab * D
    return R, D, es, copies


SLACK = 12 * 256  # every array starts at a multiple of 256 bytes


@pytest.mark.parametrize("dt", list(CODES))
@pytest.mark.parametrize("sizes", SIZES)
def test_forward_size(abi, dt, sizes):
    rows, hidden, vocab = sizes
    R, _, _, copies = _common(*sizes, dt)
    least = copies + 16 * R * (_up(vocab, 256) // 256)
    got = abi.ls_linear_cross_entropy_fw_workspace_size(rows, hidden, vocab, CODES[dt])
    assert least <= got <= least + 16 * R + SLACK


@pytest.mark.parametrize("dt", list(CODES))
@pytest.mark.parametrize("sizes", SIZES)
def test_backward_size(abi, dt, sizes):
    rows, hidden, vocab = sizes
    R, D, es, copies = _common(*sizes, dt)
    got = abi.ls_linear_cross_entropy_bw_workspace_size(rows, hidden, vocab, CODES[dt])
    rest = got - copies
    whole = es * R * _up(vocab, 256)
    piece = min(whole, max(512 << 20, es * R * 4096))
    assert rest <= piece + 32 * 4 * R * D + 16 * R + SLACK
    if whole <= 512 << 20:  # one piece: its gradients, and sums of some number of cuts
        sums = rest - whole
        cuts = sums // (4 * R * D)
        assert cuts <= 32 and cuts != 1
        assert 0 <= sums - cuts * 4 * R * D <= 16 * R + SLACK
    else:
        assert rest >= piece // 2 + 4 * R * D
