"""The per-head norm refuses outputs that overlap each other or the other side's
inputs: the two sides run in any order.  Host only."""
import pytest

FAKE = 0x10000000  # never dereferenced: every call below returns on the host


@pytest.fixture(scope="module")
def abi():
    from transformer_reduce_gb300 import build as b
    b.build()
    from transformer_reduce_gb300 import _lib
    _lib.load()
    return _lib


def _fw(abi, q_out, k_out, q, k, Hq=4, Hk=4, tokens=5, strides=(64, 64, 64, 64)):
    g = FAKE + (1 << 30)
    return abi.ls_qk_norm_rope_fw(q_out, k_out, g, g, q, k, g, g, 0, 0, 0, tokens, Hq, Hk, 16, 0,
                                  0, *strides, 0, 1e-6, abi.LS_F32)


def _bw(abi, dq, dk, dq_out, dk_out, q, k, tokens=5, s=64):
    g = FAKE + (1 << 30)
    return abi.ls_qk_norm_rope_bw(dq, dk, g, g, dq_out, dk_out, q, k, g, g, g, g, 0, 0, 0, tokens,
                                  4, 4, 16, 0, 0, s, s, s, s, s, s, 0, g, 1 << 40, abi.LS_F32)


A, B, C, D, E, F = (FAKE + (i << 20) for i in range(6))
ROW = 64 * 4  # bytes of a token's four heads


def test_forward(abi):
    bad = abi.LS_ERR_INVALID_ARG
    assert _fw(abi, A, A, A, A) == bad                    # one tensor for both sides, in place
    assert _fw(abi, A, B, A, A) == bad                    # its keys still read it
    assert _fw(abi, B, A, A, A) == bad
    assert _fw(abi, C, C, A, B) == bad                    # one output for both
    assert _fw(abi, B, A, A, B) == bad                    # exchanged
    assert _fw(abi, A + 4, C, A, B) == bad                # in place, one element on
    assert _fw(abi, A + ROW, C, A, B) == bad              # in place, one token on
    assert _fw(abi, A, C, A, B, strides=(64, 64, 100, 64)) == bad  # other strides
    # packed: a token's keys begin inside its queries
    assert _fw(abi, A, A + ROW - 4, C, D, strides=(128, 128, 64, 64)) == bad
    assert _fw(abi, A + ROW - 4, A, C, D, strides=(128, 128, 64, 64)) == bad
    assert _fw(abi, A, A + ROW - 4, C, D, tokens=1) == bad
    # the keys of each token inside the queries of the next
    assert _fw(abi, A, A + 4 * 128 + 8, C, D, tokens=2, strides=(128, 128, 64, 64)) == bad


def test_backward(abi):
    bad = abi.LS_ERR_INVALID_ARG
    assert _bw(abi, A, A, C, D, E, F) == bad              # one gradient for both
    assert _bw(abi, D, B, C, D, E, F) == bad              # over the other side's upstream
    assert _bw(abi, A, C, C, D, E, F) == bad
    assert _bw(abi, C, D, C, C, E, F) == bad              # one upstream for both, in place
    assert _bw(abi, C + 4, B, C, D, E, F) == bad          # in place, one element on
    assert _bw(abi, F, B, C, D, E, F) == bad              # over the other side's input
    assert _bw(abi, A, E, C, D, E, F) == bad
