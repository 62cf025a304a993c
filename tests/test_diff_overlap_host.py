"""Host-side refusals of the difference of two softmax maps, backward: the workspace
and the weights' gradient may not meet the scores.  No kernel is launched here."""
import pytest

FAKE = 0x10000  # never dereferenced: every call below returns on the host
STEP = 1 << 24
B, H, TQ, TK = 2, 3, 4, 8
HEAD = TQ * TK  # elements


@pytest.fixture(scope="module")
def abi():
    from transformer_reduce_gb300 import build as b
    b.build()
    from transformer_reduce_gb300 import _lib
    _lib.load()
    return _lib


def _at(i):
    return FAKE + i * STEP


def _bw(abi, dlam=_at(3), x1=_at(5), x2=_at(6), ws=_at(9), strides=(H * HEAD, HEAD)):
    dense = (H * HEAD, HEAD)
    return abi.ls_softmax_bw_diff(_at(1), _at(2), dlam, _at(4), x1, x2, _at(7), _at(8), None, B, H,
                                  TQ, TK, *dense, *dense, *strides, *strides, H, 0, 1.0, ws, 1 << 40,
                                  abi.LS_F32)


@pytest.mark.parametrize("maps", [5, 6])
def test_what_is_written_may_not_meet_the_scores(abi, maps):
    bad = abi.LS_ERR_INVALID_ARG
    last = 4 * (B * H * HEAD - 4)  # 16-byte aligned, within the last head
    for at in (_at(maps), _at(maps) + last):
        assert _bw(abi, ws=at) == bad
        assert _bw(abi, dlam=at) == bad
    # slices of one tensor's heads: in the middle of a head of either map
    inter = dict(x1=_at(5), x2=_at(5) + 4 * HEAD, strides=(2 * H * HEAD, 2 * HEAD))
    for at in (_at(5) + 4 * HEAD // 2, _at(5) + 4 * (HEAD + HEAD // 2)):
        assert _bw(abi, ws=at, **inter) == bad
        assert _bw(abi, dlam=at, **inter) == bad
