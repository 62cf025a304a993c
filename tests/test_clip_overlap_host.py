"""Clipping refuses outputs that overlap one another, or gradients of other
entries: the blocks of the scaling pass run in any order.  Host only."""
import ctypes
import random

import pytest

import transformer_reduce_gb300 as L

FAKE = 0x10000000  # never dereferenced: every call below returns on the host
ES = (4, 2, 2)


@pytest.fixture(scope="module")
def abi():
    from transformer_reduce_gb300 import build as b
    b.build()
    from transformer_reduce_gb300 import _lib
    _lib.load()
    return _lib


def _clip(abi, out, grads, sizes, dts):
    n = len(out)
    p = ctypes.c_void_p * n
    return abi.ls_grad_clip(FAKE, p(*out), p(*grads), (ctypes.c_int64 * n)(*sizes),
                            (ctypes.c_int32 * n)(*dts), n, 1.0, 0.0, FAKE, 1 << 40)


def test_overlapping_outputs_are_refused(abi):
    a, b, c = FAKE, FAKE + 4096, FAKE + 8192
    for out, grads, sizes, dts in (
            ([b, a], [a, b], [10, 10], [0, 0]),              # the gradients in another order
            ([b, c, a], [a, b, c], [5, 5, 5], [1, 1, 1]),
            ([a, b], [a, a], [10, 10], [0, 0]),              # in place beside a reader of it
            ([a, a + 36], [a, a + 36], [10, 10], [0, 0]),    # one element shared, in place
            ([c, c + 18], [a, b], [10, 10], [2, 2]),         # one element shared, elsewhere
            ([a + 4, c], [a, b], [10, 10], [0, 0]),          # its own gradient, shifted
            ([b + 4 * 9, c], [a, b], [10, 10], [0, 0]),      # the next gradient's last element
            ([a, a], [a, b], [10, 10], [0, 0])):
        assert _clip(abi, out, grads, sizes, dts) == abi.LS_ERR_INVALID_ARG
        # whatever their places in a long list
        for front, back in ((600, 0), (0, 1100), (511, 512), (1030, 700)):
            def pad(k, at):
                return [at + 64 * i for i in range(k)]
            f, g = pad(front, 1 << 40), pad(back, 1 << 41)
            assert _clip(abi, f + out + g, f + grads + g, [16] * front + sizes + [16] * back,
                         [0] * front + dts + [0] * back) == abi.LS_ERR_INVALID_ARG
        spread = [0] * len(out)
        for gap in (300, 512, 700):  # the clashing entries far from each other
            o, g, s, d = [], [], [], []
            for i in range(len(out)):
                more = [(1 << 42) + (gap * i + k) * 64 for k in range(gap)]
                o += [out[i]] + more
                g += [grads[i]] + more
                s += [sizes[i]] + [16] * gap
                d += [dts[i]] + spread[:1] * gap
            assert _clip(abi, o, g, s, d) == abi.LS_ERR_INVALID_ARG


def test_python_layer_names_the_overlap():
    def why(out, grads, sizes, es=4):
        return L._overlap(out, grads, [n * es for n in sizes])
    a, b, c = FAKE, FAKE + 4096, FAKE + 8192
    assert why([a, b], [a, b], [10, 10]) is None
    assert why([b, c], [a, a], [10, 10]) is None           # a gradient given twice is only read
    assert why([a, a + 40], [b, b], [10, 10]) is None      # neighbours
    assert why([a, a], [b, b], [0, 10]) is None
    assert why([b, a], [a, b], [10, 10]) == "out[1] overlaps grads[0]"
    assert why([a, a + 36], [a, a + 36], [10, 10]) == "out[1] overlaps out[0]"
    assert why([a + 4], [a], [10]) == "out[0] overlaps grads[0]"
    rng = random.Random(1)
    for _ in range(300):  # against the definition
        n = rng.randint(1, 6)
        sizes = [rng.choice([0, 1, 3, 8]) for _ in range(n)]
        grads = [FAKE + 4 * rng.randint(0, 60) for _ in range(n)]
        out = [g if rng.random() < 0.5 else FAKE + 4 * rng.randint(0, 60) for g in grads]
        bad = False
        for i in range(n):
            for j in range(n):
                if i != j and sizes[i] and sizes[j]:
                    bad |= out[i] < out[j] + 4 * sizes[j] and out[j] < out[i] + 4 * sizes[i]
                if sizes[i] and sizes[j] and not (i == j and out[i] == grads[i]):
                    bad |= out[i] < grads[j] + 4 * sizes[j] and grads[j] < out[i] + 4 * sizes[i]
        assert (why(out, grads, sizes) is not None) == bad
