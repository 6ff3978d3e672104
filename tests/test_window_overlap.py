"""Outputs of the window layers' attention that lie over what the call reads, or
over each other, are refused before anything is launched (no GPU needed: the
pointers are never followed), and so is an error word off its boundary."""
import ctypes

import pytest

from tests.test_window_host import C, I32, INVALID, P, ints, window  # noqa: F401

ROW = 1024           # a row of 512 bf16


def opts(C, **kw):
    f = dict(sink=None, lse=None, rope_out=0, rope_base=0.0, error=None)
    f.update(kw)
    return ctypes.byref(C.WindowOpts(**f))


def over(at, size, mine):
    """Places for `mine` bytes that touch [at, at + size) at either end, or are in it."""
    return [at + 16, at + size - 16, at - mine + 16]


@pytest.mark.parametrize("heads,n", [(64, 1), (64, 3), (128, 2)])
def test_decode(C, heads, n):
    w, ref = window(C)
    size, q = n * heads * ROW, 64 * P

    def call(out, o=None):
        return C.lib.csa2_window_attn_decode(ref, heads, n, ints([0] * n), q, P, 1.0, out, o, None)
    for out in over(q, size, size):
        assert call(out) == INVALID, out - q
    lse = n * heads * 4
    for at in over(q, size, lse) + over(128 * P, size, lse):
        assert call(128 * P, opts(C, lse=at)) == INVALID, at


@pytest.mark.parametrize("fp8", [0, 1])
def test_trees(C, fp8):
    w, ref = window(C, fp8=fp8, rows=P)
    t = C.Tree([[-1, 0], [-1]], [5, 9])
    q, kv, codes, rope, scales = (k * P for k in (64, 70, 80, 90, 100))
    size = 3 * 64 * ROW

    def call(out, o=None):
        return C.lib.csa2_window_attn_tree(ref, t.ref, 64, q, kv, codes, rope, scales, 1.0, out, o, None)
    inputs = [(q, size)] + ([(codes, 3 * 448), (rope, 3 * 128), (scales, 24)] if fp8 else [(kv, 3 * ROW)])
    for at, n in inputs:
        for out in over(at, n, size):
            assert call(out // 16 * 16) == INVALID, (at, out - at)
        for lse in over(at, n, 3 * 64 * 4):
            assert call(128 * P, opts(C, lse=lse // 16 * 16)) == INVALID, (at, lse - at)


def test_chunks(C):
    q, rows, first, size = 64 * P, 70 * P, 80 * P, 5 * 64 * ROW

    def call(out, o=None):
        return C.lib.csa2_window_attn_prefill(64, 5, 10, q, rows, 8, 7, 128, first, 2, 1.0, out, o, None)
    for at, n in ((q, size), (rows, 7 * ROW), (first, 2 * ROW)):
        for out in over(at, n, size):
            assert call(out) == INVALID, (at, out - at)
        for lse in over(at, n, 5 * 64 * 4):
            assert call(128 * P, opts(C, lse=lse)) == INVALID, (at, lse - at)
    for error in (P + 1, P + 2, P + 3):
        assert call(128 * P, opts(C, error=error)) == INVALID
    for bad in (dict(wait_cycles=-1), dict(withhold=-1)):
        assert call(128 * P, opts(C, **bad)) == INVALID
