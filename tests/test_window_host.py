"""What the window and verification calls refuse before anything is launched,
and what is nothing to do (no GPU needed: the pointers are never followed)."""
import ctypes

import pytest

P = 1 << 20      # an aligned address
I32 = ctypes.c_int32


@pytest.fixture(scope="module")
def C():
    import os
    import __graft_entry__
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    if not os.path.exists(os.path.join(root, "fp4_kv_cache_index_gb300", "libcsa2.so")):
        __graft_entry__.build()
    import fp4_kv_cache_index_gb300 as c
    return c


INVALID, UNSUPPORTED = 1, 2


def window(C, **kw):
    f = dict(n_seqs=4, swa=128, n_first=4, fp8=1, rows=None, codes=P, rope=P, scales=P, pos=P, error=P)
    f.update(kw)
    w = C.WindowStruct(**f)
    return w, ctypes.byref(w)


def ints(xs):
    return None if xs is None else (I32 * max(1, len(xs)))(*xs)


@pytest.mark.parametrize("change,status", [
    (dict(swa=0), INVALID), (dict(swa=129), UNSUPPORTED), (dict(n_first=-1), INVALID),
    (dict(n_first=9), UNSUPPORTED), (dict(n_seqs=-1), INVALID), (dict(fp8=2), INVALID),
    (dict(codes=None), INVALID), (dict(rope=P + 8), INVALID), (dict(scales=P + 4), INVALID),
    (dict(pos=None), INVALID), (dict(pos=P + 8), INVALID), (dict(fp8=0), INVALID),
    (dict(fp8=0, rows=P + 2), INVALID), (dict(error=P + 1), INVALID),
    (dict(n_seqs=2 ** 24), UNSUPPORTED)])
def test_caches(C, change, status):
    w, ref = window(C, **change)
    assert C.lib.csa2_window_reset(ref, -1, None) == status
    assert C.lib.csa2_window_append(ref, 0, None, None, P, P, None, None) == status
    assert C.lib.csa2_window_read(ref, 0, None, P, 1, P, None, None, None, None, None) == status
    assert C.lib.csa2_window_attn_decode(ref, 64, 0, None, P, P, 1.0, P, None, None) == status
    t = C.Tree([], [])
    assert C.lib.csa2_window_attn_tree(ref, t.ref, 64, P, P, None, None, None, 1.0, P, None, None) == status
    assert C.lib.csa2_window_accept_tree(ref, t.ref, P, P, None, None, None, None) == status


def test_segments(C):
    w, ref = window(C)
    f = C.lib.csa2_window_append

    def call(n, seqs=None, counts=None, pos=P, rows=P, rounded=None):
        return f(ref, n, ints(seqs), ints(counts), pos, rows, rounded, None)
    assert call(0) == 0 and call(4, counts=[0, 0, 0, 0], pos=None, rows=None) == 0
    for bad in (dict(n=-1), dict(n=5), dict(n=2, seqs=[1, 1]), dict(n=2, seqs=[0, 4]),
                dict(n=1, seqs=[-1]), dict(n=5, seqs=[0, 1, 2, 3, 0]), dict(n=2, counts=[1, -1]),
                dict(n=1, pos=None), dict(n=1, pos=P + 4), dict(n=1, rows=None),
                dict(n=1, rows=P + 8), dict(n=1, rounded=P + 8)):
        assert call(**bad) == INVALID, bad
    assert call(2, counts=[2 ** 31 - 1, 2]) == UNSUPPORTED
    g = C.lib.csa2_window_read

    def read(n=1, seqs=None, end=P, rows=128, out=P, fp8=(None, None, None), first=None):
        return g(ref, n, ints(seqs), end, rows, out, *fp8, first, None)
    assert read(n=0) == 0
    for bad in (dict(n=-1), dict(n=5), dict(seqs=[4]), dict(rows=0), dict(rows=129), dict(out=None),
                dict(out=P + 8), dict(fp8=(P, P, P)), dict(out=None, fp8=(P, P, None)),
                dict(out=None, fp8=(P, P, P + 4)), dict(end=None), dict(end=P + 4), dict(first=P + 8)):
        assert read(**bad) == INVALID, bad
    w16, ref16 = window(C, fp8=0, rows=P)
    assert g(ref16, 1, None, P, 8, None, P, P, P, None, None) == INVALID
    assert C.lib.csa2_window_reset(ref, 4, None) == INVALID
    assert C.lib.csa2_window_reset(ref, -2, None) == INVALID
    st = I32()
    assert C.lib.csa2_window_device_error(None, None, ctypes.byref(st)) == INVALID
    w0, ref0 = window(C, error=None)
    assert C.lib.csa2_window_device_error(ref0, None, ctypes.byref(st)) == INVALID


def test_attention(C):
    w, ref = window(C)
    f = C.lib.csa2_window_attn_decode
    opts = C.WindowOpts(None, None, 1, 0.5, None)

    def call(heads=64, n=2, seqs=None, q=P, pos=P, scale=1.0, out=2 * P, o=None):
        return f(ref, heads, n, ints(seqs), q, pos, scale, out, o, None)
    assert call(n=0, q=None, pos=None, out=None) == 0
    for bad in (dict(n=-1), dict(n=5), dict(seqs=[0, 4]), dict(q=None), dict(q=P + 8), dict(out=None),
                dict(out=P), dict(pos=None), dict(pos=P + 4), dict(scale=float("nan")),
                dict(scale=float("inf")), dict(o=ctypes.byref(opts)),
                dict(o=ctypes.byref(C.WindowOpts(P + 8, None, 0, 0.0, None))),
                dict(o=ctypes.byref(C.WindowOpts(None, P + 8, 0, 0.0, None))),
                dict(o=ctypes.byref(C.WindowOpts(None, None, 2, 0.0, None)))):
        assert call(**bad) == INVALID, bad
    for heads in (0, 32, 96, 256):
        assert call(heads=heads) == UNSUPPORTED
    g = C.lib.csa2_window_attn_prefill

    def chunk(heads=64, n=2, pos0=10, q=P, rows=P, band0=8, n_rows=4, swa=128, first=P, n_first=2,
              scale=1.0, out=2 * P, o=None):
        return g(heads, n, pos0, q, rows, band0, n_rows, swa, first, n_first, scale, out, o, None)
    assert chunk(n=0, q=None, rows=None, out=None) == 0
    for bad in (dict(n=-1), dict(pos0=-1, band0=0), dict(pos0=7), dict(band0=-1), dict(n_rows=3),
                dict(n_rows=-1), dict(swa=0), dict(n_first=-1), dict(first=None), dict(first=P + 8),
                dict(q=None), dict(rows=None), dict(rows=P + 8), dict(out=None), dict(out=P),
                dict(pos0=2 ** 63 - 2, band0=2 ** 63 - 2), dict(o=ctypes.byref(opts))):
        assert chunk(**bad) == INVALID, bad
    for bad in (dict(swa=129), dict(n_first=9), dict(heads=16)):
        assert chunk(**bad) == UNSUPPORTED, bad


def test_trees(C):
    w, ref = window(C)

    def tree(n_draft, pos0, parent, seqs=None):
        keep = (ints(seqs), ints(n_draft), (ctypes.c_int64 * max(1, len(pos0)))(*pos0), ints(parent))
        at = [None if k is None else ctypes.addressof(k) for k in keep]
        t = C.TreeStruct(len(n_draft), *at)
        t.keep = keep
        return t
    good = tree([2, 1], [5, 0], [-1, 0, -1])
    q = dict(codes=P, rope=P, scales=P, kv=None)

    def attn(t, **kw):
        a = dict(q, **kw)
        return C.lib.csa2_window_attn_tree(ref, ctypes.byref(t), 64, a.get("q", P), a["kv"], a["codes"],
                                           a["rope"], a["scales"], 1.0, a.get("out", 2 * P), None, None)

    def accept(t, accepted=P, **kw):
        a = dict(q, **kw)
        return C.lib.csa2_window_accept_tree(ref, ctypes.byref(t), accepted, a["kv"], a["codes"],
                                             a["rope"], a["scales"], None)
    for t, status in ((tree([2], [5], [0, 0]), INVALID), (tree([2], [5], [-1, 1]), INVALID),
                      (tree([2], [-1], [-1, 0]), INVALID), (tree([-1], [5], []), INVALID),
                      (tree([65], [5], [-1] * 65), UNSUPPORTED),
                      (tree([1, 1], [5, 5], [-1, -1], [2, 2]), INVALID),
                      (tree([1], [5], [-1], [4]), INVALID),
                      (tree([1] * 5, [5] * 5, [-1] * 5), INVALID)):
        assert attn(t) == status and accept(t) == status
    assert attn(tree([0, 0], [5, 5], []), codes=None, q=None) == 0
    for bad in (dict(codes=None), dict(rope=P + 8), dict(scales=P + 4)):
        assert attn(good, **bad) == INVALID and accept(good, **bad) == INVALID
    assert attn(good, q=None) == INVALID and attn(good, out=P) == INVALID
    assert accept(good, accepted=None) == INVALID and accept(good, accepted=P + 2) == INVALID


def test_verification(C):
    t = C.Tree([[-1, 0], [-1]], [0, 0])

    def call(tree=t, **kw):
        f = dict(vocab=100, fp32=0, token=P, target=P, target_root=P, draft=P, draft_root=P, ld=100,
                 temperature=P, uniform=P, noise=P, noise_ld=100, accepted=P, next_token=P)
        f.update(kw)
        v = C.VerifyStruct(**f)
        return C.lib.csa2_verify_tree(tree.ref, ctypes.byref(v), None)
    assert call(tree=C.Tree([], []), token=None, target=None) == 0
    for bad in (dict(vocab=0), dict(vocab=-1), dict(ld=99), dict(fp32=2), dict(token=None),
                dict(target=None), dict(target=P + 1), dict(fp32=1, target=P + 2), dict(token=P + 2),
                dict(accepted=None), dict(next_token=None), dict(uniform=None), dict(noise=None),
                dict(noise_ld=99), dict(draft=None), dict(draft_root=None), dict(target_root=None),
                dict(tree=C.Tree([[-1, -1], [-1]], [0, 0]), target_root=None, draft_root=None)):
        assert call(**bad) == INVALID, bad
    assert C.lib.csa2_verify_tree(t.ref, None, None) == INVALID
    assert C.lib.csa2_verify_tree(None, None, None) == INVALID


@pytest.mark.parametrize("rows", [1, 100])
def test_rounded_rows_lie_on_the_rows_or_apart(C, rows):
    """Nothing is launched: a sequence's count of rows makes the call's."""
    w, ref = window(C)
    for off in (16, rows * 1024 - 16, -16, 16 - rows * 1024):
        assert C.lib.csa2_window_append(ref, 1, None, ints([rows]), P, 2 * P, 2 * P + off, None) == INVALID
