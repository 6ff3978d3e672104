"""Trees of drafted tokens and the norm + rotation call, host side: paths and
depths, and the argument checks that answer before any CUDA call."""
import ctypes
import random

import pytest

import fp4_kv_cache_index_gb300 as C

L = C.lib


def paths(parent):
    n = len(parent)
    d, m = (ctypes.c_int32 * 64)(), (ctypes.c_uint64 * 64)()
    st = L.csa2_tree_paths(n, (ctypes.c_int32 * max(1, n))(*parent), d, m)
    return st, list(d[:n]), list(m[:n])


@pytest.mark.parametrize("n", [1, 2, 7, 33, 64])
def test_paths_follow_the_parents(n):
    for seed in range(20):
        r = random.Random(100 * n + seed)
        parent = [r.randrange(-1, t) for t in range(n)]
        if seed == 0:
            parent = list(range(-1, n - 1))       # a chain: depth n - 1, every bit
        if seed == 1:
            parent = [-1] * n                     # siblings only
        st, d, m = paths(parent)
        assert st == 0
        for t in range(n):
            want, a = [], t
            while a >= 0:
                want.append(a)
                a = parent[a]
            assert d[t] == len(want) - 1
            assert m[t] == sum(1 << a for a in want)


def test_paths_refuse_what_is_no_tree():
    assert paths([])[0] == 0
    assert paths([0])[0] == 1            # its own parent
    assert paths([-1, 1])[0] == 1
    assert paths([-1, 2, 0])[0] == 1     # a parent behind its child
    assert paths([-2])[0] == 1
    assert L.csa2_tree_paths(65, (ctypes.c_int32 * 65)(*[-1] * 65), None, None) == 2
    assert L.csa2_tree_paths(-1, None, None, None) == 1
    assert L.csa2_tree_paths(3, None, None, None) == 1
    assert L.csa2_tree_paths(1, (ctypes.c_int32 * 1)(-1), None, None) == 0


def test_tree_object():
    t = C.Tree([[-1, 0, 0, 2], [], [-1]], [10, 4, 7], seq_ids=[2, 0, 5])
    assert t.n_queries == 5 and t.n_draft == [4, 0, 1]
    assert t.depths == [[0, 1, 1, 2], [], [0]]
    assert t.paths == [[1, 3, 5, 13], [], [1]]
    assert t.positions("cpu").tolist() == [10, 11, 11, 12, 7]
    assert t.owners(1) == [[0, 1, 2, 3], [], [0]]
    assert t.owners(2) == [[1, 2], [], [0]]       # positions 11 and 7 complete a block of two
    assert t.owners(3) == [[1, 2], [], []]
    with pytest.raises(C.Csa2Error):
        C.Tree([[0]], [1])
    with pytest.raises(C.Csa2Error):
        C.Tree([[-1] * 65], [1])
    with pytest.raises(ValueError):
        C.Tree([[-1]], [1, 2])
    with pytest.raises(ValueError):
        C.Tree([[-1]], [1], seq_ids=[0, 1])


def test_tree_calls_refuse_a_null_cache_and_a_null_tree():
    t = C.Tree([[-1]], [4])
    one = (ctypes.c_int32 * 1)(0)
    for ref in (t.ref, None):
        assert L.csa2_index_scores_tree(None, ref, None, None, None, 4, None, None) == 1
        assert L.csa2_index_topk_tree(None, ref, None, None, None, None, None, 0, None) == 1
        assert L.csa2_sparse_attn_tree(None, ref, 1, None, None, None, 1.0, 0, 0.0, None, 0,
                                       None) == 1
        assert L.csa2_cache_accept_tree(None, ref, one, None) == 1


GOOD = dict(x=0x10000, out=0x20000, weight=None, pos=0x30000, n_tokens=3, x_token_stride=512,
            x_head_stride=512, out_token_stride=512, out_head_stride=512, n_heads=1, dim=512,
            rope_dim=64, norm=1, x_fp32=0, out_fp32=0)


def part(**kw):
    return C.NormPart(**{**GOOD, **kw})


@pytest.mark.parametrize("kw, status", [
    (dict(n_tokens=-1), 1), (dict(n_heads=0), 1), (dict(dim=96), 2), (dict(dim=1024), 2),
    (dict(rope_dim=-8), 1), (dict(rope_dim=12), 1), (dict(rope_dim=576), 1), (dict(rope_dim=256), 2),
    (dict(dim=64, rope_dim=128), 1), (dict(x=None), 1), (dict(out=None), 1), (dict(pos=None), 1),
    (dict(pos=0x30004), 1), (dict(x=0x10008), 1), (dict(out=0x20004), 1), (dict(weight=0x40004), 1),
    (dict(x_token_stride=516), 1), (dict(n_heads=2, x_head_stride=4), 1),
    (dict(out_token_stride=1), 1), (dict(n_heads=2, out_fp32=1, out_head_stride=2), 1), (dict(x_fp32=2), 1), (dict(out_fp32=-1), 1),
    (dict(n_tokens=0, x=None, out=None), 0),
])
def test_norm_rope_argument_checks(kw, status):
    """Every refusal (and a part without tokens) answers before any launch."""
    assert L.csa2_norm_rope(1, ctypes.byref(part(**kw)), 1e-6, 0.0, None) == status


def test_norm_rope_scalar_checks():
    a = part()
    nan, inf = float("nan"), float("inf")
    for eps in (0.0, -1e-6, 1e-31, nan, inf):
        assert L.csa2_norm_rope(1, ctypes.byref(a), eps, 0.0, None) == 1
    for base in (-1.0, nan, inf):
        assert L.csa2_norm_rope(1, ctypes.byref(a), 1e-6, base, None) == 1
    assert L.csa2_norm_rope(-1, ctypes.byref(a), 1e-6, 0.0, None) == 1
    assert L.csa2_norm_rope(9, ctypes.byref(a), 1e-6, 0.0, None) == 1
    assert L.csa2_norm_rope(1, None, 1e-6, 0.0, None) == 1
    assert L.csa2_norm_rope(0, None, 1e-6, 0.0, None) == 0


@pytest.mark.parametrize("kw, status", [
    (dict(out_token_stride=0), 1), (dict(out_token_stride=256), 1), (dict(out_token_stride=-256), 1),
    (dict(n_heads=2, n_tokens=1, out_head_stride=0), 1), (dict(n_heads=2), 1),
    (dict(n_tokens=(1 << 31) + 1), 2), (dict(n_tokens=1 << 62, n_heads=4, out_head_stride=1024), 2),
    (dict(n_tokens=1 << 24, n_heads=129, out_token_stride=1 << 17), 2),
])
def test_norm_rope_refuses_heads_over_each_other_and_endless_tensors(kw, status):
    assert L.csa2_norm_rope(1, ctypes.byref(part(**kw)), 1e-6, 0.0, None) == status


def test_norm_rope_refuses_an_eps_or_a_base_outside_the_formula_s_range():
    """An eps above 1 would count beside squares beyond fp32; a base below 1
    turns a channel by more than a turn per position."""
    a = part()
    for eps in (1.5, 1e30, 3.4e38):
        assert L.csa2_norm_rope(1, ctypes.byref(a), eps, 0.0, None) == 1
    for base in (1e-300, 0.5, 0.999):
        assert L.csa2_norm_rope(1, ctypes.byref(a), 1e-6, base, None) == 1
