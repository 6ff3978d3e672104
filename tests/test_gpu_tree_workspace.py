"""The readout of drafts without a workspace of the caller's: what it passes
on as one is memory of the cache's buffer that nothing else uses, not a tensor
of the call."""
import ctypes

import pytest
import torch

from tests.test_gpu_tree import SCALE, Setup, chain, rn, window

pytestmark = pytest.mark.gpu


def test_the_token_workspace_is_the_cache_s_own(monkeypatch):
    import fp4_kv_cache_index_gb300 as C
    st = Setup([chain(3), [-1]], [300, 40])
    idx = C.csa2_index_topk_tree(st.cache, st.tree, st.q_idx, st.w)
    wd, q = window(st, 5), rn(1, st.nq, 64, 512).bfloat16()
    out, seen = torch.empty_like(q), []
    real = C.lib.csa2_sparse_attn_tree

    def spy(*a):
        seen.append((ctypes.c_void_p(a[9]).value, a[10]))
        return real(*a)
    monkeypatch.setattr(C.lib, "csa2_sparse_attn_tree", spy)
    C.csa2_sparse_attn_tree(st.cache, st.tree, q, wd["win"], wd["draft"], idx, SCALE, out=out)
    (at, n), = seen
    assert n == 16 and at % 16 == 0
    for t in (idx, q, wd["win"], wd["draft"], out):      # no tensor of the call
        assert at + n <= t.data_ptr() or at >= t.data_ptr() + t.numel() * t.element_size()
    buf = st.cache.buffer                                # behind everything the cache lays out
    caps = (ctypes.c_int64 * st.batch)(*st.caps)
    nbytes = C.lib.csa2_cache_bytes(ctypes.byref(st.cfg), st.batch, caps)
    base = buf.data_ptr() + (-buf.data_ptr()) % 256
    assert base + nbytes <= at and at + n <= buf.data_ptr() + buf.numel()
