"""Trees of one draft: the selection does what decode's does on the same
cache, and takes the same way there."""
import pytest
import torch

from tests.test_gpu_tree import Setup

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("idx_layout", [0, 1])
@pytest.mark.parametrize("pos0", [[700, 30, 300], [40013, 30, 25000]])
def test_one_draft_selects_as_decode_does(idx_layout, pos0):
    """The same selection, and the same scores, histograms and segments behind
    it: the workspaces agree in every word that two decode calls agree in."""
    import fp4_kv_cache_index_gb300 as C
    st = Setup([[-1], [], [-1]], pos0, idx_layout=idx_layout)
    n = C.csa2_index_workspace_bytes(st.cache, 2)
    left = []
    for call in ("decode", "decode", "tree"):
        ws = torch.full((n,), 0xA5, dtype=torch.uint8, device="cuda")
        sc = torch.zeros(2, 512, device="cuda")
        if call == "tree":
            idx = C.csa2_index_topk_tree(st.cache, st.tree, st.q_idx, st.w, topk_score=sc, workspace=ws)
        else:
            idx = C.csa2_index_topk_decode(st.cache, st.q_idx, st.w, seq_ids=[0, 2], topk_score=sc,
                                           workspace=ws)
        left.append((idx, sc, ws[:n // 4 * 4].view(torch.int32)))
    (i0, s0, a), (i1, s1, b), (i2, s2, t) = left
    assert torch.equal(i0, i1) and torch.equal(i0, i2)
    assert torch.equal(s0, s1) and torch.equal(s0, s2)
    same = a == b
    assert torch.equal(t[same], a[same])
    assert st.cache.device_error() == 0
