"""Bounded waits of the drafted-token kernels where a CTA goes through several
groups of drafts: with the key loads withheld every wait runs out, the call
ends, the error word says so, and the cache works afterwards."""
import pytest
import torch

from tests.test_gpu_tree import Setup, check_scores, random_tree

pytestmark = pytest.mark.gpu

TIMEOUT = 6       # CSA2_ERR_TIMEOUT


def withheld(st, index_sms):
    import fp4_kv_cache_index_gb300 as C
    ld = (max(len(x) for x in st.rows()) + 3) // 4 * 4
    scores = torch.full((st.nq, ld), -5.0, device="cuda")
    st.cache.set_index_sms(index_sms)
    st.cache.set_wait_limit(200_000)
    st.cache.inject_fault(1)
    C.csa2_index_scores_tree(st.cache, st.tree, st.q_idx, st.w, scores)
    torch.cuda.synchronize()                  # the kernel ended by itself
    assert torch.all(scores == -5.0)
    assert st.cache.device_error() == TIMEOUT
    assert st.cache.device_error() == 0       # read and cleared
    st.cache.inject_fault(0)
    st.cache.set_wait_limit(0)
    C.csa2_index_scores_tree(st.cache, st.tree, st.q_idx, st.w, scores)
    check_scores(st, scores, -5.0)
    assert st.cache.device_error() == 0


@pytest.mark.parametrize("idx_layout", [1, 0])
@pytest.mark.parametrize("index_sms", [1, 3, 152])
def test_waits_run_out_across_groups(idx_layout, index_sms):
    """Sequences of at most 128 entries: a group is one tile with one M-group,
    so the two epilogue sets of the MXFP4 kernel wait in different groups."""
    trees = [random_tree(3 + i % 7, 60 + i) for i in range(12)]
    withheld(Setup(trees, [20 + 9 * i for i in range(12)], idx_layout=idx_layout), index_sms)


@pytest.mark.parametrize("idx_layout", [1, 0])
def test_waits_run_out_with_several_groups_of_keys(idx_layout):
    """Odd and even numbers of M-groups a sequence, none of them a whole tile."""
    trees = [random_tree(5 + i, 80 + i) for i in range(5)]
    withheld(Setup(trees, [300, 100, 700, 129, 400], idx_layout=idx_layout), 2)
