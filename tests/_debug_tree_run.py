"""Calls of drafted tokens under the bounds-checked library
(libcsa2_debug.so), as a child process of tests/test_gpu_tree_debug.py with
CSA2_DEBUG=1: widths of the trees from one draft to eight and more, whose
groups fill a tile of 2, 4 or 8 queries and of which several end in a smaller
group; bf16 and MXFP4 keys.  Every index of a table, a buffer or tensor memory
that a kernel forms has to stay inside (the device error word is clean), and
the scores are the formula's."""
import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, ROOT)

import torch  # noqa: E402

import fp4_kv_cache_index_gb300 as C  # noqa: E402
from tests.test_gpu_tree import (  # noqa: E402
    Setup, chain, check_scores, compare_readout, random_tree, window)

WIDTHS = [[1], [2], [2, 1, 0, 2], [3], [4, 1], [3, 4, 2], [5], [8], [9, 2, 1], [17, 6], [64]]


def run(widths, idx_layout, seed):
    trees = [random_tree(n, seed + i) for i, n in enumerate(widths)]
    st = Setup(trees, [700 - 150 * i for i in range(len(widths))], idx_layout=idx_layout, seed=seed)
    ld = (max(len(x) for x in st.rows()) + 3) // 4 * 4
    scores = torch.full((st.nq, ld), -3.0, device="cuda")
    C.csa2_index_scores_tree(st.cache, st.tree, st.q_idx, st.w, scores)
    assert st.cache.device_error() == 0, ("scores", widths, idx_layout)
    check_scores(st, scores, -3.0)
    idx = C.csa2_index_topk_tree(st.cache, st.tree, st.q_idx, st.w)
    assert st.cache.device_error() == 0, ("selection", widths, idx_layout)
    compare_readout(st, idx, window(st, seed + 50))
    assert st.cache.device_error() == 0, ("readout", widths, idx_layout)
    C.csa2_cache_accept_tree(st.cache, st.tree, [len(t) - 1 for t in trees])
    assert st.cache.device_error() == 0, ("acceptance", widths, idx_layout)


if __name__ == "__main__":
    assert C.LIB_PATH.endswith("libcsa2_debug.so"), C.LIB_PATH
    for idx_layout in (0, 1):
        for i, widths in enumerate(WIDTHS):
            run(widths, idx_layout, 900 + 20 * i)
        # many tiles a CTA, so that each goes from group to group
        st = Setup([chain(2)] * 9, [3000 - 7 * i for i in range(9)], idx_layout=idx_layout)
        st.cache.set_index_sms(5)
        scores = torch.full((st.nq, 3004), -3.0, device="cuda")
        C.csa2_index_scores_tree(st.cache, st.tree, st.q_idx, st.w, scores)
        assert st.cache.device_error() == 0
        check_scores(st, scores, -3.0)
    print("drafted tokens: all cases clean")
