"""Selections behind an indexer whose waits ran out (its key loads withheld):
scores are whatever the workspace held and histograms lack their counts.  The
call ends, reports CSA2_ERR_TIMEOUT, and what it selected are entries of the
row or -1, without any access outside a buffer; the next call is right."""
import pytest
import torch

from tests.test_gpu_tree import Setup, chain, random_tree

pytestmark = pytest.mark.gpu

TIMEOUT = 6


def rn(seed, *shape):
    return torch.randn(*shape, generator=torch.Generator("cuda").manual_seed(seed), device="cuda")


def garbage(nbytes, seed):
    g = torch.Generator("cuda").manual_seed(seed)
    return torch.randint(0, 256, (max(16, nbytes),), generator=g, device="cuda").to(torch.uint8)


def timed_out(cache, run, rows):
    """run(workspace fill seed) -> selection; rows: entries of each row."""
    good = run(1)
    assert cache.device_error() == 0
    cache.set_wait_limit(200_000)
    cache.inject_fault(1)
    for seed in (2, 3):
        bad = run(seed)
        torch.cuda.synchronize()
        assert cache.device_error() == TIMEOUT
        n = torch.tensor(rows, device="cuda")[:, None]
        assert torch.all((bad >= -1) & (bad < n))
    cache.inject_fault(0)
    cache.set_wait_limit(0)
    assert torch.equal(run(4), good)
    assert cache.device_error() == 0


@pytest.mark.parametrize("idx_layout", [0, 1])
@pytest.mark.parametrize("call", ["decode", "bf16 scores", "prefill", "reindex"])
@pytest.mark.parametrize("lens", [[900, 30, 3000], [20000, 800, 70001]])   # one pass; segments
def test_selections(idx_layout, call, lens):
    import fp4_kv_cache_index_gb300 as C
    cache = C.Cache(C.config(idx_layout=idx_layout), lens)
    C.csa2_append_entries(cache, [0, 1, 2], lens, rn(1, sum(lens), 512), rn(2, sum(lens), 128).bfloat16())
    nq = 21 if call == "prefill" else 3
    q, w = rn(3, nq, 32, 128).bfloat16(), rn(4, nq, 32)
    rows = [lens[2]] * nq if call == "prefill" else lens
    if call == "decode":
        run = lambda s: C.csa2_index_topk_decode(
            cache, q, w, workspace=garbage(C.csa2_index_workspace_bytes(cache, 3), s))
    elif call == "bf16 scores":
        run = lambda s: C.csa2_index_topk_decode_bf16(
            cache, q, w, workspace=garbage(C.csa2_index_workspace_bytes(cache, 3), s))
    elif call == "prefill":
        run = lambda s: C.csa2_index_topk_prefill(
            cache, 2, lens[2] - 21, q, w,
            workspace=garbage(C.csa2_index_prefill_workspace_bytes(cache, 2, nq), s))
    else:
        sc = torch.full((3, (max(lens) + 3) // 4 * 4), float("nan"), device="cuda")
        C.csa2_index_scores_decode(cache, q, w, sc)
        pool = C.csa2_hsi_pool(sc, lens, max_blocks=96)
        nbytes = int(C.lib.csa2_index_reindex_workspace_bytes(cache.handle, 3, 96))
        run = lambda s: C.csa2_index_topk_reindex_decode(cache, q, w, pool, workspace=garbage(nbytes, s))
    timed_out(cache, run, rows)


@pytest.mark.parametrize("idx_layout", [0, 1])
@pytest.mark.parametrize("trees, pos0", [([random_tree(9, 2), chain(5)], [1300, 40]),
                                         ([random_tree(20, 3), random_tree(7, 4)], [30011, 17000]),
                                         ([[-1], [-1]], [40000, 700])])
def test_drafts(idx_layout, trees, pos0):
    import fp4_kv_cache_index_gb300 as C
    st = Setup(trees, pos0, idx_layout=idx_layout)
    nbytes = C.csa2_index_workspace_bytes(st.cache, st.nq)
    timed_out(st.cache, lambda s: C.csa2_index_topk_tree(st.cache, st.tree, st.q_idx, st.w,
                                                         workspace=garbage(nbytes, s)),
              [len(st.ent[i]) for i, _ in st.at])


@pytest.mark.parametrize("n", [700, 9000, 40000])
@pytest.mark.parametrize("k", [512, 2048])
@pytest.mark.parametrize("segments", [False, True])
def test_histograms_that_are_not_the_row_s(n, k, segments):
    """csa2_topk with counts that are too few, too many, all of one bin, another
    row's or any words at all: indices of the row or -1."""
    import fp4_kv_cache_index_gb300 as C
    s = rn(5, 1, n).repeat(8, 1)
    key = s[:1].view(torch.int32).to(torch.int64) & 0xFFFFFFFF
    key = torch.where(key >> 31 == 1, 0xFFFFFFFF - key, key | 0x80000000)
    right = torch.bincount((key >> 21)[0], minlength=2048).to(torch.int32)
    one = torch.zeros_like(right)
    one[1030] = n
    g = torch.Generator("cuda").manual_seed(6)
    words = torch.randint(-2 ** 31, 2 ** 31, (2048,), generator=g, device="cuda").to(torch.int32)
    hist = torch.stack([right, torch.zeros_like(right), right // 2, right * 3, right.flip(0), one,
                        words, torch.full_like(right, -1)])
    ws = (garbage(C.csa2_topk_workspace_bytes(8, n), 7) if segments else None)
    score = torch.full((8, k), 9.0, device="cuda")
    idx = C.csa2_topk(s, [n] * 8, k, key_hist=hist, score_out=score, workspace=ws)
    want = C.csa2_topk(s[:1].contiguous(), [n], k)
    assert torch.equal(idx[:1], want)
    assert torch.all((idx >= -1) & (idx < n))
    for r in range(8):         # what is there has its own score, ascending
        i = idx[r][idx[r] >= 0].long()
        assert torch.equal(s[r][i], score[r][:len(i)]) and torch.all(i[1:] > i[:-1])
        assert torch.all(idx[r][len(i):] == -1) and torch.all(score[r][len(i):] == 0)
