"""Indexer queries that hold NaN or infinities: drafts get the scores of
decode, bit for bit, through the rounding of queries to MXFP4 too.  NaN of
both signs and of several payloads beside finite values, which leave MXFP4
scores finite; then infinities and the type's extremes among them."""
import pytest
import torch

from tests.test_gpu_tree import Setup, chain, path_of

pytestmark = pytest.mark.gpu


NAN = [0x7FC0, 0xFFC0, 0x7F81, 0xFF81, 0x7FFF, 0xFFFF]
REST = [0x7F80, 0xFF80, 0x0000, 0x8000, 0x0001, 0x8001, 0x7F7F, 0xFF7F]


def specials(st, seed, bits):
    """Every tenth value or so of the queries replaced by one of these."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    pool = torch.tensor([b - 65536 if b >= 32768 else b for b in bits], dtype=torch.int16, device="cuda")
    q = st.q_idx.view(torch.int16)
    pick = pool[torch.randint(0, len(bits), q.shape, generator=g, device="cuda")]
    hit = torch.rand(q.shape, generator=g, device="cuda") < 0.1
    hit[:, 7, 32:64] = True                # a whole block of 32 channels
    hit[:, 20:] = False                    # and heads without any
    q[hit] = pick[hit]


@pytest.mark.parametrize("bits", ["nan", "all"])
@pytest.mark.parametrize("idx_layout", [0, 1])
@pytest.mark.parametrize("n", [1, 2, 3, 11])
def test_scores_of_special_queries_are_decode_s(idx_layout, n, bits):
    import fp4_kv_cache_index_gb300 as C
    st = Setup([chain(n)], [900], idx_layout=idx_layout)
    specials(st, 100 + n, NAN if bits == "nan" else NAN + REST)
    scores = torch.full((n, 912), -5.0, device="cuda")
    C.csa2_index_scores_tree(st.cache, st.tree, st.q_idx, st.w, scores)
    for r in range(n):
        cols = st.rows()[r]
        assert len(path_of(st.trees[0], r)) == r + 1
        one = C.Cache(st.cfg, [len(cols)])
        C.csa2_append_entries(one, [0], [len(cols)], st.ent[0][cols].contiguous(),
                              st.key[0][cols].contiguous())
        want = torch.full((1, 912), -5.0, device="cuda")
        C.csa2_index_scores_decode(one, st.q_idx[r:r + 1].contiguous(), st.w[r:r + 1].contiguous(), want)
        got, ref = scores[r].view(torch.int32), want[0].view(torch.int32)
        assert torch.equal(got, ref), (r, int((got != ref).sum()))
    if bits == "nan" and idx_layout == 1:
        assert torch.isfinite(scores).all()
    assert st.cache.device_error() == 0
