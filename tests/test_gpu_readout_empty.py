"""Readouts in which a CTA has no tile of candidates: queries that select
nothing and have no window, and pairs of CTAs whose only tile is the first
one's.  Such a CTA stages its outputs where its query rows are still arriving
unless it waits for them, so the queries here come from HBM (a buffer larger
than L2 is written before every call) and are large: an output that holds
one of them shows."""
import pytest
import torch

pytestmark = pytest.mark.gpu

SCALE = 512 ** -0.5


def queries(nq, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (1e30 * torch.randn(nq, 64, 512, generator=g, device="cuda")).bfloat16()


def cold():
    return torch.empty(512 << 20, dtype=torch.uint8, device="cuda").fill_(1)


@pytest.mark.parametrize("nq", [1, 40, 700])
@pytest.mark.parametrize("split", [False, True])
def test_decode_with_nothing_selected_is_zero(nq, split):
    import fp4_kv_cache_index_gb300 as C
    cache = C.Cache(C.config(swa=0), [16] * nq)
    q = queries(nq, 1)
    idx = torch.full((nq, 512), -1, dtype=torch.int32, device="cuda")
    ws = None if split else torch.empty(0, dtype=torch.uint8, device="cuda")
    for _ in range(10):
        out, lse = torch.full_like(q, 3.0), torch.zeros(nq, 64, device="cuda")
        keep = cold()
        C.csa2_sparse_attn_decode(cache, q, None, idx, SCALE, out=out, lse=lse, workspace=ws)
        del keep
        assert torch.all(out == 0) and torch.all(lse == -float("inf"))
    assert cache.device_error() == 0


@pytest.mark.parametrize("nq", [5, 64])
@pytest.mark.parametrize("split", [False, True])
def test_drafts_with_nothing_selected_are_zero(nq, split):
    import fp4_kv_cache_index_gb300 as C
    cache = C.Cache(C.config(swa=0, ratio=16), [16])
    tree = C.Tree([[-1] * nq], [0])
    q = queries(nq, 2)
    idx = torch.full((nq, 512), -1, dtype=torch.int32, device="cuda")
    ws = None if split else torch.empty(0, dtype=torch.uint8, device="cuda")
    for _ in range(10):
        out, lse = torch.full_like(q, 3.0), torch.zeros(nq, 64, device="cuda")
        keep = cold()
        C.csa2_sparse_attn_tree(cache, tree, q, None, None, idx, SCALE, out=out, lse=lse, workspace=ws)
        del keep
        assert torch.all(out == 0) and torch.all(lse == -float("inf"))
    assert cache.device_error() == 0


def test_prefill_with_nothing_selected_is_zero():
    import fp4_kv_cache_index_gb300 as C
    cache = C.Cache(C.config(swa=0), [16])
    q = queries(900, 3)
    idx = torch.full((900, 512), -1, dtype=torch.int32, device="cuda")
    for _ in range(10):
        out = torch.full_like(q, 3.0)
        keep = cold()
        C.csa2_sparse_attn_prefill(cache, 0, 0, q, None, 0, idx, SCALE, out=out)
        del keep
        assert torch.all(out == 0)
    assert cache.device_error() == 0


@pytest.mark.parametrize("tree", [False, True])
def test_a_pair_with_one_tile(tree):
    """The window is the only tile, the second CTA of each pair has none: the
    mean of its rows for queries orthogonal to them (logits exactly 0)."""
    import fp4_kv_cache_index_gb300 as C
    nq, W = 30, 128
    g = torch.Generator(device="cuda").manual_seed(4)
    # rows in the first 256 channels, queries in the last 256
    win = torch.zeros(nq, W, 512, device="cuda")
    win[..., :256] = torch.randn(nq, W, 256, generator=g, device="cuda")
    win = win.bfloat16()
    q = queries(nq, 5)
    q[..., :256] = 0
    idx = torch.full((nq, 512), -1, dtype=torch.int32, device="cuda")
    if tree:        # a draft behind 130 committed tokens: 127 of the window's rows and its own
        cache, t = C.Cache(C.config(ratio=16), [16] * nq), C.Tree([[-1]] * nq, [130] * nq)
        C.csa2_append_entries(cache, list(range(nq)), [8] * nq, torch.zeros(8 * nq, 512, device="cuda"),
                              torch.zeros(8 * nq, 128, dtype=torch.bfloat16, device="cuda"))
        draft = win[:, 127].contiguous()
        rows = torch.cat([torch.full_like(win[:, :1], float("nan")), win[:, :127]], 1)
    else:
        cache = C.Cache(C.config(), [16] * nq)
    want = win.double().mean(1)[:, None].expand(nq, 64, 512)
    for _ in range(10):
        out = torch.full_like(q, 3.0)
        keep = cold()
        if tree:
            C.csa2_sparse_attn_tree(cache, t, q, rows, draft, idx, SCALE, out=out)
        else:
            C.csa2_sparse_attn_decode(cache, q, win, idx, SCALE, out=out)
        del keep
        # probabilities are exactly 1 and the sum exactly 128: the fp32 sum's 128
        # roundings (the tensor core may truncate, 2^-23 each) and the output's
        tol = 2.0 ** -8 * want.abs() + 129 * 2.0 ** -23 * win.double().abs().mean(1)[:, None]
        assert torch.all((out.double() - want).abs() <= tol)
    assert cache.device_error() == 0
