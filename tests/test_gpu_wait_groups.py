"""Waits that run out where a CTA of the decode and prefill indexers
goes through several queries' tiles (key loads withheld, few SMs): the calls
end, report CSA2_ERR_TIMEOUT and leave the cache usable.  The warps of an
epilogue meet at barriers when the query changes, which a warp that gave up
has to join as well."""
import pytest
import torch

pytestmark = pytest.mark.gpu

TIMEOUT = 6


def rn(seed, *shape):
    return torch.randn(*shape, generator=torch.Generator("cuda").manual_seed(seed), device="cuda")


@pytest.mark.parametrize("idx_layout", [0, 1])
@pytest.mark.parametrize("call", ["decode", "bf16 scores", "prefill"])
@pytest.mark.parametrize("index_sms", [1, 4])
def test_waits_run_out_across_queries(idx_layout, call, index_sms):
    import fp4_kv_cache_index_gb300 as C
    lens = [150 + 217 * i for i in range(7)]
    cache = C.Cache(C.config(idx_layout=idx_layout), lens)
    C.csa2_append_entries(cache, list(range(7)), lens, rn(1, sum(lens), 512),
                          rn(2, sum(lens), 128).bfloat16())
    nq = 40 if call == "prefill" else 7
    q, w = rn(3, nq, 32, 128).bfloat16(), rn(4, nq, 32)
    run = {"decode": lambda: C.csa2_index_topk_decode(cache, q, w),
           "bf16 scores": lambda: C.csa2_index_topk_decode_bf16(cache, q, w),
           "prefill": lambda: C.csa2_index_topk_prefill(cache, 6, 1400, q, w)}[call]
    cache.set_index_sms(index_sms)
    good = run()
    assert cache.device_error() == 0
    scores = torch.full((7, 1456), 7.0, device="cuda")
    cache.set_wait_limit(200_000)
    cache.inject_fault(1)
    if call == "decode":        # with histograms behind the scores
        hist = torch.zeros(7, 2048, dtype=torch.int32, device="cuda")
        C.csa2_index_scores_decode(cache, q, w, scores, key_hist=hist)
    elif call == "bf16 scores":
        C.csa2_index_scores_decode_bf16(cache, q, w, torch.zeros(7, 1456, dtype=torch.bfloat16, device="cuda"))
    else:
        C.csa2_index_scores_prefill(cache, 6, 1400, q, w, torch.zeros(nq, 1456, device="cuda"))
    torch.cuda.synchronize()    # the kernels ended by themselves
    assert torch.all(scores == 7.0)
    assert cache.device_error() == TIMEOUT
    cache.inject_fault(0)
    cache.set_wait_limit(0)
    assert torch.equal(run(), good)
    assert cache.device_error() == 0
