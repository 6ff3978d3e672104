"""csa2_verify_tree over a vocabulary whose sums have thousands of terms in turn
a thread: tests next to their border are decided as 64 bits decide them."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu


def test_borders_over_a_large_vocabulary():
    """4096 likely tokens, one for each thread's share, all others alike: p in closed
    form.  fp32 sums of equal terms are off by up to 6e-5 here (each addition's rounding
    is the same one until the sum doubles); u is 6e-6 beside p."""
    import fp4_kv_cache_index_gb300 as C
    V, N, x, best = 1 << 28, 4096, 40, 16
    rows = torch.full((2, V), -8.0, device="cuda")
    rows[:, :8 * N:8] = 0.0
    noise = torch.ones(2, V, device="cuda")
    noise[:, best] = 0.5                      # the best of the others
    tree = C.Tree([[-1], [-1]], [0, 0])
    tok = torch.full((2,), x, dtype=torch.int32, device="cuda")
    for k in range(16):
        # the others' sum is 50 to 200 times the likely ones', of no short binary form
        t = torch.tensor(8.0 / math.log((V - N) / (N * 50.0 * 1.0937 ** k)), dtype=torch.float32)
        p = 1.0 / (N + (V - N) * math.exp(-8.0 / float(t)))
        u = torch.tensor([p * (1 - 6e-6), p * (1 + 6e-6)], dtype=torch.float64).float()
        want = [(0 if float(v) < p else -1, best) for v in u]
        assert [a for a, _ in want] == [0, -1]
        acc, nxt = C.csa2_verify_tree(tree, tok, rows, t.expand(2).cuda().contiguous(), u.cuda(), noise,
                                      rows)
        assert list(zip(acc.tolist(), nxt.tolist())) == want, k
