"""csa2_verify_tree behind several rejections of which each leaves 1e-9 of p: what
is left is formed by one rejection after the other (p - a q would be below p's
rounding)."""
import pytest
import torch

from tests.test_gpu_verify import expect, make, run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("vocab", [300, 9001])
@pytest.mark.parametrize("kids", [1, 2, 3, 6])
def test_what_is_left_after_rejections_that_leave_little(dtype, vocab, kids):
    """p and q agree in one token but for 1e-9 to 1e-7, which is all that a rejection
    leaves; other tokens have p > q, but 1e-40 of it."""
    S = 48
    parents = [[-1] * kids] * S
    d = make(parents, vocab, dtype, 17 + kids)
    d["temperature"].fill_(1.0)
    for i in range(S):
        p, q = d["root_logits"][i], d["draft_root"][i]
        p[:] = -1e4                       # a probability of 0 in both
        q[:] = -1e4
        top, other = (5 * i + 1) % vocab, (7 * i + 4) % vocab
        p[20:40], q[20:40] = -100.0, -120.0
        p[top] = q[top] = 0.0
        p[other] = -16.0 - i / 8
        q[other] = p[other] + 0.75
        for t in range(kids):
            d["tokens"][kids * i + t] = vocab - 1 - t - i
    d["uniform"].fill_(0.5)
    want = expect(parents, d)
    assert run(parents, d) == want
    if kids < 4:   # (the other tokens' 1e-40 gain 1e8 at each)
        assert want == [(-1, (5 * i + 1) % vocab) for i in range(S)]


@pytest.mark.parametrize("kids", [1, 2])
@pytest.mark.parametrize("gap", [600.0, 700.0, 712.0, 720.0, 735.0])
def test_what_is_left_may_be_subnormal(gap, kids):
    """All that a rejection leaves is e^-600 to e^-735 of p."""
    S, V = 16, 500
    parents = [[-1] * kids] * S
    d = make(parents, V, torch.float32, 23)
    d["temperature"].fill_(1.0)
    d["root_logits"].fill_(-5e3)
    d["draft_root"].fill_(-5e3)
    for i in range(S):
        d["root_logits"][i, 3 + i] = d["draft_root"][i, 3 + i] = 0.0
        d["root_logits"][i, 99 + 7 * i] = -gap
        for t in range(kids):
            d["tokens"][kids * i + t] = 400 + i + t
    want = expect(parents, d)
    assert run(parents, d) == want == [(-1, 99 + 7 * i) for i in range(S)]
