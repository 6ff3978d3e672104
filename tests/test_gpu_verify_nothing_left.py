"""csa2_verify_tree where max(p - a q, 0) is 0 everywhere: the target's and the
draft's row are alike and a child's token is masked in both, so that it is
rejected (0 < 0 does not hold) and nothing is left.  a and b stay as they are: a
sibling is tested against p again, and without one the next token is drawn from
p."""
import math

import pytest
import torch

from tests.test_gpu_verify import expect, gen, make, run

pytestmark = pytest.mark.gpu


def alike(parents, vocab, dtype, seed, masked):
    """Both models' rows the same; the drafts in `masked` (of each tree) have
    tokens that their parent's row masks."""
    d = make(parents, vocab, dtype, seed)
    d["temperature"].copy_(torch.tensor([(1.0, 0.6, 1.7, 1.1)[i % 4] for i in range(len(parents))]))
    at = 0
    for i, ps in enumerate(parents):
        for t, p in enumerate(ps):
            if t in masked:
                row = d["root_logits"][i] if p < 0 else d["logits"][at + p]
                x = (7 * t + 5 * i) % vocab
                row[x] = -math.inf
                d["tokens"][at + t] = x
        at += len(ps)
    at = 0
    for i, ps in enumerate(parents):   # likely tokens that no sibling has masked
        for t, p in enumerate(ps):
            if t not in masked:
                row = d["root_logits"][i] if p < 0 else d["logits"][at + p]
                d["tokens"][at + t] = int(row.float().topk(3)[1][(t + i) % 3])
        at += len(ps)
    d["draft_logits"], d["draft_root"] = d["logits"].clone(), d["root_logits"].clone()
    return d


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("vocab", [12, 999, 3001, 50257, 131072])
def test_a_sibling_behind_masked_ones_is_tested_against_all_of_p(dtype, vocab):
    parents = [[-1, -1, -1, 2, 2]] * 12
    d = alike(parents, vocab, dtype, 60, (0, 1, 3))
    d["uniform"].fill_(1 - 2.0 ** -24)   # u q < p holds all the same
    want = expect(parents, d)
    assert run(parents, d) == want
    assert [a for a, _ in want] == [4] * 12


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("vocab", [12, 999, 3001, 50257, 131072])
@pytest.mark.parametrize("kids", [1, 3])
def test_the_token_is_drawn_from_p_behind_masked_ones(dtype, vocab, kids):
    parents = [[-1] * kids] * 24
    d = alike(parents, vocab, dtype, 70, tuple(range(kids)))
    d["uniform"].copy_(torch.rand(24 * kids, generator=gen(3), device="cuda"))
    want = expect(parents, d)
    assert run(parents, d) == want
    assert all(a == -1 and t >= 0 for a, t in want)


def test_rows_that_are_shifted_against_each_other():
    """The draft's logits are the target's plus a number of few bits: the same
    probabilities, in other memory (and at another distance to 16 bytes)."""
    parents = [[-1, -1]] * 8
    d = alike(parents, 4096, torch.float32, 80, (0,))
    for k in ("logits", "root_logits"):
        d[k].copy_((d[k] * 64).round() / 64)
    for k, f in (("draft_logits", "logits"), ("draft_root", "root_logits")):
        n = d[f].shape[0]
        d[k] = torch.empty(n * 4096 + 1, device="cuda")[1:].view(n, 4096).copy_(d[f] + 4.0)
    d["uniform"].fill_(0.999)
    # (the walk divides by T before it subtracts, which rounds shifted rows apart)
    want = expect(parents, dict(d, draft_logits=d["logits"], draft_root=d["root_logits"]))
    assert run(parents, d) == want and [a for a, _ in want] == [1] * 8
