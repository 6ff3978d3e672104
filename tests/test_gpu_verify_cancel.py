"""csa2_verify_tree where p and a q all but cancel, and where two candidates'
scores of what is left are nearer than fp32 tells: the token is that of 64-bit
arithmetic, after one and after two rejections."""
import math

import pytest
import torch

from tests.test_gpu_verify import expect, gen, make, run

pytestmark = pytest.mark.gpu

TOP = 1 - 2.0 ** -24


def near_rows(parents, vocab, dtype, seed, spread, kind):
    """Draft rows that differ from the target's by `spread`; every draft is
    rejected: its token is masked in both rows, or the draft's model is sure of
    it and u is the largest."""
    S, n = len(parents), len(parents[0])
    d = make(parents, vocab, dtype, seed)
    d["temperature"].copy_(torch.tensor([(1.0, 0.75, 1.3)[i % 3] for i in range(S)]))
    noise = spread * torch.randn(S, vocab, generator=gen(seed + 9), device="cuda")
    for i in range(S):
        if kind == "masked":
            for t in range(n):
                x = (11 * t + 3 * i) % vocab
                d["root_logits"][i, x] = -math.inf
                d["tokens"][n * i + t] = x
        else:   # tokens that the draft's model likes better
            x = d["root_logits"][i].float().topk(n)[1]
            noise[i, x] = noise[i, x].abs() + 2 * spread
            d["tokens"][n * i:n * i + n] = x.int()
    d["draft_root"] = (d["root_logits"].float() + noise).to(dtype)
    d["uniform"].fill_(TOP)
    return d


def left(d, i, n):
    """What is left of p behind n rejections of tree i, in 64 bits."""
    T = float(d["temperature"][i])
    p = torch.softmax(d["root_logits"][i].double() / T, 0)
    q = torch.softmax(d["draft_root"][i].double() / T, 0)
    for _ in range(n):
        r = (p - q).clamp(min=0)
        if float(r.sum()) > 0:
            p = r / r.sum()
    return p


@pytest.mark.parametrize("kind", ["masked", "liked"])
@pytest.mark.parametrize("n", [1, 2])
@pytest.mark.parametrize("spread", [1e-1, 1e-2, 1e-3, 1e-4, 1e-5, 2e-6])
def test_rows_that_all_but_cancel(spread, n, kind):
    parents = [[-1] * n] * 48
    d = near_rows(parents, 20000, torch.float32, 40 + n, spread, kind)
    want = expect(parents, d)
    assert run(parents, d) == want
    if kind == "masked":
        assert all(a == -1 for a, _ in want)


@pytest.mark.parametrize("kind", ["masked", "liked"])
@pytest.mark.parametrize("spread", [2e-3, 2e-2])
def test_bf16_rows_that_all_but_cancel(spread, kind):
    parents = [[-1]] * 96
    d = near_rows(parents, 4001, torch.bfloat16, 50, spread, kind)
    assert run(parents, d) == expect(parents, d)


def test_rows_that_differ_in_an_unlikely_token():
    """fp32 finds nothing left; 64 bits find the one token that the draft's model
    likes less, by 1e-9 of the probability or less."""
    V, S = 3000, 24
    parents = [[-1, -1]] * S
    d = near_rows(parents, V, torch.float32, 55, 0.0, "masked")
    for i in range(S):
        x = (100 + 17 * i) % V
        if torch.isinf(d["root_logits"][i, x]):
            x += 1
        d["root_logits"][i, x] = d["root_logits"][i].max() - 18.0
        d["draft_root"][i] = d["root_logits"][i]
        d["draft_root"][i, x] -= 1.0
        d["tokens"][2 * i + 1] = x        # the second draft: all that is left
    d["temperature"].fill_(1.0)
    want = expect(parents, d)
    assert run(parents, d) == want
    assert [a for a, _ in want] == [1] * S


@pytest.mark.parametrize("kind", ["masked", "liked"])
@pytest.mark.parametrize("spread", [0.7, 0.05])
@pytest.mark.parametrize("n", [1, 2])
def test_near_ties_of_what_is_left_are_decided_exactly(n, spread, kind):
    """The second candidate's noise makes its score the first's but for fp32's
    rounding of that noise."""
    S = 64
    parents = [[-1] * n] * S
    d = near_rows(parents, 20000, torch.float32, 90 + n, spread, kind)
    for i in range(S):
        p = left(d, i, n)
        s = p / d["noise"][i].double()
        a, b = s.topk(2)[1].tolist()
        d["noise"][i, b] = (p[b] / s[a]).float()
    assert run(parents, d) == expect(parents, d)
