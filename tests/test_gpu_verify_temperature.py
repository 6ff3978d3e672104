"""csa2_verify_tree at the smallest and largest temperatures."""
import math

import pytest
import torch

from tests.test_gpu_verify import expect, gen, make, random_tree, run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("temperature", [1e-45, 1e-40, 1e-38, 1e-37, 1e-31])
@pytest.mark.parametrize("draft", ["logits", "certain"])
def test_the_smallest_temperatures_take_the_largest_logit(temperature, draft):
    """Subnormal numbers among them: their reciprocal is no fp32 number."""
    parents = [random_tree(7, i) for i in range(5)] + [[]] * 3
    d = make(parents, 5000, torch.float32, 30, spread=30.0)
    if draft == "certain":
        d["draft_logits"] = d["draft_root"] = None
    d["temperature"].fill_(temperature)
    want = expect(parents, d)
    assert run(parents, d) == want
    assert all(t >= 0 for _, t in want) and any(a >= 0 for a, _ in want)


@pytest.mark.parametrize("temperature", [1e-3, 1e-6, 1e-9, 1e-12, 1e-20])
def test_near_logits_at_small_temperatures(temperature):
    """A leaf's first two logits a few steps of fp32 apart, or alike: their scores
    are up to 1e22, and what tells them apart is the difference."""
    S, V = 48, 700
    parents = [[]] * S
    d = make(parents, V, torch.float32, 31)
    d["temperature"].fill_(temperature)
    for i in range(S):
        x, y = 3 + i, 650 - 7 * i
        v = torch.tensor(20.0 + i, dtype=torch.float32)
        d["root_logits"][i, x] = v
        for _ in range(i % 4):
            v = torch.nextafter(v, torch.tensor(0.0 if i % 3 else 99.0))
        d["root_logits"][i, y] = v
    want = expect(parents, d)
    assert run(parents, d) == want


def test_an_infinite_temperature_makes_all_tokens_alike():
    """All but the masked ones."""
    parents = [[-1], []] * 6
    d = make(parents, 777, torch.bfloat16, 32)
    d["root_logits"][:, ::3] = -math.inf
    d["tokens"].fill_(3)                 # masked: rejected
    d["draft_logits"] = d["draft_root"] = None
    d["temperature"].fill_(math.inf)
    got = run(parents, d)
    ok = d["noise"].clone()
    ok[:, ::3] = math.inf
    assert got == [(-1, int(t)) for t in ok.argmin(1)]
