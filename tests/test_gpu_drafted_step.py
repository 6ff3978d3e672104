"""Steps of speculative decoding through a layer of window attention -- the tree's
attention, the verification, the accepted rows' way into the cache -- against
token by token decoding with the same operators.

A small made-up model: a token's row and query are its own random vectors (the
row with a part for its position), its logits the sum of the attention's outputs
over the heads times a random matrix, in 64 bits.  With one query an item (128
heads) the attention of a tree sums in the order of the single token's, so both
runs have the same outputs, bit for bit, and take the same tokens."""
import random

import pytest
import torch

pytestmark = pytest.mark.gpu
V, HEADS, SCALE = 61, 128, 512 ** -0.5


def C():
    import fp4_kv_cache_index_gb300 as c
    return c


def dev64(xs):
    return torch.tensor(xs, dtype=torch.int64, device="cuda")


def dev32(xs):
    return torch.tensor(xs, dtype=torch.int32, device="cuda")


class Toy:
    def __init__(self, seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        def r(*s):
            return torch.randn(*s, generator=g, device="cuda")
        self.e, self.p, self.q = r(V, 512), r(997, 512), r(V, HEADS, 512).bfloat16()
        self.head = r(512, V).double()

    def rows(self, tokens, pos):
        at = torch.tensor([p % 997 for p in pos], device="cuda")
        return (self.e[torch.tensor(tokens, device="cuda")] + 0.5 * self.p[at]).bfloat16()

    def queries(self, tokens):
        return self.q[torch.tensor(tokens, device="cuda")].contiguous()

    def logits(self, out):
        return (out.double().sum(1) @ self.head).float()


def greedy(c, toy, win, seqs, tokens, pos, steps):
    """Each sequence's tokens: the given ones, then those of the largest logit."""
    said = [[t] for t in tokens]
    for k in range(steps):
        now = [s[-1] for s in said]
        at = dev64([p + k for p in pos])
        c.csa2_window_append(win, toy.rows(now, [p + k for p in pos]), at, None, seqs)
        out = c.csa2_window_attn_decode(win, toy.queries(now), at, SCALE, seqs, rope_out=True)
        for s, t in zip(said, toy.logits(out).argmax(1).tolist()):
            s.append(t)
    return said


def draft_tree(rng, said, at, n_right):
    """Tokens and parents: the sequence's next token, n_right of those that follow,
    and others beside them."""
    tokens, parents, last = [said[at]], [-1], 0
    for k in range(1, n_right + 1):
        for _ in range(rng.randrange(3)):
            tokens.append((said[at + k] + 1 + rng.randrange(V - 1)) % V)
            parents.append(last)
        tokens.append(said[at + k])
        parents.append(last)
        last = len(tokens) - 1
    for _ in range(rng.randrange(4)):   # and below the last right one, wrong again
        tokens.append((said[at + n_right + 1] + 1 + rng.randrange(V - 1)) % V)
        parents.append(last)
    return tokens, parents, last


@pytest.mark.parametrize("fp8", [True, False])
@pytest.mark.parametrize("swa,n_first", [(128, 4), (6, 2)])
def test_drafted_steps_are_greedy_decoding(fp8, swa, n_first):
    c, rng, toy = C(), random.Random(3), Toy(5)
    seqs, lens, steps = [2, 0, 3], [150, 1, 37], 24
    fresh = [rng.randrange(V) for _ in seqs]
    prompts = [[rng.randrange(V) for _ in range(n)] for n in lens]

    def filled():
        win = c.Window(4, swa, n_first, fp8)
        rows = torch.cat([toy.rows(p, range(len(p))) for p in prompts])
        c.csa2_window_append(win, rows, dev64([0] * 3), lens, seqs)
        return win

    plain = filled()
    said = greedy(c, toy, plain, seqs, fresh, lens, steps)
    win, at = filled(), [0] * 3
    while min(at) + 9 < steps:
        drafted = [draft_tree(rng, s, a, rng.randrange(6)) for s, a in zip(said, at)]
        tokens = [t for d in drafted for t in d[0]]
        tree = c.Tree([d[1] for d in drafted], [n + a for n, a in zip(lens, at)], seqs)
        places = [n + a + d for n, a, depths in zip(lens, at, tree.depths) for d in depths]
        rows = toy.rows(tokens, places)
        drafts = c.csa2_swa_fp8_quantise(rows) if fp8 else rows
        q, tok = toy.queries(tokens), dev32(tokens)
        accepted, following = dev32([0] * 3), dev32([0] * 3)

        def step():
            out = c.csa2_window_attn_tree(win, tree, q, drafts, SCALE, rope_out=True)
            c.csa2_verify_tree(tree, tok, toy.logits(out), accepted=accepted, next_token=following)
            c.csa2_window_accept_tree(win, tree, drafts, accepted)

        # once as it is, then captured and replayed from the same cache
        arrays = [t for t in (win.rows, win.codes, win.rope, win.scales, win.pos) if t is not None]
        before = [t.clone() for t in arrays]
        step()
        torch.cuda.synchronize()
        first = [t.clone() for t in arrays] + [accepted.clone(), following.clone()]
        for t, b in zip(arrays, before):
            t.copy_(b)
        accepted.zero_()
        following.zero_()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step()
        graph.replay()
        torch.cuda.synchronize()
        for t, b in zip(arrays + [accepted, following], first):
            assert torch.equal(t.view(torch.uint8), b.view(torch.uint8))
        for i, (a, f) in enumerate(zip(accepted.tolist(), following.tolist())):
            assert a == drafted[i][2], (i, at[i])
            at[i] += tree.depths[i][a] + 1
            assert f == said[i][at[i]], (i, at[i])
    # what the drafted run has kept is what the plain one has
    for i, s in enumerate(seqs):
        end = dev64([lens[i] + at[i]])
        want = filled()
        kept = said[i][:at[i]]
        c.csa2_window_append(want, toy.rows(kept, range(lens[i], lens[i] + at[i])), dev64([lens[i]]),
                             [at[i]], [s])
        got, ref = (c.csa2_window_read(x, end, swa, [s]) for x in (win, want))
        assert torch.equal(got, ref) and ref.any()
    assert win.device_error() == 0


def test_readme_window_example_runs():
    import os
    import re
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    blocks = re.findall(r"```python\n(.*?)```", open(os.path.join(root, "README.md")).read(), re.S)
    code, = [b for b in blocks if "C.Window(" in b]
    exec(compile(code, "README.md", "exec"), {})
