"""csa2_verify_tree against a walk in 64 bits written from the definition, at
the shapes, masks and trees where it can go wrong, and the distribution of the
tokens that come out."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu


def C():
    import fp4_kv_cache_index_gb300 as c
    return c


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def walk(parents, tokens, target, root, draft, draft_root, temp, u, noise):
    """(accepted, next token) of one tree; logits and numbers as CPU doubles."""
    def probs(row):
        if row.isnan().any() or (row == math.inf).any() or (row == -math.inf).all():
            return None
        if temp == 0:
            p = torch.zeros_like(row)
            p[int((row == row.max()).nonzero()[0])] = 1
            return p
        return torch.softmax(row / temp, 0)

    V, node, last = target.shape[1], -1, -1
    if root is None:
        if not parents:
            return -1, -1
        node = last = 0
    while True:
        p = probs(root if node < 0 else target[node])
        kids = [t for t, a in enumerate(parents) if a == node]
        if p is None:
            return last, -1
        q = None
        if draft is not None and kids and temp > 0:
            q = probs(draft_root if node < 0 else draft[node])
            if q is None:
                return last, -1
        taken = None
        for t in kids:
            x = int(tokens[t])
            if not 0 <= x < V:
                continue
            if temp == 0 or q is None:
                qq = torch.zeros(V, dtype=torch.float64)
                qq[x] = 1
            else:
                qq = q
            uu = 0.5 if temp == 0 else float(u[t])
            if uu * float(qq[x]) < float(p[x]):
                taken = t
                break
            rest = (p - qq).clamp(min=0)
            if float(rest.sum()) > 0:
                p = rest / rest.sum()
        if taken is None:
            s = p if temp == 0 else p / noise
            return last, int((s == s.max()).nonzero()[0])
        node = last = taken


def random_tree(n, seed, deep=0.5):
    import random
    rng = random.Random(seed)
    return [t - 1 if t and rng.random() < deep else rng.randrange(-1, t) for t in range(n)]


def make(parents, vocab, dtype, seed, ld=None, spread=3.0):
    """Logits, tokens and numbers for trees; rows `ld` apart."""
    S, nq = len(parents), sum(len(p) for p in parents)

    def rows(n, part, base=None):
        z = spread * torch.randn(n, vocab, generator=gen(seed + part), device="cuda")
        if base is not None:
            z = base.float() + 0.7 * torch.randn(n, vocab, generator=gen(seed + part), device="cuda")
        t = torch.full((n, ld or vocab), math.nan, dtype=dtype, device="cuda")[:, :vocab]
        return t.copy_(z)

    d = {"logits": rows(nq, 1), "root_logits": rows(S, 2)}
    d["draft_logits"], d["draft_root"] = rows(nq, 3, d["logits"]), rows(S, 4, d["root_logits"])
    d["temperature"] = torch.tensor([(0.0, 1.0, 0.6, 1.7)[(i + 1) % 4] for i in range(S)],
                                    device="cuda")
    d["uniform"] = torch.rand(nq, generator=gen(seed + 5), device="cuda")
    nz = torch.full((S, (ld or vocab) + 3), math.nan, device="cuda")[:, :vocab]
    d["noise"] = nz.copy_(torch.empty(S, vocab, device="cuda").exponential_(
        generator=gen(seed + 6)).clamp(min=1e-20))
    # likely tokens: the largest of their parent's draft logits, siblings alike
    # now and then
    tok, at = [], 0
    for i, ps in enumerate(parents):
        for t, p in enumerate(ps):
            row = d["draft_root"][i] if p < 0 else d["draft_logits"][at + p]
            k = min(vocab, 3)
            tok.append(int(row.float().topk(k)[1][(t * 7 + seed) % k]))
        at += len(ps)
    d["tokens"] = torch.tensor(tok, dtype=torch.int32, device="cuda")
    return d


def expect(parents, d):
    S, out, at = len(parents), [], 0
    cpu = {k: (None if v is None else v.cpu().double()) for k, v in d.items()}
    for i, ps in enumerate(parents):
        r = slice(at, at + len(ps))
        root = None if cpu["root_logits"] is None else cpu["root_logits"][i]
        dr = None if cpu.get("draft_logits") is None else cpu["draft_logits"][r]
        dq = None if cpu.get("draft_root") is None else cpu["draft_root"][i]
        temp = 0.0 if cpu["temperature"] is None else float(cpu["temperature"][i])
        out.append(walk(ps, cpu["tokens"][r], cpu["logits"][r], root, dr, dq, temp,
                        None if cpu["uniform"] is None else cpu["uniform"][r],
                        None if cpu["noise"] is None else cpu["noise"][i]))
        at += len(ps)
    return out


def run(parents, d, **more):
    c = C()
    acc, tok = c.csa2_verify_tree(c.Tree(parents, [0] * len(parents)), d["tokens"], d["logits"],
                                  d["temperature"], d["uniform"], d["noise"], d["root_logits"],
                                  d.get("draft_logits"), d.get("draft_root"), **more)
    return list(zip(acc.tolist(), tok.tolist()))


TREES = [[[-1, 0, 1, 2, 3]], [random_tree(9, i) for i in range(7)], [[], [-1], [-1, -1, -1]],
         [random_tree(64, 1, 0.3), random_tree(64, 2, 0.8), list(range(-1, 63)), [-1] * 64]]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("vocab,ld", [(1, None), (2, None), (7, 16), (257, None), (1000, 1001),
                                      (4096, 4104), (9000, None), (50257, None), (131072, None)])
@pytest.mark.parametrize("draft", ["logits", "certain"])
def test_walks(dtype, vocab, ld, draft):
    for k, parents in enumerate(TREES if vocab < 20000 else TREES[1:3]):
        d = make(parents, vocab, dtype, 100 * k, ld)
        if draft == "certain":
            d["draft_logits"] = d["draft_root"] = None
        assert run(parents, d) == expect(parents, d)
        # the root's child drawn by the step before
        one = [[-1] + [max(0, a) for a in p[1:]] if p else [] for p in parents]
        d["root_logits"] = d["draft_root"] = None
        assert run(one, d) == expect(one, d)


def test_many_sequences():
    """More trees than one launch's tables hold, with none and one draft among
    them; outputs given by the caller."""
    parents = [random_tree(i % 9, i) for i in range(1100)]
    d = make(parents, 300, torch.bfloat16, 5)
    acc = torch.full((1100,), 77, dtype=torch.int32, device="cuda")
    tok = torch.full((1100,), 77, dtype=torch.int32, device="cuda")
    want = expect(parents, d)
    assert run(parents, d, accepted=acc, next_token=tok) == want
    assert list(zip(acc.tolist(), tok.tolist())) == want


def test_greedy_alone_needs_no_numbers():
    """Largest logits, equal ones (bf16 has many) to the lower token."""
    parents = [random_tree(20, i) for i in range(6)]
    d = make(parents, 40000, torch.bfloat16, 9, spread=1.0)
    d["temperature"] = d["uniform"] = d["noise"] = d["draft_logits"] = d["draft_root"] = None
    d["logits"].clamp_(max=2.0)
    d["root_logits"].clamp_(max=2.0)
    at = 0
    for i, ps in enumerate(parents):   # some of the drafts are the first largest
        for t, p in enumerate(ps):
            row = d["root_logits"][i] if p < 0 else d["logits"][at + p]
            if t % 3:
                d["tokens"][at + t] = int((row == row.max()).nonzero()[0])
        at += len(ps)
    got = run(parents, d)
    assert got == expect(parents, d) and any(a >= 0 for a, _ in got)


@pytest.mark.parametrize("temperature", [0.0, 0.8])
def test_masked_and_broken_rows(temperature):
    """Masked tokens, rows with nothing left, NaN and infinities: the walk ends
    there, and rows that it does not come to do not matter."""
    V = 5000
    parents = [[-1, 0, 1]] * 8
    d = make(parents, V, torch.float32, 3)
    d["temperature"].fill_(temperature)
    d["uniform"].fill_(0.0)   # every draft with a probability is accepted
    for i in range(8):
        if temperature == 0:   # and is the largest
            rows = [d["root_logits"][i], d["logits"][3 * i], d["logits"][3 * i + 1]]
            for t, row in enumerate(rows):
                d["tokens"][3 * i + t] = int(row.argmax())
    d["root_logits"][0, 1:] = -math.inf             # one token is left, and it is drafted
    d["tokens"][0] = 0
    d["root_logits"][1] = -math.inf                 # none is
    d["logits"][6, 77] = math.nan                   # after the first draft of tree 2
    d["root_logits"][3, 4999] = math.inf
    d["logits"][3 * 4 + 2] = -math.inf              # after the last draft of tree 4
    d["draft_logits"][3 * 5 + 2] = math.nan         # a leaf's draft row: not read
    keep = int(d["tokens"][18])
    d["root_logits"][6, keep] = -math.inf           # a draft whose probability is 0
    d["tokens"][21] = 5000                          # outside the vocabulary
    if temperature:
        d["draft_root"][7, 0] = math.nan            # the draft row of a node that is tested
    want = expect(parents, d)
    assert run(parents, d) == want
    assert want[1] == (-1, -1) and want[2] == (0, -1) and want[3] == (-1, -1) and want[4] == (2, -1)
    assert want[5][0] == 2 and want[5][1] >= 0 and want[6][0] == -1


def test_siblings():
    """The same token twice, siblings that take all the mass, the largest uniform
    numbers."""
    V = 12
    parents = [[-1] * 6, [-1] * 6, [-1, -1, 0, 0, 0, 1]]
    top = 1 - 2.0 ** -24
    for seed in range(20):
        d = make(parents, V, torch.float32, 50 + seed)
        d["temperature"] = torch.tensor([1.0, 1.0, 0.7], device="cuda")
        d["tokens"] = torch.randint(0, 4, (18,), generator=gen(seed), device="cuda").int()
        d["uniform"] = torch.rand(18, generator=gen(99 + seed), device="cuda") * 0.5 + 0.5
        d["uniform"][::3] = top
        if seed % 2:
            d["draft_logits"] = d["draft_root"] = None
            d["root_logits"][0, 4:] = -math.inf   # all of the mass is drafted
        assert run(parents, d) == expect(parents, d), seed


def test_identical_models_accept_everything():
    """q = p: u q < p for every u below 1."""
    parents = [list(range(-1, 15))] * 40
    d = make(parents, 3001, torch.bfloat16, 3)
    d["draft_logits"], d["draft_root"] = d["logits"].clone(), d["root_logits"].clone()
    d["temperature"].fill_(1.1)
    d["uniform"].fill_(1 - 2.0 ** -24)
    got = run(parents, d)
    assert [a for a, _ in got] == [15] * 40 and got == expect(parents, d)


@pytest.mark.parametrize("kind", ["logits", "certain"])
@pytest.mark.parametrize("n_kids", [1, 3])
def test_tokens_are_distributed_as_the_target(kind, n_kids):
    """The first token of a step (the first accepted draft, or the next token) has
    the target's distribution, whatever the drafts' is.  Each of V counts of N
    draws is binomial: within 5 standard deviations (a probability of 6e-7 each
    under the normal law)."""
    c = C()
    V, N = 8, 1 << 16
    g = gen(11)
    target = torch.randn(V, generator=g, device="cuda") * 1.5
    draft = target + torch.randn(V, generator=g, device="cuda")
    q = torch.softmax(draft, 0)
    # drafts that count as certain may be drawn from anything: here from q
    tok = torch.multinomial(q, N * n_kids, True, generator=g).int()
    tree = c.Tree([[-1] * n_kids] * N, [0] * N)
    t, dr = target.expand(N, V).contiguous(), draft.expand(N, V).contiguous()
    kids = target.expand(N * n_kids, V).contiguous()
    acc, nxt = c.csa2_verify_tree(
        tree, tok, kids, torch.ones(N, device="cuda"), torch.rand(N * n_kids, generator=g, device="cuda"),
        torch.empty(N, V, device="cuda").exponential_(generator=g).clamp(min=1e-30), t,
        kids if kind == "logits" else None, dr if kind == "logits" else None)
    first = torch.where(acc >= 0, tok.view(N, n_kids).gather(1, acc.clamp(min=0).long()[:, None])[:, 0], nxt)
    p = torch.softmax(target.double(), 0)
    count = torch.bincount(first.long(), minlength=V).double()
    assert count.sum() == N
    assert ((count - N * p).abs() <= 5 * (N * p * (1 - p)).sqrt()).all(), (count / N, p)
    # of single drafts sum min(p, q) are accepted, or, where they count as
    # certain, sum p q
    qd = q.double()
    a = (torch.minimum(p, qd) if kind == "logits" else p * qd).sum()
    n = (acc >= 0).sum()
    if n_kids == 1:
        assert (n - N * a).abs() <= 5 * (N * a * (1 - a)).sqrt()
    else:
        assert N * a < n < N


def test_near_ties_are_decided_exactly():
    """Two candidates whose scores fp32 cannot tell apart."""
    V = 20000
    parents = [[]] * 64
    d = make(parents, V, torch.float32, 1)
    d["temperature"].fill_(0.9)
    for i in range(64):
        # the best token and another one given a noise that makes their scores
        # the same but for a part in 2^24
        p = torch.softmax(d["root_logits"][i].double() / 0.9, 0)
        s = p / d["noise"][i].double()
        a, b = s.topk(2)[1].tolist()
        d["noise"][i, b] = (p[b] / s[a]).float()
    d["temperature"].copy_(torch.full((64,), 0.9))
    got, want = run(parents, d), expect(parents, d)
    # the temperature is fp32: the reference takes the same one
    assert got == want


@pytest.mark.parametrize("kind", ["logits", "certain"])
def test_tests_at_their_border_are_decided_exactly(kind):
    """Uniform numbers next to the probability that they are compared with, nearer
    than fp32 can tell: first children, and second ones after a rejection."""
    V, S = 3000, 120
    parents = [[-1, -1, 0, 1]] * S
    d = make(parents, V, torch.float32, 31)
    d["temperature"].fill_(0.75)
    if kind == "certain":
        d["draft_logits"] = d["draft_root"] = None
    d["uniform"].fill_(0.999999)
    for i in range(S):
        p = torch.softmax(d["root_logits"][i].double() / 0.75, 0)
        x, y = d["tokens"][4 * i].item(), (d["tokens"][4 * i].item() + 1 + i) % V
        d["tokens"][4 * i + 1] = y
        if kind == "certain":
            q = torch.zeros_like(p)
            q[x] = 1
        else:
            q = torch.softmax(d["draft_root"][i].double() / 0.75, 0)
        if i % 2 == 0:
            u, c = (p[x] / q[x]).item(), 4 * i
        else:
            rest = (p - q).clamp(min=0)
            rest /= rest.sum()
            u, c = (rest[y] / (1.0 if kind == "certain" else q[y])).item(), 4 * i + 1
        u = torch.tensor(u if u < 0.9 else 0.5, dtype=torch.float32)
        for _ in range(i % 3):
            u = torch.nextafter(u, torch.tensor(float(i % 4 < 2)))
        d["uniform"][c] = u
    got, want = run(parents, d), expect(parents, d)
    assert got == want
    assert 10 < sum(a >= 0 for a, _ in want) < S


def test_strides_streams_and_graphs():
    c = C()
    parents = [random_tree(6, i) for i in range(5)]
    d = make(parents, 3001, torch.bfloat16, 21, ld=3008)
    want = expect(parents, d)
    assert run(parents, d) == want
    tree = c.Tree(parents, [0] * 5)
    acc, tok = (torch.empty(5, dtype=torch.int32, device="cuda") for _ in range(2))

    def call(stream=None):
        c.csa2_verify_tree(tree, d["tokens"], d["logits"], d["temperature"], d["uniform"], d["noise"],
                           d["root_logits"], d["draft_logits"], d["draft_root"], acc, tok,
                           stream=stream)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    call(s)
    s.synchronize()
    assert list(zip(acc.tolist(), tok.tolist())) == want
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    e = make(parents, 3001, torch.bfloat16, 22, ld=3008)
    for k, v in e.items():
        d[k].copy_(v)
    acc.fill_(9)
    g.replay()
    assert list(zip(acc.tolist(), tok.tolist())) == expect(parents, d)


def test_refusals():
    c = C()
    parents = [[-1, 0], [-1]]
    tree = c.Tree(parents, [0, 0])
    d = make(parents, 100, torch.bfloat16, 1)

    def call(**change):
        e = dict(d, **change)
        return c.csa2_verify_tree(e.get("tree", tree), e["tokens"], e["logits"], e["temperature"],
                                  e["uniform"], e["noise"], e["root_logits"], e["draft_logits"],
                                  e["draft_root"])
    call()
    two_roots = c.Tree([[-1, -1], [-1]], [0, 0])
    wide = torch.zeros(3, 200, dtype=torch.bfloat16, device="cuda")[:, :100]
    for change in (dict(tokens=d["tokens"].long()), dict(tokens=d["tokens"][:2]),
                   dict(logits=d["logits"].half()), dict(logits=wide), dict(logits=d["logits"][:2]),
                   dict(root_logits=d["root_logits"].float()), dict(uniform=None), dict(noise=None),
                   dict(noise=d["noise"][:1]), dict(temperature=d["temperature"].double()),
                   dict(draft_root=None), dict(draft_logits=None), dict(root_logits=None),
                   dict(logits=d["logits"].cpu()), dict(logits=d["logits"].t()),
                   dict(tree=two_roots, root_logits=None, draft_root=None)):
        with pytest.raises((ValueError, RuntimeError)):
            call(**change)
            pytest.fail(str(change))
