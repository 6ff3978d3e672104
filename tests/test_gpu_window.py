"""Window rows in a cache and the attention of window layers over them, against
64-bit references: rounding, places, what a query sees, masks, orders, streams
and graphs.

Tolerance of an output o = sum_x p_x v_x.  The probabilities are rounded to
bf16 (half a step, 2^-8 relative) in the sum as in the product, so a weight is
off by up to 2 * 2^-8 of itself and o by 2^-7 * sum p |v|; the output is
rounded once (2^-8 |o|); the logits' fp32 sums of 512 products (of the order
of 1 after scaling) move the weights by less than 2^-12.  lse: the sum of
rounded probabilities is off by 2^-8 relative at most, so is exp(lse)."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu
SCALE = 512 ** -0.5


def C():
    import fp4_kv_cache_index_gb300 as c
    return c


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def make_rows(n, seed):
    return (torch.randn(n, 512, generator=gen(seed), device="cuda") *
            torch.exp(0.5 * torch.randn(512, generator=gen(seed + 1), device="cuda"))).bfloat16()


def make_q(n, heads, seed):
    return torch.randn(n, heads, 512, generator=gen(seed), device="cuda").bfloat16()


def dev64(xs):
    return torch.tensor(xs, dtype=torch.int64, device="cuda")


def power_below(x):
    return (x.view(torch.int64) >> 52 << 52).view(torch.float64)


def round8(rows):
    """Rows as 8 bits hold them, in 64 bits, from the format's definition."""
    x = rows.double()
    v = x[:, :448].reshape(-1, 7, 64)
    top = v.abs().amax(-1, keepdim=True)
    s = torch.where(top > 0, power_below(top) / 256, 1.0)
    a = (v / s).clamp(-448, 448)
    step = power_below(a.abs().clamp(min=2.0 ** -6)) / 8
    return torch.cat([(torch.round(a / step) * step * s).reshape(-1, 448), x[:, 448:]], 1)


class Model:
    """A cache as a dict of the rows that it is given, by sequence and position."""

    def __init__(self, n_seqs, swa, n_first, fp8):
        self.swa, self.n_first, self.fp8 = swa, n_first, fp8
        self.held = [{} for _ in range(n_seqs)]

    def append(self, rows, pos, counts, seqs):
        vals = round8(rows) if self.fp8 else rows.double()
        at = 0
        for p, n, s in zip(pos, counts, seqs):
            for k in range(n):
                if p >= 0:
                    self.held[s][p + k] = vals[at + k]
            at += n

    def seen(self, seq, p):
        """Positions and rows that a query at position p sees."""
        xs = [x for x in self.held[seq] if x <= p and (p - x < self.swa or x < self.n_first)]
        return sorted(xs)


def attend(q, kv, scale=SCALE, sink=None, at=None, base=10000.0):
    """(out, lse, weight) of one query [heads, 512] over rows kv [n, 512], in 64
    bits; weight: sum p |v|."""
    h = q.shape[0]
    x = q.double() @ kv.T * scale if kv.shape[0] else torch.zeros(h, 0, device="cuda").double()
    if sink is not None:
        x = torch.cat([x, sink.double()[:, None]], 1)
    if x.shape[1] == 0:
        z = torch.zeros(h, 512, dtype=torch.float64, device="cuda")
        return z, torch.full((h,), -math.inf, device="cuda").double(), z
    p = torch.softmax(x, 1)[:, :kv.shape[0]]
    out, weight = p @ kv, p @ kv.abs()
    if at is not None:
        t = torch.arange(32, device="cuda", dtype=torch.float64)
        ang = -float(at) * base ** (-t / 32)
        a, b = out[:, 448::2].clone(), out[:, 449::2].clone()
        out[:, 448::2] = a * ang.cos() - b * ang.sin()
        out[:, 449::2] = a * ang.sin() + b * ang.cos()
        w = weight[:, 448::2] + weight[:, 449::2]
        weight[:, 448::2] = weight[:, 449::2] = w
    return out, torch.logsumexp(x, 1), weight


def check(out, lse, ref):
    o, l, w = ref
    tol = 2.0 ** -8 * o.abs() + (2.0 ** -7 + 2.0 ** -11) * w + 1e-30
    bad = (out.double() - o).abs() > tol
    assert not bad.any(), ((out.double() - o).abs() / tol).max().item()
    if lse is not None:
        inf = torch.isinf(l)
        assert torch.equal(torch.isinf(lse), inf)
        assert ((lse.double() - l)[~inf].abs() <= 2.0 ** -7.9 + 1e-5).all()


# ------------------------------------------------------------------ rows
@pytest.mark.parametrize("fp8", [True, False])
@pytest.mark.parametrize("swa,n_first", [(128, 0), (128, 8), (7, 3), (1, 1), (100, 5)])
def test_append_and_read(fp8, swa, n_first):
    c = C()
    n_seqs = 5
    win, model = c.Window(n_seqs, swa, n_first, fp8), Model(n_seqs, swa, n_first, fp8)
    # prompts of many lengths (none, one, the window's and more), then steps; a
    # sequence that starts late, one that is not stored
    steps = [([0, 3, 1, 4], [0, 0, 0, 0], [swa + 50, 1, swa, 3 * swa + 1]),
             ([4, 1], [3 * swa + 1, swa], [2, 0]),
             ([2], [10 ** 10 + 3], [swa // 2 + 1]),
             (None, [swa + 50, swa, -1, 1, 3 * swa + 3], None),
             ([0], [-5], [4])]
    end = [0] * n_seqs
    for k, (seqs, pos, counts) in enumerate(steps):
        ids = list(range(n_seqs)) if seqs is None else seqs
        n = [1] * len(ids) if counts is None else counts
        rows = make_rows(sum(n), 10 * k)
        rows[:1] *= 2.0 ** -100
        rows[-1, 64:128] = 0
        rounded = torch.full_like(rows, 7)
        c.csa2_window_append(win, rows, dev64(pos), counts, seqs, rounded=rounded)
        model.append(rows, pos, n, ids)
        want = round8(rows) if fp8 else rows.double()
        assert torch.equal(rounded.double(), want)
        for s, p, m in zip(ids, pos, n):
            if p >= 0 and m:
                end[s] = max(end[s], p + m)
    # in place, nothing stored
    rows = make_rows(3, 99)
    want = round8(rows) if fp8 else rows.double()
    c.csa2_window_append(win, rows, dev64([-1]), [3], [2], rounded=rows)
    assert torch.equal(rows.double(), want)

    for n_rows in {1, max(1, swa // 2), swa}:
        order = [4, 0, 0, 2, 3, 1]
        ends = [end[4], end[0], max(0, end[0] - 1), end[2], end[3], 0]
        first = torch.full((len(order), n_first, 512), 7, dtype=torch.bfloat16, device="cuda")
        got = c.csa2_window_read(win, dev64(ends), n_rows, order, first=first if n_first else None)
        f8 = c.csa2_window_read(win, dev64(ends), n_rows, order, fp8=True) if fp8 else None
        for i, (s, e) in enumerate(zip(order, ends)):
            # a ring holds the newest swa rows only
            held = {x: v for x, v in model.held[s].items() if x > end[s] - 1 - swa}
            for j in range(n_rows):
                x = max(0, e - n_rows) + j
                want = held[x] if x < e and x in held else torch.zeros(512, device="cuda")
                assert torch.equal(got[i, j].double(), want.double()), (i, j)
            for f in range(n_first):
                v = model.held[s].get(f) if f < e else None
                assert torch.equal(first[i, f].double(), torch.zeros(512, device="cuda").double()
                                   if v is None else v)
        if fp8:   # the codes are those of the quantiser
            flat = got.view(-1, 512)
            for a, b in zip(f8, c.csa2_swa_fp8_quantise(flat)):
                live = (flat != 0).any(1)
                assert torch.equal(a[live], b[live])
    assert win.device_error() == 0
    win.reset(0)
    assert not c.csa2_window_read(win, dev64([end[0]]), swa, [0]).any()
    assert c.csa2_window_read(win, dev64([end[4]]), swa, [4]).any()


def test_append_leaves_the_rest_of_the_cache():
    c = C()
    win = c.Window(3, 16, 2)
    for t in (win.codes, win.scales):
        t.fill_(0xA5)
    win.rope.fill_(3.0)
    before = [t.clone() for t in (win.codes, win.rope, win.scales, win.pos)]
    c.csa2_window_append(win, make_rows(5, 1), dev64([30]), [5], [1])
    hit = {16 + x % 16 for x in range(30, 35)}
    for t, b in zip((win.codes, win.rope, win.scales, win.pos), before):
        for r in range(t.shape[0]):
            assert torch.equal(t[r], b[r]) == (r not in hit), r


def test_large_tables():
    """More segments than one launch's tables hold."""
    c = C()
    n = 5000
    win = c.Window(n, 4)
    ids = list(range(n - 1, -1, -1))
    rows = make_rows(2 * n, 3)
    c.csa2_window_append(win, rows, dev64([3 * s for s in ids]), [2] * n, ids)
    got = c.csa2_window_read(win, dev64([3 * s + 2 for s in ids]), 2, ids)
    assert torch.equal(got.view(-1, 512).double(), round8(rows))
    q = make_q(n, 64, 4)
    out = c.csa2_window_attn_decode(win, q, dev64([3 * s + 1 for s in ids]), SCALE, seq_ids=ids)
    for i in (0, 1, 4095, 4096, n - 1):
        check(out[i], None, attend(q[i], got[i].double()))


def test_rows_behind_the_last_position():
    """Positions end at 2^63 - 1: rows behind it are rounded, and not stored."""
    c = C()
    win = c.Window(3, 4, 2, False)
    win.rows.fill_(3.0)
    top = 2 ** 63 - 1
    rows = make_rows(9, 1)
    rounded = torch.empty_like(rows)
    # the newest four of the segment are 2^63 - 2 .. and two that are none
    c.csa2_window_append(win, rows[:4].contiguous(), dev64([top - 1]), [4], [1], rounded=rounded[:4])
    assert torch.equal(rounded[:4], rows[:4])
    for x, row in ((top - 1, rows[0]), (top, rows[1])):
        at = 4 + x % 4
        assert win.pos[at].item() == x and torch.equal(win.rows[at], row)
    kept = [4 + x % 4 for x in (top - 1, top)]
    assert all((win.rows[r] == 3.0).all() for r in range(win.rows.shape[0]) if r not in kept)
    q = make_q(1, 64, 2)
    out = c.csa2_window_attn_decode(win, q, dev64([top]), SCALE, [1])
    check(out[0], None, attend(q[0], rows[:2].double()))
    assert win.device_error() == 0


# ------------------------------------------------------------------ one token a sequence
@pytest.mark.parametrize("heads,swa,n_first,fp8,extra", [
    (64, 128, 4, True, False), (64, 128, 0, False, True), (128, 128, 8, True, True),
    (128, 96, 1, False, False), (64, 1, 0, True, True), (64, 5, 8, False, True),
    (128, 127, 2, True, False)])
def test_decode(heads, swa, n_first, fp8, extra):
    c = C()
    # lengths before the query's own token; None: a query that sees nothing
    lens = [0, 1, 2, swa - 1, swa, swa + 1, 700, 2 ** 33 + 11, None, 5]
    S = len(lens)
    win, model = c.Window(S, swa, n_first, fp8), Model(S, swa, n_first, fp8)
    for part in range(2):   # first tokens, then the newest rows and the query's own
        ids, pos, counts = [], [], []
        for s, n in enumerate(lens):
            if n is None:
                continue
            a, b = (0, min(n, n_first)) if part == 0 else (max(0, n - swa - 3), n + 1)
            ids.append(s)
            pos.append(a)
            counts.append(b - a)
        rows = make_rows(sum(counts), 5 + part)
        c.csa2_window_append(win, rows, dev64(pos), counts, ids)
        model.append(rows, pos, counts, ids)
    sink = torch.randn(heads, generator=gen(3), device="cuda") if extra else None
    # two queries of one sequence, and sequences out of order
    order = [9, 0, 1, 2, 3, 4, 5, 6, 6, 7, 8]
    at = [-1 if lens[s] is None else lens[s] for s in order]
    q = make_q(len(order), heads, 7)
    lse = torch.full((len(order), heads), 9.0, device="cuda")
    out = c.csa2_window_attn_decode(win, q, dev64(at), SCALE, seq_ids=order, lse=lse, sink=sink,
                                    rope_out=extra)
    for i, (s, p) in enumerate(zip(order, at)):
        # the ring has only the newest rows, the first tokens their own place
        xs = [] if p < 0 else model.seen(s, p)
        kv = torch.stack([model.held[s][x] for x in xs]) if xs else torch.zeros(0, 512, device="cuda").double()
        far = extra and p < 2 ** 30   # a far position's angle is off by 2^-51 of it
        if extra and not far:
            continue
        check(out[i], lse[i], attend(q[i], kv, sink=sink, at=p if extra else None))
    none = order.index(8)
    assert not out[none].any()
    assert torch.equal(lse[none], sink if extra else torch.full((heads,), -math.inf, device="cuda"))
    assert win.device_error() == 0


@pytest.mark.parametrize("heads", [64, 128])
def test_every_code_and_scale(heads):
    """A query that sees one row answers that row: all codes but the NaNs, scales from
    2^-126 to where bf16 ends, exact.  (Below, a bf16 has fewer bits.)"""
    c = C()
    code = torch.tensor([x for x in range(256) if x & 0x7F != 0x7F], dtype=torch.uint8, device="cuda")
    # byte b: 2^(b - 127); the largest code is 448 < 2^9, the least 2^-9
    bytes_ = [10, 64, 118, 127, 133, 134, 135, 136, 200, 244, 245]
    win = c.Window(len(bytes_), 1)
    win.codes.copy_(code.repeat(2)[:448].expand(len(bytes_), 448))
    win.scales.copy_(torch.tensor(bytes_, dtype=torch.uint8, device="cuda")[:, None].expand(-1, 8))
    win.rope.copy_(torch.randn(len(bytes_), 64, generator=gen(1), device="cuda"))
    win.pos.zero_()
    q = torch.zeros(len(bytes_), heads, 512, dtype=torch.bfloat16, device="cuda")
    out = c.csa2_window_attn_decode(win, q, dev64([0] * len(bytes_)), SCALE)
    x = code.repeat(2)[:448].long()
    e, m, sign = (x >> 3) & 15, x & 7, 1.0 - 2.0 * (x >> 7).double()
    power = ((e - 10 + 1023) << 52).view(torch.float64)   # 2^(e - 10), from its bits
    value = sign * torch.where(e > 0, (8 + m).double() * power, m.double() * 2.0 ** -9)
    for i, b in enumerate(bytes_):
        want = torch.cat([value * 2.0 ** (b - 127), win.rope[i].double()])
        assert torch.equal(out[i].double(), want.expand(heads, 512)), b
    # the same rows of a tree's draft
    tree = c.Tree([[-1]] * len(bytes_), [0] * len(bytes_))
    again = c.csa2_window_attn_tree(win, tree, q, (win.codes, win.rope, win.scales), SCALE)
    assert torch.equal(again, out)


def test_rows_that_are_not_held_are_not_seen():
    """Stale, missing and never written rows, NaN in all of them."""
    c = C()
    for fp8 in (True, False):
        win = c.Window(2, 128, 4, fp8)
        for t in (win.rows, win.rope) if not fp8 else (win.rope,):
            if t is not None:
                t.fill_(math.nan)
        if fp8:
            win.codes.fill_(0x7F)
            win.scales.fill_(0xFE)
        # an old sequence's rows at later positions, then a new one in their place
        c.csa2_window_append(win, make_rows(40, 1), dev64([300]), [40], [1])
        rows = make_rows(20, 2)
        c.csa2_window_append(win, rows, dev64([150]), [20], [1])
        q = make_q(1, 64, 3)
        kv = round8(rows) if fp8 else rows.double()
        for p in (160, 169, 175):
            out = c.csa2_window_attn_decode(win, q, dev64([p]), SCALE, seq_ids=[1])
            check(out[0], None, attend(q[0], kv[:p - 149]))
        # the window has moved on past all of it
        out = c.csa2_window_attn_decode(win, q, dev64([1000]), SCALE, seq_ids=[1])
        assert not out.any()


def test_nan_in_8_bits():
    """A row that held a NaN keeps it (the code of all ones, of either sign)."""
    c = C()
    win = c.Window(2, 128)
    rows = make_rows(40, 1)
    rows[30, 64 * 3 + 5] = math.nan
    rows[31, 447] = -math.nan
    rounded = torch.empty_like(rows)
    c.csa2_window_append(win, rows, dev64([0, 0]), [20, 20], rounded=rounded)
    assert rounded[30].isnan().sum() == 1 and rounded[31].isnan().sum() == 1
    q = make_q(2, 64, 2)
    out = c.csa2_window_attn_decode(win, q, dev64([19, 19]), SCALE)
    check(out[0], None, attend(q[0], round8(rows[:20])))
    assert out[1].isnan().all()


def test_values_that_are_not_finite():
    """A NaN or an infinity of a query's own stays with that query."""
    c = C()
    win = c.Window(3, 128, 0, False)
    rows = make_rows(3 * 60, 1)
    rows[70, 5] = math.nan
    c.csa2_window_append(win, rows, dev64([0, 0, 0]), [60] * 3)
    q = make_q(3, 64, 2)
    q[2, 7, 100] = math.inf
    out = c.csa2_window_attn_decode(win, q, dev64([59] * 3), SCALE)
    check(out[0], None, attend(q[0], rows[:60].double()))
    assert out[1].isnan().all()
    assert out[2, 7].isnan().all()
    keep = [h for h in range(64) if h != 7]
    check(out[2, keep], None, attend(q[2, keep], rows[120:].double()))


@pytest.mark.parametrize("scale", [0.0, -0.05, 3.0])
def test_scales(scale):
    """Any finite scale; with a large one the softmax takes one row."""
    c = C()
    win = c.Window(1, 128, 0, False)
    rows = make_rows(100, 1)
    c.csa2_window_append(win, rows, dev64([0]), [100])
    q = (0.125 * make_q(1, 64, 2).float()).bfloat16()
    lse = torch.empty(1, 64, device="cuda")
    out = c.csa2_window_attn_decode(win, q, dev64([99]), scale, lse=lse)
    o, l, w = attend(q[0], rows.double(), scale)
    # logits of some tens: a few 2^-24 of that, far below 2^-9
    tol = 2.0 ** -8 * o.abs() + (2.0 ** -7 + 2.0 ** -9) * w
    assert ((out[0].double() - o).abs() <= tol).all()


# ------------------------------------------------------------------ trees
def random_tree(n, seed):
    import random
    rng = random.Random(seed)
    return [t - 1 if t and rng.random() < 0.5 else rng.randrange(-1, t) for t in range(n)]


def tree_rows(model, tree, i, t, rows, first):
    """The rows that draft t of tree i sees; its tree's rows begin at `first`."""
    seq, pos0 = i if tree._seq is None else tree._seq[i], tree.pos0[i]
    path = [k for k in range(t + 1) if (tree.paths[i][t] >> k) & 1]
    vals = rows[[first + k for k in path]]
    vals = round8(vals) if model.fp8 else vals.double()
    held = {**{x: v for x, v in model.held[seq].items() if x < pos0},
            **{pos0 + j: v for j, v in enumerate(vals)}}
    p = pos0 + len(path) - 1
    xs = sorted(x for x in held if p - x < model.swa or x < model.n_first)
    return torch.stack([held[x] for x in xs])


@pytest.mark.parametrize("heads,swa,n_first,fp8", [(64, 128, 4, True), (128, 128, 0, False),
                                                   (64, 9, 8, False), (128, 70, 3, True)])
def test_tree_is_decoding_its_paths(heads, swa, n_first, fp8):
    """A tree's drafts, and their paths appended and decoded token by token."""
    c = C()
    pos0 = [0, 1, 150, 6, 2 ** 31 + 77]
    parents = [random_tree(12, 1), random_tree(64, 2), list(range(-1, 63)), [], random_tree(30, 4)]
    seqs = [3, 0, 4, 1, 2]
    tree = c.Tree(parents, pos0, seqs)
    win, model = c.Window(5, swa, n_first, fp8), Model(5, swa, n_first, fp8)
    counts = [min(p, swa + 5) for p in pos0]
    head = [min(p, n_first) for p in pos0]
    for k, (n, at) in enumerate(((head, [0] * 5), (counts, [p - n for p, n in zip(pos0, counts)]))):
        before = make_rows(sum(n), 5 + k)
        c.csa2_window_append(win, before, dev64(at), n, seqs)
        model.append(before, at, n, seqs)
    nq = tree.n_queries
    q, rows = make_q(nq, heads, 8), make_rows(nq, 9)
    draft = c.csa2_swa_fp8_quantise(rows) if fp8 else rows
    sink = torch.randn(heads, generator=gen(3), device="cuda")
    lse = torch.empty(nq, heads, device="cuda")
    out = c.csa2_window_attn_tree(win, tree, q, draft, SCALE, lse=lse, sink=sink, rope_out=True)
    held = [t.clone() for t in (win.codes, win.rope, win.scales, win.rows, win.pos) if t is not None]
    arrays = [t for t in (win.codes, win.rope, win.scales, win.rows, win.pos) if t is not None]
    first = 0
    for i, par in enumerate(parents):
        for t in range(len(par)):
            path = [k for k in range(t + 1) if (tree.paths[i][t] >> k) & 1]
            for a, b in zip(arrays, held):
                a.copy_(b)
            c.csa2_window_append(win, rows[[first + k for k in path]].contiguous(),
                                 dev64([pos0[i]]), [len(path)], [seqs[i]])
            l1 = torch.empty(1, heads, device="cuda")
            one = c.csa2_window_attn_decode(win, q[first + t:first + t + 1].contiguous(),
                                            dev64([pos0[i] + len(path) - 1]), SCALE, [seqs[i]],
                                            lse=l1, sink=sink, rope_out=True)
            if heads == 128:   # one query an item: the same sums in the same order
                assert torch.equal(one[0], out[first + t]) and torch.equal(l1[0], lse[first + t]), (i, t)
            ref = attend(q[first + t], tree_rows(model, tree, i, t, rows, first), sink=sink,
                         at=pos0[i] + len(path) - 1)
            check(out[first + t], lse[first + t], ref)
            check(one[0], l1[0], ref)
        first += len(par)
    # acceptance writes what appending the path writes
    for a, b in zip(arrays, held):
        a.copy_(b)
    accepted = [5, 60, 63, -1, 64]   # the last one is no draft: nothing
    c.csa2_window_accept_tree(win, tree, draft,
                              torch.tensor(accepted, dtype=torch.int32, device="cuda"))
    got = [t.clone() for t in arrays]
    for a, b in zip(arrays, held):
        a.copy_(b)
    first = 0
    for i, par in enumerate(parents):
        if 0 <= accepted[i] < len(par):
            path = [k for k in range(len(par)) if (tree.paths[i][accepted[i]] >> k) & 1]
            c.csa2_window_append(win, rows[[first + k for k in path]].contiguous(),
                                 dev64([pos0[i]]), [len(path)], [seqs[i]])
        first += len(par)
    bits = lambda t: t.view(torch.uint8)   # memory that was never written may hold NaN
    assert all(torch.equal(bits(a), bits(b)) for a, b in zip(arrays, got))


def test_many_trees():
    """More drafts than one launch's tables hold."""
    c = C()
    n = 600
    parents = [random_tree(1 + i % 7, i) for i in range(n)]
    tree = c.Tree(parents, [10 + i for i in range(n)])
    win, model = c.Window(n, 8, 1, False), Model(n, 8, 1, False)
    before = make_rows(n * 10, 1)
    c.csa2_window_append(win, before, dev64([i for i in range(n)]), [10] * n)
    model.append(before, list(range(n)), [10] * n, range(n))
    q, rows = make_q(tree.n_queries, 64, 2), make_rows(tree.n_queries, 3)
    out = c.csa2_window_attn_tree(win, tree, q, rows, SCALE)
    acc = [len(p) - 1 for p in parents]
    c.csa2_window_accept_tree(win, tree, rows, torch.tensor(acc, dtype=torch.int32, device="cuda"))
    last = [sum(len(p) for p in parents[:i + 1]) - 1 for i in range(n)]
    at = dev64([10 + i + tree.depths[i][-1] for i in range(n)])
    again = c.csa2_window_attn_decode(win, q[last].contiguous(), at, SCALE)
    for i, x in enumerate(last):
        kv = tree_rows(model, tree, i, acc[i], rows, x - acc[i])
        ref = attend(q[x], kv)
        check(out[x], None, ref)
        check(again[i], None, ref)


@pytest.mark.parametrize("heads", [64, 128])
@pytest.mark.parametrize("fp8", [True, False])
@pytest.mark.parametrize("swa,n_first", [(128, 8), (128, 0), (1, 0), (3, 2), (64, 5)])
def test_branches(swa, n_first, fp8, heads):
    """Neighbouring drafts of all kinds: of one parent, of far branches, deep and
    shallow in turn; NaN and an infinity of a draft reach those who see it only."""
    c = C()
    star, comb = [-1] * 64, [x for k in range(32) for x in (2 * k - 2 if k else -1, 2 * k - 2 if k else -1)]
    deep = list(range(-1, 29)) + [-1, 4, 31, 32, 33, 34, 35, 36, 37, 38, 39, 40, 41, 10, 43]
    parents = [star, comb, deep, random_tree(64, 5), [-1], [-1, -1], [-1, 0, -1]]
    pos0 = [200, 5, 0, 1000, 3, 64, 131]
    bad = [7, 20, 12, 33, None, 1, 0]     # a draft of each tree
    S = len(parents)
    tree = c.Tree(parents, pos0)
    win, model = c.Window(S, swa, n_first, fp8), Model(S, swa, n_first, fp8)
    for part in range(2):
        n = [min(p, n_first if part == 0 else swa) for p in pos0]
        at = [0 if part == 0 else p - k for p, k in zip(pos0, n)]
        before = make_rows(sum(n), 20 + part)
        c.csa2_window_append(win, before, dev64(at), n)
        model.append(before, at, n, range(S))
    q, rows = make_q(tree.n_queries, heads, 8), make_rows(tree.n_queries, 9)
    starts = [sum(len(p) for p in parents[:i]) for i in range(S)]
    draft_rows = rows.clone()
    for i, b in enumerate(bad):
        if b is not None:
            draft_rows[starts[i] + b, 13 * i] = math.nan if fp8 or i % 2 else math.inf
    draft = c.csa2_swa_fp8_quantise(draft_rows) if fp8 else draft_rows
    lse = torch.empty(tree.n_queries, heads, device="cuda")
    out = c.csa2_window_attn_tree(win, tree, q, draft, SCALE, lse=lse)
    for i, par in enumerate(parents):
        for t in range(len(par)):
            x = starts[i] + t
            b = bad[i]
            on = b is not None and (tree.paths[i][t] >> b) & 1
            far = on and tree.depths[i][t] - tree.depths[i][b]   # behind the query
            if on and (far < swa or pos0[i] + tree.depths[i][b] < n_first):
                assert out[x].isnan().all() and lse[x].isnan().all(), (i, t)
            else:
                check(out[x], lse[x], attend(q[x], tree_rows(model, tree, i, t, rows, starts[i])))
    assert win.device_error() == 0


# ------------------------------------------------------------------ chunks
@pytest.mark.parametrize("heads,swa,n_first,pos0,n", [
    (64, 128, 4, 0, 1), (64, 128, 4, 0, 2), (64, 128, 0, 0, 301), (128, 128, 8, 0, 40),
    (64, 128, 4, 3, 5), (64, 128, 4, 1000, 1), (64, 96, 3, 777, 250), (128, 1, 0, 5, 33),
    (64, 17, 8, 2, 64), (64, 128, 1, 2 ** 40 + 1, 131), (128, 128, 5, 129, 160)])
def test_chunk(heads, swa, n_first, pos0, n):
    c = C()
    back = min(swa - 1, pos0)
    band0 = pos0 - back
    band = make_rows(back + n, 1)
    first = make_rows(n_first, 2) if n_first and band0 else None
    sink = torch.randn(heads, generator=gen(3), device="cuda")
    q = make_q(n, heads, 4)
    lse = torch.empty(n, heads, device="cuda")
    rope = pos0 < 2 ** 30
    out = c.csa2_window_attn_prefill(q, pos0, band, band0, SCALE, swa, n_first, first, lse=lse,
                                     sink=sink, rope_out=rope)
    for i in sorted({0, 1, 2, 3, 7, 8, n // 2, n - 2, n - 1} & set(range(n))):
        p = pos0 + i
        xs = [x for x in range(band0, p + 1) if p - x < swa or x < n_first]
        kv = [band[x - band0] for x in xs]
        if first is not None:
            kv = [first[f] for f in range(min(n_first, band0))] + kv
        check(out[i], lse[i], attend(q[i], torch.stack(kv).double(), sink=sink, at=p if rope else None))


@pytest.mark.parametrize("heads,n", [(64, 6001), (128, 2000)])
def test_long_chunk(heads, n):
    """Many items a CTA: bit for bit what short chunks over the same rows give."""
    c = C()
    rows, q = make_rows(n + 100, 1), make_q(n, heads, 2)
    first = make_rows(4, 3)
    whole = c.csa2_window_attn_prefill(q, 1100, rows, 1000, SCALE, 90, 4, first)
    for a in range(0, n, 200):
        b = min(n, a + 200)
        back = min(89, a + 100)
        part = c.csa2_window_attn_prefill(q[a:b], 1100 + a, rows[a + 100 - back:b + 100],
                                          1100 + a - back, SCALE, 90, 4, first)
        assert torch.equal(part, whole[a:b]), a
    for i in (0, 1, n // 2, n - 1):
        kv = torch.cat([first, rows[max(0, i + 11):i + 101]]).double()
        check(whole[i], None, attend(q[i], kv))


@pytest.mark.parametrize("fp8", [True, False])
def test_chunks_of_any_length_agree(fp8):
    """A prompt in chunks gives bit for bit what it gives as a whole, through the
    cache as an engine would run it; decoding its tokens gives nearly that."""
    c = C()
    n, swa, F, H = 400, 128, 4, 64
    rows, q = make_rows(n, 1), make_q(n, H, 2)
    win = c.Window(1, swa, F, fp8)
    rounded = torch.empty_like(rows)
    c.csa2_window_append(win, rows, dev64([0]), [n], rounded=rounded)
    whole = c.csa2_window_attn_prefill(q, 0, rounded, 0, SCALE, swa, F)
    win.reset()
    at, parts = 0, []
    for m in (1, 2, 127, 130, 9, 131):
        back = min(swa - 1, at)
        band = torch.empty(back + m, 512, dtype=torch.bfloat16, device="cuda")
        first = torch.empty(1, F, 512, dtype=torch.bfloat16, device="cuda")
        if back:
            c.csa2_window_read(win, dev64([at]), back, out=band[:back].view(1, back, 512), first=first)
        c.csa2_window_append(win, rows[at:at + m], dev64([at]), [m], rounded=band[back:])
        parts.append(c.csa2_window_attn_prefill(q[at:at + m], at, band, at - back, SCALE, swa, F,
                                                first[0], error=win.error))
        at += m
    assert at == n and torch.equal(torch.cat(parts), whole)
    assert win.device_error() == 0
    # token by token
    one = c.Window(1, swa, F, fp8)
    for p in range(n):
        c.csa2_window_append(one, rows[p:p + 1], dev64([p]))
        if p in (0, 1, 126, 127, 128, 129, 399):
            out = c.csa2_window_attn_decode(one, q[p:p + 1].contiguous(), dev64([p]), SCALE)
            xs = [x for x in range(p + 1) if p - x < swa or x < F]
            ref = attend(q[p], rounded[xs].double())
            check(out[0], None, ref)
            check(whole[p], None, ref)


def test_chunk_rows_that_are_not_finite():
    """NaN and infinities of a row reach the queries that see it, no other:
    not the ones before it nor those whose window has passed it."""
    c = C()
    n, swa = 300, 128
    rows, q = make_rows(n, 1), make_q(n, 64, 2)
    clean = c.csa2_window_attn_prefill(q, 0, rows, 0, SCALE, swa, 2)
    for at, value in ((100, math.nan), (7, math.inf), (299, -math.inf), (1, math.nan)):
        bad = rows.clone()
        bad[at, 3] = value
        out = c.csa2_window_attn_prefill(q, 0, bad, 0, SCALE, swa, 2)
        sees = torch.tensor([p >= at and (p - at < swa or at < 2) for p in range(n)], device="cuda")
        assert out[sees].isnan().all()
        assert torch.equal(out[~sees], clean[~sees])
    # rows of the band behind the chunk and before its window, first tokens not in use
    band = torch.cat([torch.full_like(rows[:1], math.nan), rows, torch.full_like(rows[:9], math.inf)])
    out = c.csa2_window_attn_prefill(q[128:], 129, band, 0, SCALE, swa, 0)
    ref = c.csa2_window_attn_prefill(q[128:], 129, torch.cat([rows[:1] * 0, rows]), 0, SCALE, swa, 0)
    assert torch.equal(out, ref) and not out.isnan().any()


# ------------------------------------------------------------------ streams, graphs, the rest
def test_graph_replays_decode_steps():
    """A step captured once and replayed with the next positions in its memory;
    two graphs that share the cache."""
    c = C()
    S, H = 3, 64
    win, model = c.Window(S, 128, 2), Model(S, 128, 2, True)
    start = [0, 5, 126]
    rows0 = make_rows(sum(start), 1)
    c.csa2_window_append(win, rows0, dev64([0] * S), start)
    model.append(rows0, [0] * S, start, range(S))
    pos, row, q = dev64(start), make_rows(S, 2), make_q(S, H, 3)
    out = [torch.empty(S, H, 512, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    graphs = []
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        c.csa2_window_attn_decode(win, q, pos, SCALE, out=out[0])   # loads the kernels
    torch.cuda.synchronize()
    for k in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            c.csa2_window_append(win, row, pos)
            c.csa2_window_attn_decode(win, q, pos, SCALE, out=out[k])
            pos.add_(1)
        graphs.append(g)
    for step in range(5):
        row.copy_(make_rows(S, 20 + step))
        q.copy_(make_q(S, H, 40 + step))
        k = step % 2
        graphs[k].replay()
        at = [s + step for s in start]
        model.append(row, at, [1] * S, range(S))
        for s in range(S):
            kv = torch.stack([model.held[s][x] for x in model.seen(s, at[s])])
            check(out[k][s], None, attend(q[s], kv))
    assert win.device_error() == 0


def test_another_stream():
    c = C()
    win = c.Window(2, 128)
    rows, q = make_rows(60, 1), make_q(2, 64, 2)
    c.csa2_window_append(win, rows, dev64([0, 0]), [30, 30])
    ref = c.csa2_window_attn_decode(win, q, dev64([29, 29]), SCALE)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    pos = dev64([29, 29])
    torch.cuda.synchronize()
    out = c.csa2_window_attn_decode(win, q, pos, SCALE, stream=s)
    back = c.csa2_window_read(win, pos + 0, 5, stream=s)
    s.synchronize()
    assert torch.equal(out, ref) and back.shape == (2, 5, 512)


def test_the_sparse_readout_takes_the_ring():
    """The cache's rows are the window of csa2_sparse_attn_decode as they are."""
    c = C()
    S, n = 2, 200
    cache = c.Cache(c.config(), [256] * S)
    for s in range(S):
        c.csa2_append_entries(cache, [s], [n], torch.randn(n, 512, generator=gen(s), device="cuda"),
                              torch.randn(n, 128, generator=gen(9 + s), device="cuda").bfloat16())
    topk = torch.arange(512, dtype=torch.int32, device="cuda").repeat(S, 1)
    topk[topk >= n] = -1
    q, rows = make_q(S, 64, 5), make_rows(S * n, 6)
    for fp8 in (True, False):
        win = c.Window(S, 128, fp8=fp8)
        rounded = torch.empty_like(rows)
        c.csa2_window_append(win, rows, dev64([0] * S), [n] * S, rounded=rounded)
        want = c.csa2_sparse_attn_decode(cache, q, rounded.view(S, n, 512)[:, -128:].contiguous(), topk,
                                         SCALE)
        if fp8:
            got = c.csa2_sparse_attn_decode(cache, q, None, topk, SCALE, swa_fp8=win.swa_fp8)
        else:
            got = c.csa2_sparse_attn_decode(cache, q, win.swa_kv, topk, SCALE)
        # another order of the same sums: both are within the tolerance above of
        # the same value, and sum p |v| is at most the largest |v|
        big = max(rounded.float().abs().max().item(), 6.0)
        assert (got.float() - want.float()).abs().max() <= 2.0 ** -6 * big + 2.0 ** -7 * want.float().abs().max()
        assert (got.float() - want.float()).abs().mean() <= 2.0 ** -7 * want.float().abs().mean()


def test_refusals():
    c = C()
    win, rows, q, pos = c.Window(2, 16, 1), make_rows(2, 1), make_q(2, 64, 2), dev64([0, 0])
    tree = c.Tree([[-1], [-1]], [0, 0])
    bad = [
        lambda: c.Window(1, 129), lambda: c.Window(1, 0), lambda: c.Window(1, 8, 9),
        lambda: c.csa2_window_append(win, rows.float(), pos),
        lambda: c.csa2_window_append(win, rows[:1], pos),
        lambda: c.csa2_window_append(win, rows, pos.int()),
        lambda: c.csa2_window_append(win, rows, pos, [1]),
        lambda: c.csa2_window_append(win, rows, pos, seq_ids=[0, 0]),
        lambda: c.csa2_window_append(win, rows, pos, seq_ids=[0, 2]),
        lambda: c.csa2_window_append(win, rows, pos, [3, -1]),
        lambda: c.csa2_window_append(win, make_rows(3, 1), dev64([0] * 3)),
        lambda: c.csa2_window_read(win, pos, 17), lambda: c.csa2_window_read(win, pos, 0),
        lambda: c.csa2_window_read(c.Window(2, 16, fp8=False), pos, fp8=True),
        lambda: c.csa2_window_attn_decode(win, q.float(), pos, SCALE),
        lambda: c.csa2_window_attn_decode(win, q[:, :32].contiguous(), pos, SCALE),
        lambda: c.csa2_window_attn_decode(win, q, pos, math.inf),
        lambda: c.csa2_window_attn_decode(win, q, pos, SCALE, out=q),
        lambda: c.csa2_window_attn_decode(win, q, pos, SCALE, rope_out=True, rope_base=0.5),
        lambda: c.csa2_window_attn_decode(win, q.transpose(0, 1), pos, SCALE),
        lambda: c.csa2_window_attn_tree(win, tree, q, rows, SCALE),
        lambda: c.csa2_window_attn_prefill(q, 5, rows, 3, SCALE, 16),
        lambda: c.csa2_window_attn_prefill(q, 1, rows, 2, SCALE, 16),
        lambda: c.csa2_window_attn_prefill(q, 3, rows, 3, SCALE, 16, 1),
        lambda: c.csa2_window_attn_prefill(q, 0, rows, 0, SCALE, 200)]
    for k, call in enumerate(bad):
        with pytest.raises((ValueError, RuntimeError)):
            call()
            pytest.fail(f"call {k} was taken")
    # nothing to do is no error
    none = c.Window(0, 16)
    c.csa2_window_append(none, rows[:0], pos[:0])
    assert c.csa2_window_attn_decode(none, q[:0], pos[:0], SCALE).shape == (0, 64, 512)
    assert c.csa2_window_attn_prefill(q[:0], 0, rows[:0], 0, SCALE).shape == (0, 64, 512)
    assert win.device_error() == 0


@pytest.mark.parametrize("n_trees,drafts", [(50, 4), (150, 1), (40, 9), (300, 3)])
def test_items_over_the_multiprocessors(n_trees, drafts):
    """About as many items as multiprocessors, fewer and more: each draft is answered."""
    c = C()
    parents = [random_tree(drafts, i) for i in range(n_trees)]
    tree = c.Tree(parents, [20 + i for i in range(n_trees)])
    win, model = c.Window(n_trees, 16), Model(n_trees, 16, 0, True)
    before = make_rows(n_trees * 16, 1)
    c.csa2_window_append(win, before, dev64([4 + i for i in range(n_trees)]), [16] * n_trees)
    model.append(before, [4 + i for i in range(n_trees)], [16] * n_trees, range(n_trees))
    q, rows = make_q(tree.n_queries, 64, 2), make_rows(tree.n_queries, 3)
    out = torch.full_like(q, 7.0)
    c.csa2_window_attn_tree(win, tree, q, c.csa2_swa_fp8_quantise(rows), SCALE, out=out)
    for i in range(n_trees):
        for t in range(drafts):
            x = i * drafts + t
            check(out[x], None, attend(q[x], tree_rows(model, tree, i, t, rows, i * drafts)))
