"""What the window layers' operators and the verification of drafts are measured on.

A model over the FP4 cache has layers that see the sliding window alone, and
every layer keeps the rows of its own window.  A step of drafted tokens ends
with the decision which of them are kept.  Three operators, each measured
here in its own cases:

  rows    the window's rows rounded to 8 bits as they are written into the
          cache, a row or a chunk of rows for every sequence, and the windows
          read back in position order
  attn    attention of window layers over that cache: the newest rows and a
          few first tokens that stay visible; one token a sequence, a tree of
          drafted tokens, or a chunk of a prompt
  verify  the walk through every sequence's tree of drafted tokens: each draft
          is tested against the target's probabilities with a given uniform
          number, what is left after a rejection is renormalised, and the
          token that follows the accepted path is drawn by given exponential
          numbers

`own` false: plain torch in 32 bits (64 in the verification, whose results
are whole numbers decided at borders).  `own` true: the package's calls.
"""
import math
import random

import torch

own = False

DEV = "cuda"
D = 512
BASE = 10000.0
SCALE = D ** -0.5
ROW8 = 584          # bytes of a row in 8 bits: codes, rotated channels, scales


# ------------------------------------------------------------------ cases
def listed():
    return [
        # a decode step: one row a sequence, and the windows as the readout of
        # drafts takes them; launch latency
        _rows("rows-decode-16", 16, 1, False),
        # a chunk of a long prompt, rounded as the chunk's attention reads it
        _rows("rows-chunk-8192", 1, 8192, False),
        # the prompts of a batch, of many lengths
        _rows("rows-prompts-192", 192, 1021, True),
        # one chat
        _attn("attn-chat", "decode", 1, 1, 900, 64, 128, 4, True, False),
        # a decode step of a batch, few of its windows still filling up
        _attn("attn-batch-128", "decode", 128, 1, 40000, 64, 128, 0, True, True),
        # a large batch of the 128-head layer over 16-bit rows, a narrow window
        _attn("attn-batch-509-bf16", "decode", 509, 1, 5000, 128, 96, 8, False, False),
        # full trees of drafted tokens with sink logits and the output rotation
        _attn("attn-trees", "tree", 16, 64, 30000, 64, 128, 4, True, True),
        # a short prompt from its first token
        _attn("attn-prompt-509", "prefill", 1, 509, 0, 64, 128, 4, False, False),
        # a chunk of a long prompt
        _attn("attn-chunk-8192", "prefill", 1, 8192, 131072, 64, 128, 4, False, True),
        # one chat, a chain of drafts
        _verify("verify-chat", 1, 5, 32000, "bf16", "logits"),
        # a batch with chains of drafts
        _verify("verify-batch-64", 64, 8, 131072, "bf16", "logits"),
        # full trees, 32-bit logits over an odd vocabulary, drafts without
        # probabilities of their own
        _verify("verify-trees", 12, 64, 100003, "f32", "none"),
    ]


def _rows(name, seqs, n, ragged):
    return {"name": name, "op": "rows", "seqs": seqs, "n": n, "ragged": ragged}


def _attn(name, mode, seqs, n, ctx, heads, window, first, fp8, epilogue):
    return {"name": name, "op": "attn", "mode": mode, "seqs": seqs, "n": n, "ctx": ctx,
            "heads": heads, "window": window, "first": first, "fp8": fp8, "epilogue": epilogue}


def _verify(name, seqs, drafts, vocab, dtype, draft):
    return {"name": name, "op": "verify", "seqs": seqs, "drafts": drafts, "vocab": vocab,
            "dtype": dtype, "draft": draft}


def _spread(rng, lo, hi):
    """An integer of [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    while True:
        op = rng.choice(["rows", "attn", "attn", "verify"])
        if op == "rows":
            case = _rows("", _spread(rng, 1, 512), _spread(rng, 1, 8192), rng.random() < 0.5)
        elif op == "attn":
            mode = rng.choice(["decode", "tree", "prefill"])
            seqs = {"decode": _spread(rng, 1, 600), "tree": _spread(rng, 1, 16), "prefill": 1}[mode]
            n = {"decode": 1, "tree": _spread(rng, 1, 64), "prefill": _spread(rng, 1, 8192)}[mode]
            ctx = rng.choice([0, _spread(rng, 1, 1 << 20)]) if mode == "prefill" else _spread(rng, 1, 1 << 20)
            case = _attn("", mode, seqs, n, ctx, rng.choice([64, 128]),
                         rng.choice([128, 128, rng.randrange(1, 129)]), rng.randrange(0, 9),
                         mode != "prefill" and rng.random() < 0.6, rng.random() < 0.5)
        else:
            case = _verify("", _spread(rng, 1, 64), _spread(rng, 1, 64), _spread(rng, 300, 131072),
                           rng.choice(["bf16", "f32"]), rng.choice(["logits", "none"]))
        del case["name"]
        w = work(case)
        rows = case["seqs"] * (case.get("drafts", 0) + 1)
        if w["bytes"] <= 1.1e9 and w["flops"] <= 140e9 and rows * case.get("vocab", 0) <= 8e7:
            return case


# ------------------------------------------------------------------ geometry
def _counts(case):
    """Rows that each sequence writes: all alike, or of many lengths."""
    S, n = case["seqs"], case["n"]
    return [max(1, n - (i * 389) % n) if case["ragged"] else n for i in range(S)]


def _context(case):
    """Tokens of each sequence before the call."""
    if case["mode"] == "prefill":
        return [case["ctx"]]
    return [max(1, case["ctx"] - (i * 997) % (case["ctx"] // 2 + 1)) if i % 16 != 3 else 1 + i % 100
            for i in range(case["seqs"])]


def _tree(rng, n, deep):
    """Parents of n drafts: mostly short branches off a likely chain."""
    parent, depth = [], []
    for t in range(n):
        p = t - 1 if (t > 0 and rng.random() < deep) else rng.randrange(-1, t)
        while p >= 0 and depth[p] >= 15:
            p = parent[p]
        parent.append(p)
        depth.append(depth[p] + 1 if p >= 0 else 0)
    return parent, depth


def _path(parent, t):
    """The drafts on draft t's path, from the root."""
    out = []
    while t >= 0:
        out.append(t)
        t = parent[t]
    return out[::-1]


# Nodes of a tree that a walk comes to: few, whatever the tree's size.  Counted
# over the listed cases' inputs.
VISITED = {"logits": 3.0, "none": 2.0}


def work(case):
    if case["op"] == "rows":
        n, S = sum(_counts(case)), case["seqs"]
        held = sum(min(128, c) for c in _counts(case))
        # rows in, rounded rows out, the rows held, and the windows as read back
        return {"bytes": n * 2048 + held * (2 * ROW8 + 1024), "flops": 2 * n * 448}
    if case["op"] == "attn":
        W, F, H, n = case["window"], case["first"], case["heads"], case["n"]
        row = ROW8 if case["fp8"] else 1024
        ctx = _context(case)
        if case["mode"] == "prefill":
            keys = sum(min(case["ctx"] + i + 1, W + F) for i in range(n))
            rows, q = min(W, case["ctx"]) + F + n, n
        else:
            keys = sum(n * min(c + 1, W + F) for c in ctx)
            rows, q = sum(min(c, W + F) + n for c in ctx), n * len(ctx)
        return {"bytes": rows * row + q * H * 2048, "flops": 4 * D * H * keys}
    el = 2 if case["dtype"] == "bf16" else 4
    nodes = 1 + (VISITED[case["draft"]] - 1) * (1 - 0.5 ** min(case["drafts"], 16))
    rows = nodes * (2 if case["draft"] == "logits" else 1)
    return {"bytes": case["seqs"] * case["vocab"] * (rows * el + 4),
            "flops": case["seqs"] * case["vocab"] * rows * 4}


# ------------------------------------------------------------------ formats
def _gen(seed, part):
    return torch.Generator(device=DEV).manual_seed((seed * 1000003 + part) & 0x7FFFFFFFFFFF)


def _randn(seed, part, *shape):
    return torch.randn(*shape, generator=_gen(seed, part), device=DEV)


def _make_rows(seed, part, *shape):
    """Rows of a window as a norm and a rotation leave them: a few channels are
    much larger than the rest."""
    gain = torch.exp(0.7 * _randn(seed, part + 1, D))
    return (_randn(seed, part, *shape, D) * gain).bfloat16()


def _pow2(b):
    """2^(b - 127) exactly (exp2 may be a unit off in the last place)."""
    return torch.where(b == 0, 0x00400000, b.int() << 23).view(torch.float32)


def _encode8(rows):
    """(codes, rotated channels, scales): channels 0..447 in E4M3 with a power
    of two for each 64, the exponent of the largest minus 8; 448..511 as they
    are."""
    x = rows[..., :448].float().unflatten(-1, (7, 64))
    top = x.abs().amax(-1)
    _, e = torch.frexp(top)
    b = torch.where(top > 0, (e - 1 - 8 + 127).clamp(0, 254), 0).to(torch.uint8)
    v = (x / _pow2(b)[..., None]).clamp(-448, 448)
    return v.to(torch.float8_e4m3fn).flatten(-2), rows[..., 448:], b


def _decode8(codes, rope, b):
    v = codes.float().unflatten(-1, (7, 64)) * _pow2(b)[..., None]
    return torch.cat([v.flatten(-2), rope.float()], -1)


# ------------------------------------------------------------------ inputs
def prepare(case, seed):
    return {"rows": _prepare_rows, "attn": _prepare_attn, "verify": _prepare_verify}[case["op"]](case, seed)


def _prepare_rows(case, seed):
    counts = _counts(case)
    n, S = sum(counts), case["seqs"]
    # a decode step writes the row behind a full window's other 127, a chunk
    # is longer than a window or starts its sequence
    past = 127 if max(counts) == 1 else 0
    start = [random.Random(seed).randrange(0, 1 << 20) * 128 for _ in range(S)] if past else [0] * S
    st = {"case": case, "rows": _make_rows(seed, 1, n), "old": _make_rows(seed, 3, S, past),
          "pos": torch.tensor([a + past for a in start], device=DEV),
          "end": torch.tensor([a + past + c for a, c in zip(start, counts)], device=DEV)}
    # place of each window row among the rows (old ones first), -1 where the
    # sequence has none there
    at, place = 0, torch.full((S, 128), -1, dtype=torch.int64)
    for i, c in enumerate(counts):
        both = torch.cat([torch.arange(i * past, (i + 1) * past), S * past + at + torch.arange(c)])
        place[i, :min(128, past + c)] = both[-128:]
        at += c
    st["place"] = place.to(DEV)
    if own:
        import fp4_kv_cache_index_gb300 as C
        st["counts"] = None if max(counts) == 1 else counts
        st["win"] = C.Window(S, 128)
        if past:
            C.csa2_window_append(st["win"], st["old"].view(-1, D), st["pos"] - past, [past] * S)
        st["rounded"] = torch.empty_like(st["rows"])
        st["out"] = torch.empty(S, 128, D, dtype=torch.bfloat16, device=DEV)
    return st


def _attn_inputs(case, seed):
    """Rows of the cache [S, window + first], the position that each holds (-1:
    none), queries, their sequences and positions, rows of drafts or of a
    chunk with their positions, and what of them each query may see."""
    rng = random.Random(seed * 7919 + 5)
    W, F, H, n, S = case["window"], case["first"], case["heads"], case["n"], case["seqs"]
    ctx = torch.tensor(_context(case), device=DEV)
    j = torch.arange(W, device=DEV)
    newest = ctx[:, None] - 1 - j                       # the ring, the newest first
    pos = torch.cat([newest, torch.arange(F, device=DEV).expand(S, F)], 1)
    pos = torch.where((pos >= 0) & (pos < ctx[:, None]), pos, -1)
    # a first token that is still inside the window is one row, not two
    pos[:, :W] = torch.where(pos[:, :W] < F, -1, pos[:, :W])
    held = _make_rows(seed, 1, S, W + F)
    q = _randn(seed, 3, (S if case["mode"] == "decode" else S * n), H, D).bfloat16()
    fresh = _make_rows(seed, 5, S * n)                  # rows of drafts, of a chunk, of the new tokens
    sink = _randn(seed, 7, H) if case["epilogue"] else None
    g = {"ctx": ctx, "pos": pos, "held": held, "q": q, "fresh": fresh, "sink": sink}
    if case["mode"] == "tree":
        g["parents"], where, depth = [], [], []
        for i in range(S):
            parent, d = _tree(rng, n, 0.45)
            g["parents"].append(parent)
            depth += d
            where += [[i * n + t for t in _path(parent, u)] for u in range(n)]
        deep = max(len(w) for w in where)
        g["path"] = torch.tensor([w + [-1] * (deep - len(w)) for w in where], device=DEV)
        g["seq"] = torch.arange(S, device=DEV).repeat_interleave(n)
        g["at"] = ctx[g["seq"]] + torch.tensor(depth, device=DEV)
    else:
        g["seq"] = torch.arange(S, device=DEV).repeat_interleave(n)
        g["at"] = ctx[g["seq"]] + torch.arange(n, device=DEV).repeat(S)
    return g


def _prepare_attn(case, seed):
    g = _attn_inputs(case, seed)
    W, F, S, n = case["window"], case["first"], case["seqs"], case["n"]
    st = {"case": case, "q": g["q"], "sink": g["sink"], "at": g["at"], "seq": g["seq"]}
    rows = torch.cat([g["held"].view(-1, D), g["fresh"]])
    st["held"] = _encode8(rows) if case["fp8"] else rows
    # which rows a query reads: the cache's of its sequence, then its own path
    # or the chunk's; and the positions they hold
    here = torch.arange(S * (W + F), device=DEV).view(S, -1)[g["seq"]]
    if case["mode"] == "tree":
        steps = torch.arange(g["path"].shape[1], device=DEV)
        mine, mpos = g["path"], torch.where(g["path"] >= 0, g["ctx"][g["seq"]][:, None] + steps, -1)
    elif case["mode"] == "prefill":
        back = torch.arange(n, device=DEV)[:, None] - torch.arange(W, device=DEV)
        mine, mpos = back, torch.where(back >= 0, case["ctx"] + back, -1)
        # first tokens among the chunk's own
        first = torch.arange(F, device=DEV).expand(n, F)
        mine = torch.cat([mine, first - case["ctx"]], 1)
        mpos = torch.where(mpos < F, -1, mpos)
        mpos = torch.cat([mpos, torch.where(first >= case["ctx"], first, -1)], 1)
    else:
        mine, mpos = torch.arange(S, device=DEV)[:, None], g["at"][:, None]
    rel, keypos = torch.cat([here, S * (W + F) + mine.clamp(min=0)], 1), torch.cat([g["pos"][g["seq"]], mpos], 1)
    at = g["at"][:, None]
    st["rows"] = rel.clamp(max=rows.shape[0] - 1)
    st["live"] = (keypos >= 0) & (keypos <= at) & ((keypos > at - W) | (keypos < F))
    st["out"] = torch.empty_like(g["q"])
    if own:
        import fp4_kv_cache_index_gb300 as C
        st["win"] = win = C.Window(S, W, n_first=F, fp8=case["fp8"])
        ctx = g["ctx"].tolist()
        # the rows that the cache holds, written as their tokens came
        parts, counts, start = [], [], []
        for lo_hi in ("first", "window"):
            for i, c in enumerate(ctx):
                if lo_hi == "first":
                    k = min(F, c)
                    part = g["held"][i, W:W + k]
                else:
                    k = max(0, min(W, c - F))
                    part = g["held"][i, :k].flip(0)
                parts.append(part)
                counts.append(k)
                start.append(0 if lo_hi == "first" else c - k)
        for h in range(2):
            C.csa2_window_append(win, torch.cat(parts[h * S:(h + 1) * S]),
                                 torch.tensor(start[h * S:(h + 1) * S], device=DEV),
                                 counts[h * S:(h + 1) * S])
        if case["mode"] == "tree":
            st["tree"] = C.Tree(g["parents"], ctx)
            st["fresh"] = C.csa2_swa_fp8_quantise(g["fresh"]) if case["fp8"] else g["fresh"]
        elif case["mode"] == "decode":
            C.csa2_window_append(win, g["fresh"], g["at"])
        else:
            # the rows before the chunk and the chunk's, one band
            back = min(W - 1, case["ctx"])
            band = torch.empty(back + n, D, dtype=torch.bfloat16, device=DEV)
            if back:
                C.csa2_window_read(win, g["ctx"], back, out=band[:back].view(1, back, D))
            band[back:] = g["fresh"]
            st["band"], st["band0"] = band, case["ctx"] - back
            # first tokens that lie before the band
            st["first"] = g["held"][0, W:].contiguous() if F and st["band0"] else None
    return st


def _verify_inputs(case, seed):
    rng = random.Random(seed * 7919 + 13)
    S, n, V = case["seqs"], case["drafts"], case["vocab"]
    dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
    target = 5 * _randn(seed, 1, S * (n + 1), V)
    draft = (target + 0.7 * _randn(seed, 2, S * (n + 1), V)).to(dt)
    target = target.to(dt)
    parents = [_tree(rng, n, 0.9 if n < 16 else 0.45)[0] for _ in range(S)]
    temp = torch.tensor([0.0 if i % 8 == 5 else 0.6 + 0.1 * (i % 5) for i in range(S)], device=DEV)
    # rows S.. belong to the drafts, row i to sequence i's last committed token
    row = torch.tensor([S + i * n + p if p >= 0 else i for i, ps in enumerate(parents) for p in ps],
                       device=DEV)
    seq = torch.arange(S, device=DEV).repeat_interleave(n)
    # each draft is drawn from its parent's draft probabilities; drafts that
    # come without probabilities are likely tokens
    sharp = 1.0 if case["draft"] == "logits" else 0.3
    tok = torch.empty(S * n, dtype=torch.int32, device=DEV)
    for lo in range(0, S * n, 64):
        r = slice(lo, min(S * n, lo + 64))
        e = torch.empty(r.stop - lo, V, device=DEV).exponential_(generator=_gen(seed, 100 + lo))
        z = draft[row[r]].float() / (sharp * temp[seq[r]].clamp(min=0.05))[:, None] - e.log()
        tok[r] = z.argmax(1).int()
    u = torch.rand(S * n, generator=_gen(seed, 3), device=DEV)
    noise = torch.empty(S, V, device=DEV).exponential_(generator=_gen(seed, 4)).clamp(min=1e-30)
    return {"target": target, "draft": draft if case["draft"] == "logits" else None, "tok": tok,
            "u": u, "noise": noise, "temp": temp, "parents": parents, "row": row, "seq": seq}


def _prepare_verify(case, seed):
    g = _verify_inputs(case, seed)
    S, n = case["seqs"], case["drafts"]
    st = dict(g, case=case)
    # what is tested after a draft is accepted (its first child) or rejected
    # (its next sibling): rows of the drafts, -1 for none
    down, right, first = [-1] * (S * n), [-1] * (S * n), [-1] * S
    for i, ps in enumerate(g["parents"]):
        last = {}
        for t, p in enumerate(ps):
            if p in last:
                right[i * n + last[p]] = i * n + t
            elif p >= 0:
                down[i * n + p] = i * n + t
            else:
                first[i] = i * n + t
            last[p] = t
    st.update(down=torch.tensor(down, device=DEV), right=torch.tensor(right, device=DEV),
              start=torch.tensor(first, device=DEV))
    # the longest walk: every draft is tested once at most
    st["steps"] = max(_longest(ps) for ps in g["parents"])
    if own:
        import fp4_kv_cache_index_gb300 as C
        st["tree"] = C.Tree(g["parents"], [1000] * S)
    return st


def _longest(parents):
    """Tests of the longest walk through a tree: at each node of a path all of
    its children."""
    kids = {}
    for t, p in enumerate(parents):
        kids.setdefault(p, []).append(t)
    best = [0] * (len(parents) + 1)
    for t in range(len(parents) - 1, -2, -1):
        best[t + 1] = max((k + 1 + best[c + 1] for k, c in enumerate(kids.get(t, []))), default=0)
    return best[0]


# ------------------------------------------------------------------ the pass
def run(state):
    return {"rows": _run_rows, "attn": _run_attn, "verify": _run_verify}[state["case"]["op"]](state)


def _run_rows(st):
    if own:
        import fp4_kv_cache_index_gb300 as C
        C.csa2_window_append(st["win"], st["rows"], st["pos"], st["counts"], rounded=st["rounded"])
        return st["rounded"], C.csa2_window_read(st["win"], st["end"], 128, out=st["out"])
    rounded = _decode8(*_encode8(st["rows"])).bfloat16()
    every = torch.cat([_decode8(*_encode8(st["old"].view(-1, D))).bfloat16(), rounded])
    place = st["place"]
    return rounded, torch.where(place[..., None] >= 0, every[place.clamp(min=0)], 0.0)


def _rotate(y, pos):
    """Channel pairs (2t, 2t + 1) of the last 64 channels by -pos *
    BASE^(-2t / 64); y [n, heads, dim], pos [n]."""
    t = torch.arange(0, 64, 2, device=y.device, dtype=torch.float64)
    ang = torch.remainder(pos.double()[:, None] * BASE ** (-t / 64), 2 * math.pi).float()
    c, s = ang.cos()[:, None], -ang.sin()[:, None]
    a, b = y[..., -64::2], y[..., -63::2]
    r = torch.stack([a * c - b * s, a * s + b * c], -1).flatten(-2)
    return torch.cat([y[..., :-64], r], -1)


def _run_attn(st):
    case, sink = st["case"], st["sink"]
    rope = case["epilogue"]
    if own:
        import fp4_kv_cache_index_gb300 as C
        more = {"out": st["out"], "sink": sink, "rope_out": rope, "rope_base": BASE}
        if case["mode"] == "decode":
            return C.csa2_window_attn_decode(st["win"], st["q"], st["at"], SCALE, **more)
        if case["mode"] == "tree":
            return C.csa2_window_attn_tree(st["win"], st["tree"], st["q"], st["fresh"], SCALE, **more)
        return C.csa2_window_attn_prefill(st["q"], case["ctx"], st["band"], st["band0"], SCALE,
                                          swa=case["window"], n_first=case["first"],
                                          first=st["first"], **more)
    kv = st["held"] if not case["fp8"] else _decode8(*st["held"])
    kv = kv[st["rows"]].float()
    x = torch.matmul(st["q"].float(), kv.transpose(1, 2)) * SCALE
    x = torch.where(st["live"][:, None], x, -math.inf)
    top = x.amax(-1, keepdim=True)
    if sink is not None:
        top = torch.maximum(top, sink[:, None])
    p = torch.exp(x - top)
    den = p.sum(-1, keepdim=True)
    if sink is not None:
        den = den + torch.exp(sink[:, None] - top)
    o = torch.matmul(p, kv) / den
    return (_rotate(o, st["at"]) if rope else o).bfloat16()


def _run_verify(st):
    case = st["case"]
    S, n = case["seqs"], case["drafts"]
    if own:
        import fp4_kv_cache_index_gb300 as C
        t, d = st["target"], st["draft"]
        return C.csa2_verify_tree(st["tree"], st["tok"], t[S:], st["temp"], st["u"], st["noise"],
                                  root_logits=t[:S], draft_logits=None if d is None else d[S:],
                                  draft_root=None if d is None else d[:S])
    seqs = torch.arange(S, device=DEV)
    temp = st["temp"][:, None].double()
    greedy = st["temp"] == 0

    def probs(x, node):
        """Probabilities of row `node` of each sequence; at temperature 0 all
        on the first of the largest logits."""
        z = x[node].double()
        big = z == z.amax(1, keepdim=True)
        hot = big & (big.cumsum(1) == 1)
        return torch.where(greedy[:, None], hot.double(),
                           torch.softmax(z / torch.where(temp > 0, temp, 1.0), 1))

    node, test, last = seqs, st["start"], torch.full((S,), -1, device=DEV)
    left = probs(st["target"], node)
    for _ in range(st["steps"]):
        c = test.clamp(min=0)
        tok = st["tok"][c].long()
        if st["draft"] is None:
            q = torch.zeros_like(left).scatter_(1, tok[:, None], 1.0)
        else:
            q = probs(st["draft"], node)
        # at temperature 0 the target's first choice alone is accepted
        q = torch.where(greedy[:, None], torch.zeros_like(left).scatter_(1, tok[:, None], 1.0), q)
        u = torch.where(greedy, 0.5, st["u"][c].double())
        pick = tok[:, None]
        take = (test >= 0) & (u * q.gather(1, pick)[:, 0] < left.gather(1, pick)[:, 0])
        drop = (test >= 0) & ~take
        rest = (left - q).clamp(min=0)
        total = rest.sum(1, keepdim=True)
        left = torch.where(drop[:, None] & (total > 0), rest / torch.where(total > 0, total, 1.0), left)
        last = torch.where(take, c, last)
        node = torch.where(take, S + c, node)
        left = torch.where(take[:, None], probs(st["target"], node), left)
        test = torch.where(take, st["down"][c], torch.where(drop, st["right"][c], test))
    score = left / torch.where(greedy[:, None], 1.0, st["noise"].double())
    best = score == score.amax(1, keepdim=True)
    token = torch.where(best, torch.arange(case["vocab"], device=DEV), case["vocab"]).amin(1)
    return torch.where(last >= 0, last - seqs * n, -1).int(), token.int()


# ------------------------------------------------------------------ 64 bits
def _power_below(x):
    """The largest power of two that is not above x."""
    return (x.view(torch.int64) >> 52 << 52).view(torch.float64)


def _round8(rows):
    """Rows as 8 bits hold them, in 64 bits: the nearest of the format's
    numbers, a tie to the even one."""
    x = rows.double()
    v = x[..., :448].unflatten(-1, (7, 64))
    top = v.abs().amax(-1, keepdim=True)
    s = torch.where(top > 0, _power_below(top) / 256, 1.0)
    a = (v / s).clamp(-448, 448)
    step = _power_below(a.abs().clamp(min=2.0 ** -6)) / 8
    return torch.cat([(torch.round(a / step) * step * s).flatten(-2), x[..., 448:]], -1)


def exact(case, seed):
    if case["op"] == "rows":
        st = _prepare_rows(case, seed)
        out = torch.zeros(case["seqs"], 128, D, dtype=torch.float64, device=DEV)
        at = 0
        for i, c in enumerate(_counts(case)):
            mine = torch.cat([_round8(st["old"][i]), _round8(st["rows"][at:at + c])])[-128:]
            out[i, :mine.shape[0]] = mine
            at += c
        return _round8(st["rows"]), out
    if case["op"] == "verify":
        return None     # whole numbers
    g = _attn_inputs(case, seed)
    W, F, S, n = case["window"], case["first"], case["seqs"], case["n"]
    held = _round8(g["held"]) if case["fp8"] else g["held"].double()
    fresh = _round8(g["fresh"]) if case["fp8"] else g["fresh"].double()
    out = torch.empty(g["q"].shape, dtype=torch.float64, device=DEV)
    if case["mode"] == "prefill":
        # all rows of the sequence that any query may see, blocks of queries
        keep = g["pos"][0] >= 0
        kv, kpos = torch.cat([held[0][keep], fresh]), torch.cat([g["pos"][0][keep], g["at"]])
        blocks = [(slice(a, min(n, a + 512)), kv, kpos) for a in range(0, n, 512)]
    else:
        blocks = []
        for r in range(g["q"].shape[0]):
            i = int(g["seq"][r]) if case["mode"] == "tree" else r
            keep = g["pos"][i] >= 0
            own_rows = [i * n + t for t in _path(g["parents"][i], r - i * n)] if case["mode"] == "tree" else [r]
            kpos = torch.arange(len(own_rows), device=DEV) + g["ctx"][i]
            blocks.append((slice(r, r + 1), torch.cat([held[i][keep], fresh[own_rows]]),
                           torch.cat([g["pos"][i][keep], kpos])))
    for r, kv, kpos in blocks:
        at = g["at"][r][:, None]
        near = (kpos <= at) & ((at - kpos < W) | (kpos < F))
        used = near.any(0)
        kv, near = kv[used], near[:, used]
        x = torch.einsum("qhd,kd->qhk", g["q"][r].double(), kv) / math.sqrt(512.0)
        x = x.masked_fill(~near[:, None], -math.inf)
        if g["sink"] is not None:
            x = torch.cat([x, g["sink"].double()[None, :, None].expand(x.shape[0], -1, 1)], -1)
        out[r] = torch.softmax(x, -1)[..., :kv.shape[0]] @ kv
    if case["epilogue"]:
        k = torch.arange(32, device=DEV, dtype=torch.float64)
        ang = -g["at"].double()[:, None] / BASE ** (2 * k / 64)
        z = torch.view_as_complex(out[..., -64:].unflatten(-1, (32, 2)).contiguous())
        out[..., -64:] = torch.view_as_real(z * torch.polar(torch.ones_like(ang), ang)[:, None]).flatten(-2)
    return out
