"""What the drafted-token operators are measured on.

Speculative decoding over the FP4 cache: a small model drafts a tree of tokens
for every sequence, and one step of the large model checks the whole tree.
Three operators run next to the cache then, each measured here in its own
cases:

  norm_rope    RMS norm of every head and the position rotation of its last
               channels, for queries, KV rows, indexer queries and indexer
               keys of the step in one call
  tree_scores  index scores of the drafted queries against their sequence's
               committed entries and the entries of their own path
  tree_attn    the sparse readout of the drafted queries: selected FP4
               entries, the committed window rows still in reach and the
               path's own rows, one softmax

Geometry of a tree case.  Sequence i holds `L` committed tokens and
floor(L / ratio) committed entries; draft t of its tree has a parent (a draft
before it, or the last committed token) and sits at position L + depth(t).  A
draft whose position completes a block of `ratio` tokens owns one entry,
appended after the committed ones in draft order.  A draft sees the committed
entries and those of its own path.  Row q of the scores is laid out as
decoding its path token by token would lay it out: the committed entries, then
the path's.

`own` false: plain torch in 32 bits.  `own` true: the package's calls.
"""
import math
import random

import numpy as np
import torch

own = False

DEV = "cuda"
ROPE = 64           # rotated channels, the last of each head
BASE = 10000.0
EPS = 1e-6
MAX_TREE = 64       # drafts of one tree


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one decode step of a few sequences: launch latency
        _norm("norm-decode-3", 3, 64, False),
        # the drafted tokens of a batch
        _norm("norm-drafts-509", 509, 64, False),
        # the 128-head layer, queries and KV row read out of one fused projection
        _norm("norm-fused-1536", 1536, 128, True),
        # a prefill chunk
        _norm("norm-prefill-8192", 8192, 64, False),
        # a short chat with a short chain of drafts
        _scores("scores-chat", 1, 5, 4096, False, 2, "bf16"),
        # a batch at long context, few drafts: every key is read once from HBM
        _scores("scores-batch8-128k", 8, 8, 131072, True, 1, "bf16"),
        # the paper's key format, odd tree sizes
        _scores("scores-mxfp4-ragged", 4, 29, 131072, True, 1, "mxfp4"),
        # full trees at long context: bound by the tensor cores
        _scores("scores-full-trees", 2, 64, 131072, False, 1, "bf16"),
        # one sequence, a chain of drafts
        _attn("attn-chat", 1, 5, 4096, False, 2, "L32", 64, 1, "bf16", False, False),
        # a group's four layers over a batch of small trees
        _attn("attn-batch8-4layers", 8, 9, 32768, True, 1, "L32", 64, 4, "bf16", False, False),
        # the paper's cache formats with the sink and the output rotation
        _attn("attn-fp8-sink", 6, 23, 32768, True, 1, "L16", 128, 1, "fp8", True, True),
        # full trees of a batch
        _attn("attn-full-trees", 16, 64, 16384, False, 2, "L16", 64, 1, "fp8", False, False),
    ]


def _norm(name, tokens, heads, fused):
    return {"name": name, "op": "norm_rope", "tokens": tokens, "heads": heads, "fused": fused}


def _scores(name, seqs, drafts, ctx, ragged, ratio, keys):
    return {"name": name, "op": "tree_scores", "seqs": seqs, "drafts": drafts, "ctx": ctx,
            "ragged": ragged, "ratio": ratio, "keys": keys}


def _attn(name, seqs, drafts, ctx, ragged, ratio, layout, heads, layers, window, sink, rope):
    return {"name": name, "op": "tree_attn", "seqs": seqs, "drafts": drafts, "ctx": ctx,
            "ragged": ragged, "ratio": ratio, "layout": layout, "heads": heads, "layers": layers,
            "window": window, "sink": sink, "rope": rope}


def _spread(rng, lo, hi):
    """An integer of [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    while True:
        op = rng.choice(["norm_rope", "tree_scores", "tree_attn"])
        if op == "norm_rope":
            case = _norm("", _spread(rng, 1, 8192), rng.choice([64, 128]), rng.random() < 0.5)
        elif op == "tree_scores":
            case = _scores("", _spread(rng, 1, 16), _spread(rng, 1, MAX_TREE),
                           _spread(rng, 200, 131072), rng.random() < 0.7, rng.choice([1, 2]),
                           rng.choice(["bf16", "mxfp4"]))
        else:
            case = _attn("", _spread(rng, 1, 16), _spread(rng, 1, MAX_TREE),
                         _spread(rng, 200, 32768), rng.random() < 0.7, rng.choice([1, 2]),
                         rng.choice(["L32", "L16"]), rng.choice([64, 128]), rng.choice([1, 1, 2, 4]),
                         rng.choice(["bf16", "fp8"]), rng.random() < 0.5, rng.random() < 0.5)
        del case["name"]
        w = work(case)
        if w["bytes"] <= 1.2e9 and w["flops"] <= 137e9:
            return case


# ------------------------------------------------------------------ geometry
W = 128             # window rows
TOPK = 512


def _lengths(case):
    """(committed tokens, drafts) of each sequence."""
    out = []
    for i in range(case["seqs"]):
        tok, n = case["ctx"], case["drafts"]
        if case["ragged"]:
            tok -= (i * 997) % (case["ctx"] // 3 + 1) + i % 2
            n -= (5 * i) % (n // 2 + 1)
        out.append((tok, n))
    return out


def _capacity(case):
    return case["ctx"] // case["ratio"] + MAX_TREE + 5


def _row_len(case):
    """Row stride of the scores: a multiple of 4, at least the longest row."""
    return (_capacity(case) + 3) // 4 * 4


def work(case):
    if case["op"] == "norm_rope":
        n, H = case["tokens"], case["heads"]
        heads512, heads128 = H + 1, 32 + 1
        el = n * (heads512 * 512 + heads128 * 128)
        # bf16 in and out, the KV row's output in fp32, positions, weights
        return {"bytes": 4 * el + 2 * n * 512 + 8 * n + 4 * (2 * 512 + 2 * 128), "flops": 4 * el}
    seqs = _lengths(case)
    nq = sum(n for _, n in seqs)
    m = case["ratio"]
    if case["op"] == "tree_scores":
        key = 256 if case["keys"] == "bf16" else 68
        keys = sum(t // m + n // m for t, n in seqs)
        cells = sum(n * (t // m + 1) for t, n in seqs)
        return {"bytes": key * keys + nq * (32 * 128 * 2 + 128) + 4 * cells,
                "flops": 2 * 32 * 129 * cells}
    entry = 272 if case["layout"] == "L32" else 288
    row = 1024 if case["window"] == "bf16" else 584
    H, L = case["heads"], case["layers"]
    picked = sum(min(t // m, _pool_size(t // m)) + n // m for t, n in seqs)
    rows = sum(min(W, t) + n for t, n in seqs)
    per_q = sum(n * (min(t // m + 1, TOPK) + min(t + 1, W)) for t, n in seqs)
    return {"bytes": entry * picked + 4 * nq * TOPK + L * (row * rows + 2 * nq * H * 1024),
            "flops": 4 * 512 * H * L * per_q}


def _pool_size(n):
    """Entries of a sequence that any of its drafts selects: neighbouring
    tokens choose mostly the same ones."""
    return min(n, TOPK + TOPK // 4)


def _tree(rng, n):
    """Parents of n drafts: mostly short branches off a likely chain."""
    parent, depth = [], []
    for t in range(n):
        p = t - 1 if (t > 0 and rng.random() < 0.45) else rng.randrange(-1, t)
        while p >= 0 and depth[p] >= 15:
            p = parent[p]
        parent.append(p)
        depth.append(depth[p] + 1 if p >= 0 else 0)
    return parent, depth


def _geometry(case, seed):
    """Host lists: per query its sequence, position, path (drafts, ascending)
    and path entries (rows after the committed ones)."""
    rng = random.Random(seed * 7919 + 11)
    m = case["ratio"]
    g = {"parents": [], "pos0": [], "n_com": [], "n_ent": [], "seq": [], "pos": [], "path": [],
         "ents": []}
    for i, (tok, n) in enumerate(_lengths(case)):
        parent, depth = _tree(rng, n)
        owner = [t for t in range(n) if (tok + depth[t] + 1) % m == 0]
        slot = {t: e for e, t in enumerate(owner)}
        for t in range(n):
            path, a = [], t
            while a >= 0:
                path.append(a)
                a = parent[a]
            path.reverse()
            g["path"].append(path)
            g["ents"].append([slot[a] for a in path if a in slot])
            g["seq"].append(i)
            g["pos"].append(tok + depth[t])
        g["parents"].append(parent)
        g["pos0"].append(tok)
        g["n_com"].append(tok // m)
        g["n_ent"].append(len(owner))
    return g


def _padded(lists, width):
    a = np.full((len(lists), max(1, width)), -1, np.int64)
    for i, x in enumerate(lists):
        a[i, :len(x)] = x
    return torch.from_numpy(a).to(DEV)


def _gen(seed, part):
    return torch.Generator(device=DEV).manual_seed((seed * 1000003 + part) & 0x7FFFFFFFFFFF)


def _randn(seed, part, *shape):
    return torch.randn(*shape, generator=_gen(seed, part), device=DEV)


# ------------------------------------------------------------------ formats
def _e2m1_index(a):
    """Code (0..7) of magnitudes: nearest of {0, .5, 1, 1.5, 2, 3, 4, 6}, a tie
    to the even code."""
    c = (a > 0.25).to(torch.uint8)
    for edge, strict in ((0.75, 0), (1.25, 1), (1.75, 0), (2.5, 1), (3.5, 0), (5.0, 1)):
        c += (a > edge) if strict else (a >= edge)
    return c


def _e2m1_pack(x, scale, group):
    """Codes of x / scale, two a byte, the even channel in the low nibble."""
    v = x.view(*x.shape[:-1], -1, group) / scale[..., None]
    c = _e2m1_index(v.abs()) | (torch.signbit(v).to(torch.uint8) << 3)
    c = c.reshape(*x.shape[:-1], -1, 2)
    return c[..., 0] | (c[..., 1] << 4)


def _ue8m0_bytes(x, group, emax):
    """Scale byte of each block: the exponent of its largest magnitude minus
    the element type's largest exponent."""
    amax = x.view(*x.shape[:-1], -1, group).abs().amax(-1)
    _, e = torch.frexp(amax)
    return torch.where(amax > 0, (e - 1 - emax + 127).clamp(0, 254), 0).to(torch.uint8)


def _pow2(b):
    return torch.exp2(b.float() - 127.0)


def _unpack(codes):
    """E2M1 values of packed codes, 32 bits."""
    lut = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=codes.device)
    lut = torch.cat([lut, -lut])
    n = torch.stack([codes & 15, codes >> 4], -1).flatten(-2)
    return lut[n.long()]


def _quantise_entries(x, layout):
    if layout == "L32":
        b = _ue8m0_bytes(x, 32, 2)
        return _e2m1_pack(x, _pow2(b), 32), b
    s = (x.view(*x.shape[:-1], -1, 16).abs().amax(-1) / 6).clamp(max=448).to(torch.float8_e4m3fn)
    return _e2m1_pack(x, s.float().clamp(min=2.0 ** -9), 16), s.view(torch.uint8)


def _entry_values(codes, scales, layout):
    v = _unpack(codes)
    s = _pow2(scales) if layout == "L32" else scales.view(torch.float8_e4m3fn).float()
    return (v.view(*s.shape, -1) * s[..., None]).flatten(-2)


def _window_fp8(rows):
    """(codes, rotated channels, scales) of bf16 rows."""
    x = rows[..., :448].float()
    b = _ue8m0_bytes(x, 64, 8)
    v = (x.view(*x.shape[:-1], 7, 64) / _pow2(b)[..., None]).clamp(-448, 448)
    codes = v.to(torch.float8_e4m3fn).view(torch.uint8).flatten(-2)
    pad = torch.zeros_like(b[..., :1])
    return codes.contiguous(), rows[..., 448:].contiguous(), torch.cat([b, pad], -1).contiguous()


def _window_values(w):
    if isinstance(w, torch.Tensor):
        return w.float()
    codes, rope, scales = w
    v = codes.view(torch.float8_e4m3fn).float().view(*codes.shape[:-1], 7, 64)
    v = v * _pow2(scales[..., :7])[..., None]
    return torch.cat([v.flatten(-2), rope.float()], -1)


# ------------------------------------------------------------------ inputs
def prepare(case, seed):
    return {"norm_rope": _prepare_norm, "tree_scores": _prepare_scores,
            "tree_attn": _prepare_attn}[case["op"]](case, seed)


def _prepare_norm(case, seed):
    n, H = case["tokens"], case["heads"]
    # channel scales differ by a few times, as projections' outputs do
    gain = torch.exp(0.5 * _randn(seed, 1, 512))
    if case["fused"]:
        # one projection's output row: the queries, then the KV row
        row = (_randn(seed, 2, n, H + 1, 512) * gain).bfloat16()
        q, kv = row[:, :H], row[:, H:]
    else:
        q = (_randn(seed, 2, n, H, 512) * gain).bfloat16()
        kv = (_randn(seed, 3, n, 1, 512) * gain).bfloat16()
    qi = (_randn(seed, 4, n, 32, 128) * gain[:128]).bfloat16()
    ki = (_randn(seed, 5, n, 1, 128) * gain[:128]).bfloat16()
    weights = [1 + 0.1 * _randn(seed, 6, 512), 1 + 0.1 * _randn(seed, 7, 512),
               1 + 0.1 * _randn(seed, 8, 128), 1 + 0.1 * _randn(seed, 9, 128)]
    first = random.Random(seed).randrange(0, 1 << 20)
    if n >= 1024:       # a chunk: consecutive positions
        pos = torch.arange(first, first + n, device=DEV)
    else:               # tokens of a batch
        pos = torch.randint(0, 1 << 20, (n,), generator=_gen(seed, 10), device=DEV)
    xs = [q, kv, qi, ki]
    # the KV row goes on to the quantiser, which takes 32-bit rows
    outs = [torch.empty(x.shape, dtype=torch.float32 if i == 1 else torch.bfloat16, device=DEV)
            for i, x in enumerate(xs)]
    return {"case": case, "xs": xs, "pos": pos, "weights": weights, "outs": outs}


def _cache(case, g, entries, keys):
    """The package's cache with the committed and drafted entries of every
    sequence appended."""
    import fp4_kv_cache_index_gb300 as C
    cfg = C.config(n_heads=case.get("heads", 64), ratio=case["ratio"], topk=TOPK, swa=W,
                   layout=1 if case.get("layout") == "L16" else 0,
                   idx_layout=1 if case.get("keys") == "mxfp4" else 0)
    S, cap = case["seqs"], _capacity(case)
    cache = C.Cache(cfg, [cap] * S)
    for i in range(S):
        n = g["n_com"][i] + g["n_ent"][i]
        C.csa2_append_entries(cache, [i], [n], entries[i, :n].contiguous(),
                              keys[i, :n].contiguous())
    return cache, C.Tree(g["parents"], g["pos0"])


def _plan(case, g):
    """Index tensors of the plain form."""
    dev = {"device": DEV}
    seq = torch.tensor(g["seq"], **dev)
    n_com = torch.tensor(g["n_com"], **dev)[seq]
    slot = torch.cat([torch.arange(n) for _, n in _lengths(case)]).to(DEV)
    ents = _padded(g["ents"], max(len(e) for e in g["ents"]))
    return {"seq": seq, "n_com": n_com, "slot": slot, "ents": ents,
            "pos": torch.tensor(g["pos"], **dev), "row_len": _row_len(case)}


def _score_inputs(case, seed):
    g = _geometry(case, seed)
    S, cap, nq = case["seqs"], _capacity(case), len(g["seq"])
    keys = _randn(seed, 1, S, cap, 128).bfloat16()
    q = _randn(seed, 2, nq, 32, 128).bfloat16()
    w = _randn(seed, 3, nq, 32)
    if case["keys"] == "mxfp4":     # the cache holds codes: 16-bit keys that the codes stand for
        x = keys.float()
        b = _ue8m0_bytes(x, 32, 2)
        codes = _e2m1_pack(x, _pow2(b), 32)
        keys = _entry_values(codes, b, "L32").bfloat16()
        return g, keys, (codes, b), q, w
    return g, keys, keys, q, w


def _prepare_scores(case, seed):
    g, keys, held, q, w = _score_inputs(case, seed)
    st = {"case": case, "held": held, "q": q, "w": w,
          "scores": torch.zeros(len(g["seq"]), _row_len(case), device=DEV)}
    st.update(_plan(case, g))
    if own:
        blank = torch.zeros(1, _capacity(case), 512, device=DEV).expand(case["seqs"], -1, -1)
        st["cache"], st["tree"] = _cache(case, g, blank, keys)
    return st


def _attn_inputs(case, seed):
    g = _geometry(case, seed)
    S, cap, nq, H = case["seqs"], _capacity(case), len(g["seq"]), case["heads"]
    codes, scales = _quantise_entries(_randn(seed, 1, S, cap, 512), case["layout"])
    layers = []
    for l in range(case["layers"]):
        q = _randn(seed, 10 + 4 * l, nq, H, 512).bfloat16()
        win = _randn(seed, 11 + 4 * l, S, W, 512).bfloat16()
        draft = _randn(seed, 12 + 4 * l, nq, 512).bfloat16()
        if case["window"] == "fp8":
            win, draft = _window_fp8(win), _window_fp8(draft)
        sink = _randn(seed, 13 + 4 * l, H) if case["sink"] else None
        layers.append({"q": q, "win": win, "draft": draft, "sink": sink})
    # selections: most of a shared pool of the sequence, then the path's own
    idx = torch.full((nq, TOPK), -1, dtype=torch.int32, device=DEV)
    at = 0
    for i, (_, n) in enumerate(_lengths(case)):
        nc = g["n_com"][i]
        pool = torch.rand(nc, generator=_gen(seed, 100 + i), device=DEV).topk(_pool_size(nc))[1]
        pick = torch.rand(n, pool.numel(), generator=_gen(seed, 200 + i), device=DEV)
        own_e = [len(e) for e in g["ents"][at:at + n]]
        order = pool[pick.argsort(1)]
        for t in range(n):
            c = min(pool.numel(), TOPK - own_e[t])
            row = order[t, :c].sort()[0]
            tail = torch.tensor([nc + e for e in g["ents"][at + t]], device=DEV, dtype=row.dtype)
            idx[at + t, :c + own_e[t]] = torch.cat([row, tail]).int()
        at += n
    # rows of the window: position order, the newest last
    win_len = [min(W, t) for t, _ in _lengths(case)]
    return g, codes, scales, layers, idx, win_len


def _prepare_attn(case, seed):
    g, codes, scales, layers, idx, win_len = _attn_inputs(case, seed)
    S, cap = case["seqs"], _capacity(case)
    first = np.concatenate([[0], np.cumsum([n for _, n in _lengths(case)])])
    rows = []
    for i, path in zip(g["seq"], g["path"]):
        p = path[-W:]
        keep = max(0, min(win_len[i], W - len(p)))
        rows.append([i * W + r for r in range(win_len[i] - keep, win_len[i])] +
                    [S * W + int(first[i]) + t for t in p])
    st = {"case": case, "codes": codes.view(S * cap, -1), "scales": scales.view(S * cap, -1),
          "layers": layers, "idx": idx, "rows": _padded(rows, W)}
    st.update(_plan(case, g))
    if own:
        st["cache"], st["tree"] = _cache(
            case, g, _entry_values(codes, scales, case["layout"]),
            torch.zeros(1, cap, 128, device=DEV, dtype=torch.bfloat16).expand(S, -1, -1))
        st["outs"] = [torch.empty_like(l["q"]) for l in layers]
    return st


# ------------------------------------------------------------------ the pass
def run(state):
    return {"norm_rope": _run_norm, "tree_scores": _run_scores,
            "tree_attn": _run_attn}[state["case"]["op"]](state)


def _rotate(y, pos, sign):
    """Channel pairs (2t, 2t + 1) of the last ROPE channels by sign * pos *
    BASE^(-2t / ROPE); y [n, heads, dim], pos [n]."""
    t = torch.arange(0, ROPE, 2, device=y.device, dtype=torch.float64)
    ang = torch.remainder(pos.double()[:, None] * BASE ** (-t / ROPE), 2 * math.pi).float() * sign
    c, s = ang.cos()[:, None], ang.sin()[:, None]
    a, b = y[..., -ROPE::2], y[..., -ROPE + 1::2]
    r = torch.stack([a * c - b * s, a * s + b * c], -1).flatten(-2)
    return torch.cat([y[..., :-ROPE], r], -1)


def _run_norm(st):
    if own:
        import fp4_kv_cache_index_gb300 as C
        return C.csa2_norm_rope(st["xs"], st["pos"], weights=st["weights"], outs=st["outs"],
                                rope_dim=ROPE, eps=EPS, rope_base=BASE)

    def one(x, w, out):
        y = x.float()
        y = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + EPS) * w
        return _rotate(y, st["pos"], 1.0).to(out.dtype)
    return [one(x, w, o) for x, w, o in zip(st["xs"], st["weights"], st["outs"])]


def _run_scores(st):
    if own:
        import fp4_kv_cache_index_gb300 as C
        return C.csa2_index_scores_tree(st["cache"], st["tree"], st["q"], st["w"], st["scores"])
    case = st["case"]
    S, T, cap = case["seqs"], case["drafts"], _capacity(case)
    q = st["q"].float()
    if case["keys"] == "mxfp4":     # the queries are rounded to the keys' format
        b = _ue8m0_bytes(q, 32, 2)
        q = _entry_values(_e2m1_pack(q, _pow2(b), 32), b, "L32")
        keys = _entry_values(*st["held"], "L32")
    else:
        keys = st["held"].float()
    # queries padded to T a sequence, one product a sequence
    qp = torch.zeros(S, T, 32, 128, device=q.device)
    qp[st["seq"], st["slot"]] = q
    wp = torch.zeros(S, T, 32, 1, device=q.device)
    wp[st["seq"], st["slot"], :, 0] = st["w"]
    dots = torch.matmul(qp.view(S, T * 32, 128), keys.transpose(1, 2)).relu_()
    full = (dots.view(S, T, 32, cap) * wp).sum(2)[st["seq"], st["slot"]]
    del dots
    nc, e = st["n_com"][:, None], st["ents"]
    out = torch.zeros(full.shape[0], st["row_len"], device=q.device)
    out[:, :cap] = torch.where(torch.arange(cap, device=q.device) < nc, full, 0.0)
    # the path's entries follow the committed ones without gaps
    j = torch.arange(e.shape[1], device=q.device)
    vals = torch.where(e >= 0, full.gather(1, (nc + e).clamp(min=0, max=cap - 1)), 0.0)
    return out.scatter_add(1, nc + j, vals)


def _run_attn(st):
    case = st["case"]
    scale = 512 ** -0.5
    if own:
        import fp4_kv_cache_index_gb300 as C
        ls, fp8 = st["layers"], case["window"] == "fp8"
        wins, drafts = [l["win"] for l in ls], [l["draft"] for l in ls]
        return C.csa2_sparse_attn_tree_layers(
            st["cache"], st["tree"], [l["q"] for l in ls], None if fp8 else wins,
            None if fp8 else drafts, st["idx"], scale, st["outs"],
            sinks=[l["sink"] for l in ls] if case["sink"] else None, rope_out=case["rope"],
            rope_base=BASE, swa_fp8s=wins if fp8 else None, draft_fp8s=drafts if fp8 else None)
    idx, rows = st["idx"].long(), st["rows"]
    flat = (st["seq"] * _capacity(case))[:, None] + idx.clamp(min=0)
    sel = _entry_values(st["codes"][flat], st["scales"][flat], case["layout"])
    live = torch.cat([idx >= 0, rows >= 0], 1)[:, None]

    def one(l):
        win = torch.cat([_window_values(l["win"]).view(-1, 512), _window_values(l["draft"])])
        kv = torch.cat([sel, win[rows.clamp(min=0)]], 1)
        x = torch.matmul(l["q"].float(), kv.transpose(1, 2)) * scale
        x = torch.where(live, x, -math.inf)
        top = x.amax(-1, keepdim=True)
        if l["sink"] is not None:
            top = torch.maximum(top, l["sink"][:, None])
        p = torch.exp(x - top)
        den = p.sum(-1, keepdim=True)
        if l["sink"] is not None:
            den = den + torch.exp(l["sink"][:, None] - top)
        o = torch.matmul(p, kv) / den
        return (_rotate(o, st["pos"], -1.0) if case["rope"] else o).bfloat16()
    return [one(l) for l in st["layers"]]


# ------------------------------------------------------------------ 64 bits
_GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _round_mx(x):
    """x [.., 128] rounded to blocks of 32 E2M1 values with a power-of-two
    scale, in 64 bits: the nearest grid point, a tie to the even index."""
    v = x.double().reshape(*x.shape[:-1], 4, 32)
    top = v.abs().amax(-1, keepdim=True)
    s = torch.where(top > 0, torch.exp2(torch.floor(torch.log2(top.clamp(min=1e-300))) - 2), 1.0)
    a = (v / s).abs()
    grid = torch.tensor(_GRID, dtype=torch.float64, device=x.device)
    dist = (a[..., None] - grid).abs()
    # even indices get their ties by a nudge below any true difference
    odd = (torch.arange(8, device=x.device) % 2).double() * 1e-12
    return (torch.copysign(grid[(dist + odd).argmin(-1)], v) * s).reshape(x.shape)


def exact(case, seed):
    if case["op"] == "norm_rope":
        st = _prepare_norm(case, seed)
        outs = []
        for x, w in zip(st["xs"], st["weights"]):
            parts = []
            for a in range(0, x.shape[0], 1024):
                v = x[a:a + 1024].double()
                v = v / ((v * v).sum(-1, keepdim=True) / v.shape[-1] + EPS).sqrt() * w.double()
                z = torch.view_as_complex(v[..., -ROPE:].reshape(*v.shape[:-1], ROPE // 2, 2).contiguous())
                k = torch.arange(ROPE // 2, device=v.device, dtype=torch.float64)
                ang = st["pos"][a:a + 1024].double()[:, None] / BASE ** (2 * k / ROPE)
                z = z * torch.polar(torch.ones_like(ang), ang)[:, None]
                v[..., -ROPE:] = torch.view_as_real(z).flatten(-2)
                parts.append(v)
            outs.append(torch.cat(parts))
        return outs
    if case["op"] == "tree_scores":
        g, keys, _, q, w = _score_inputs(case, seed)
        mx = case["keys"] == "mxfp4"
        out = torch.zeros(len(g["seq"]), _row_len(case), device=DEV, dtype=torch.float64)
        k64 = None
        for r, i in enumerate(g["seq"]):
            if r == 0 or i != g["seq"][r - 1]:
                k64 = keys[i].double()
            qr = _round_mx(q[r]) if mx else q[r].double()
            nc = g["n_com"][i]
            cols = torch.tensor([nc + e for e in g["ents"][r]], device=DEV, dtype=torch.long)
            k = torch.cat([k64[:nc], k64[cols]])
            out[r, :k.shape[0]] = w[r].double() @ (qr @ k.T).clamp(min=0)
        return out
    g, codes, scales, layers, idx, win_len = _attn_inputs(case, seed)
    first = np.concatenate([[0], np.cumsum([n for _, n in _lengths(case)])])
    grid = torch.tensor(_GRID + tuple(-x for x in _GRID), dtype=torch.float64, device=DEV)
    outs = []
    for l in layers:
        win, draft = l["win"], l["draft"]
        if case["window"] == "fp8":
            win, draft = _fp8_rows64(*win), _fp8_rows64(*draft)
        else:
            win, draft = win.double(), draft.double()
        o = torch.zeros(l["q"].shape, device=DEV, dtype=torch.float64)
        for r, i in enumerate(g["seq"]):
            pick = idx[r][idx[r] >= 0].long()
            c, s = codes[i][pick].long(), scales[i][pick]
            v = torch.empty(len(pick), 512, device=DEV, dtype=torch.float64)
            v[:, 0::2], v[:, 1::2] = grid[c % 16], grid[c // 16]
            s64 = (s.double() - 127).exp2() if case["layout"] == "L32" else s.view(torch.float8_e4m3fn).double()
            v = v * s64.repeat_interleave(512 // s.shape[1], 1)
            path = [int(first[i]) + t for t in g["path"][r]][-W:]
            keep = max(0, min(win_len[i], W - len(path)))
            kv = torch.cat([v, win[i, win_len[i] - keep:win_len[i]], draft[path]])
            x = l["q"][r].double() @ kv.T / math.sqrt(512.0)
            if l["sink"] is not None:
                x = torch.cat([x, l["sink"].double()[:, None]], 1)
            p = torch.softmax(x, -1)
            o[r] = p[:, :kv.shape[0]] @ kv
        if case["rope"]:
            k = torch.arange(ROPE // 2, device=DEV, dtype=torch.float64)
            ang = -torch.tensor(g["pos"], device=DEV).double()[:, None] / BASE ** (2 * k / ROPE)
            z = torch.view_as_complex(o[..., -ROPE:].reshape(*o.shape[:-1], ROPE // 2, 2).contiguous())
            o[..., -ROPE:] = torch.view_as_real(z * torch.polar(torch.ones_like(ang), ang)[:, None]).flatten(-2)
        outs.append(o)
    return outs


def _fp8_rows64(codes, rope, scales):
    s = (scales[..., :7].double() - 127).exp2().repeat_interleave(64, -1)
    return torch.cat([codes.view(torch.float8_e4m3fn).double() * s, rope.double()], -1)
