"""Trees of drafted tokens over the cache (csa2_index_scores_tree,
csa2_index_topk_tree, csa2_sparse_attn_tree, csa2_cache_accept_tree).

Two references.  A plain one in 64 bits, written here from the formulas, and
the library's own decode calls over a second cache into which a draft's path
is appended token by token: the tree calls promise the same bits as those.

Tolerances, derived.  Scores: an fp32 sum of 128 products and 32 weighted
heads, each addition within one step (the tensor core may truncate) of the sum
of magnitudes: 2^-23 * 170 * sum_h |w_h| sum_d |q_d k_d|.  Readout: each
probability is rounded to bf16 (2^-8 relative) in the numerator and in the sum
alike, the logits' fp32 error (512 products) is below 2^-10, and the output is
rounded to bf16: (2 * 2^-8 + 2^-9) sum_j p_j |kv_j| + 2^-8 |o|; that bound is
for the worst alignment of the roundings, so over 100 and more candidates,
whose roundings have random signs (a tenth and less of the worst, and half of
that on average), the mean error is held to a sixteenth of its mean as well.
"""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

SCALE = 512 ** -0.5


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def rn(seed, *shape):
    return torch.randn(*shape, generator=gen(seed), device="cuda")


def chain(n):
    return list(range(-1, n - 1))


def random_tree(n, seed):
    r = np.random.RandomState(seed)
    return [int(r.randint(-1, t)) if r.rand() < 0.5 or t == 0 else t - 1 for t in range(n)]


def path_of(parent, t):
    p = []
    while t >= 0:
        p.append(t)
        t = parent[t]
    return p[::-1]


class Setup:
    """A cache with committed and drafted entries, and everything by hand."""

    def __init__(self, trees, pos0, ratio=1, layout=0, idx_layout=0, heads=64, swa=128, topk=512,
                 seq_ids=None, seed=0, extra_seqs=0):
        import fp4_kv_cache_index_gb300 as C
        self.trees, self.pos0, self.m, self.W, self.H, self.k = trees, pos0, ratio, swa, heads, topk
        self.cfg = C.config(n_heads=heads, ratio=ratio, layout=layout, idx_layout=idx_layout,
                            swa=swa, topk=topk)
        self.seq = list(seq_ids) if seq_ids is not None else list(range(len(trees)))
        self.batch = max(self.seq, default=0) + 1 + extra_seqs
        self.tree = C.Tree(trees, pos0, seq_ids)
        self.n_com = [p // ratio for p in pos0]
        self.own = self.tree.owners(ratio)
        self.caps = [37] * self.batch
        for s, n in zip(self.seq, self.n_com):
            self.caps[s] = n + 64 + 3
        self.ent = [rn(seed + 1000 + i, n + len(o), 512) for i, (n, o) in enumerate(zip(self.n_com, self.own))]
        self.key = [rn(seed + 2000 + i, n + len(o), 128).bfloat16()
                    for i, (n, o) in enumerate(zip(self.n_com, self.own))]
        self.cache = C.Cache(self.cfg, self.caps)
        for i, s in enumerate(self.seq):
            C.csa2_append_entries(self.cache, [s], [len(self.ent[i])], self.ent[i], self.key[i])
        nq = self.tree.n_queries
        self.nq = nq
        self.q_idx = rn(seed + 1, nq, 32, 128).bfloat16()
        self.w = rn(seed + 2, nq, 32)
        self.at = [(i, t) for i, p in enumerate(trees) for t in range(len(p))]
        self.vals = None

    def path_entries(self, i, t):
        p = path_of(self.trees[i], t)
        return [e for e, o in enumerate(self.own[i]) if o in p]

    def values(self):
        """Dequantised entries and indexer keys of each tree's sequence."""
        if self.vals is None:
            v = self.cache.views()
            off = v["entry_offset"]
            grid = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6],
                                dtype=torch.float64, device="cuda")
            self.vals = []
            for i, s in enumerate(self.seq):
                a, n = off[s], len(self.ent[i])

                def unpack(codes, sc):
                    c = codes[a:a + n].long()
                    x = torch.stack([grid[c & 15], grid[c >> 4]], -1).flatten(1)
                    return x * sc.repeat_interleave(x.shape[1] // max(1, sc.shape[1]), 1)
                raw = v["scales"][a:a + n]
                sc = (torch.exp2(raw.double() - 127) if v["group"] == 32
                      else raw.view(torch.float8_e4m3fn).double())
                ent = unpack(v["codes"], sc)
                if v["idx_k"] is not None:
                    key = v["idx_k"][a:a + n].double()
                else:
                    key = unpack(v["idx_codes"], torch.exp2(v["idx_scales"][a:a + n].double() - 127))
                self.vals.append((ent, key))
        return self.vals

    def queries64(self):
        if self.cfg.idx_layout == 0:
            return self.q_idx.double()
        x = self.q_idx.double().view(self.nq, 32, 4, 32)
        top = x.abs().amax(-1, keepdim=True)
        s = torch.where(top > 0, torch.exp2(torch.floor(torch.log2(top)) - 2), 1.0)
        a = (x / s).abs()
        edges = torch.tensor([.25, .75, 1.25, 1.75, 2.5, 3.5, 5.], dtype=torch.float64, device="cuda")
        # a tie goes to the even code: past an even code's upper edge only beyond it
        up = torch.stack([(a > e) if j % 2 == 0 else (a >= e) for j, e in enumerate(edges)], -1).sum(-1)
        mag = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6.], dtype=torch.float64, device="cuda")[up]
        return (torch.copysign(mag, x) * s).view(self.nq, 32, 128)

    def rows(self):
        """Per query: cache entries of its score row, in order."""
        return [list(range(self.n_com[i])) + [self.n_com[i] + e for e in self.path_entries(i, t)]
                for i, t in self.at]


def check_scores(st, scores, sentinel):
    q = st.queries64()
    for r, (i, t) in enumerate(st.at):
        cols = st.rows()[r] if st.nq <= 64 else st_rows(st, r)
        key = st.values()[i][1][cols]
        d = q[r] @ key.T
        ref = (st.w[r].double()[:, None] * d.clamp(min=0)).sum(0)
        mag = (st.w[r].double().abs()[:, None] * (q[r].abs() @ key.abs().T)).sum(0)
        got = scores[r].double()
        n = len(cols)
        assert torch.all((got[:n] - ref).abs() <= 170 * 2.0 ** -23 * mag + 1e-30), (r, i, t)
        assert torch.all(scores[r, n:] == sentinel), (r, i, t)


def st_rows(st, r):
    i, t = st.at[r]
    return list(range(st.n_com[i])) + [st.n_com[i] + e for e in st.path_entries(i, t)]


CASES = {
    "one draft": dict(trees=[[-1]], pos0=[300]),
    "first tokens": dict(trees=[[-1, 0, 0, -1, 3]], pos0=[0]),
    "two drafts": dict(trees=[[-1, -1]], pos0=[131]),
    "chain of 3": dict(trees=[chain(3), [-1]], pos0=[511, 128]),
    "ragged": dict(trees=[random_tree(9, 1), [], random_tree(1, 2), random_tree(17, 3)],
                   pos0=[1025, 40, 0, 700]),
    "other sequences": dict(trees=[random_tree(8, 4), random_tree(5, 5)], pos0=[257, 640],
                            seq_ids=[4, 1]),
    "full tree": dict(trees=[random_tree(64, 6)], pos0=[390]),
    "full chain": dict(trees=[chain(64)], pos0=[64]),
    "ratio 2": dict(trees=[random_tree(13, 7), chain(6), [-1]], pos0=[601, 256, 7], ratio=2),
    "ratio 3, none complete": dict(trees=[[-1, -1, -1], chain(7)], pos0=[300, 299], ratio=3),
    "ratio 16": dict(trees=[random_tree(40, 8)], pos0=[1000], ratio=16),
}


def setup(name, **kw):
    return Setup(**{**CASES[name], **kw})


@pytest.mark.parametrize("idx_layout", [0, 1])
@pytest.mark.parametrize("name", list(CASES))
def test_scores(name, idx_layout):
    import fp4_kv_cache_index_gb300 as C
    st = setup(name, idx_layout=idx_layout)
    ld = (max(len(x) for x in st.rows()) + 3) // 4 * 4 + 4
    scores = torch.full((st.nq, ld), -777.0, device="cuda")
    C.csa2_index_scores_tree(st.cache, st.tree, st.q_idx, st.w, scores)
    check_scores(st, scores, -777.0)
    assert st.cache.device_error() == 0


def test_score_histograms():
    import fp4_kv_cache_index_gb300 as C
    st = setup("ragged")
    ld = 1100
    scores = torch.full((st.nq, ld), -777.0, device="cuda")
    hist = torch.full((st.nq, 2048), 5, dtype=torch.int32, device="cuda")
    C.csa2_index_scores_tree(st.cache, st.tree, st.q_idx, st.w, scores, key_hist=hist)
    for r, cols in enumerate(st.rows()):
        u = scores[r, :len(cols)].cpu().numpy().view(np.uint32).astype(np.int64)
        key = np.where(u >> 31, ~u & 0xFFFFFFFF, u | 0x80000000)
        assert np.array_equal(np.bincount(key >> 21, minlength=2048), hist[r].cpu().numpy())


def test_more_queries_than_one_launch_takes():
    import fp4_kv_cache_index_gb300 as C
    for idx_layout in (0, 1):
        trees = [random_tree(64 if i % 3 else 61, 50 + i) for i in range(11)]
        st = Setup(trees, [130 + 7 * i for i in range(11)], idx_layout=idx_layout)
        scores = torch.full((st.nq, 300), -777.0, device="cuda")
        C.csa2_index_scores_tree(st.cache, st.tree, st.q_idx, st.w, scores)
        check_scores(st, scores, -777.0)
        idx = C.csa2_index_topk_tree(st.cache, st.tree, st.q_idx, st.w)
        for r in range(st.nq):
            want = st_rows(st, r)
            assert idx[r].tolist() == want + [-1] * (512 - len(want))
        compare_readout(st, idx, window(st, 7))


def rule(scores, cols, k):
    """The k largest, ties to the lower index, ascending, -1 padded."""
    s = np.where(scores == 0, 0.0, scores)
    order = np.lexsort((np.arange(len(s)), -s))[:k]
    got = [cols[j] for j in sorted(order)]
    return got + [-1] * (k - len(got))


@pytest.mark.parametrize("idx_layout", [0, 1])
@pytest.mark.parametrize("name", list(CASES))
def test_topk_is_the_rule_on_the_scores(name, idx_layout):
    import fp4_kv_cache_index_gb300 as C
    st = setup(name, idx_layout=idx_layout, topk=128 if name != "ragged" else 512)
    ld = (max(len(x) for x in st.rows()) + 3) // 4 * 4
    scores = torch.zeros(st.nq, max(ld, 4), device="cuda")
    C.csa2_index_scores_tree(st.cache, st.tree, st.q_idx, st.w, scores)
    sc = torch.full((st.nq, st.k), 9.0, device="cuda")
    idx = C.csa2_index_topk_tree(st.cache, st.tree, st.q_idx, st.w, topk_score=sc).cpu().numpy()
    for r, cols in enumerate(st.rows()):
        s = scores[r, :len(cols)].cpu().numpy()
        want = rule(s, cols, st.k)
        assert idx[r].tolist() == want, (r, st.at[r])
        place = {c: j for j, c in enumerate(cols)}
        vals = [s[place[c]] if c >= 0 else 0.0 for c in want]
        assert np.array_equal(sc[r].cpu().numpy(), np.array(vals, np.float32))


def test_topk_prefers_the_lower_of_equal_scores():
    """Zero queries: every score is 0, so the first k of the row are kept; the
    path's entries come in only where the committed ones run out."""
    import fp4_kv_cache_index_gb300 as C
    st = Setup([random_tree(20, 3), random_tree(30, 4)], [300, 100], topk=128)
    st.q_idx.zero_()
    idx = C.csa2_index_topk_tree(st.cache, st.tree, st.q_idx, st.w).cpu().numpy()
    for r, cols in enumerate(st.rows()):
        want = cols[:128]
        assert idx[r].tolist() == want + [-1] * (128 - len(want))


def test_long_rows():
    """Rows beyond the segment size of the selection, odd lengths."""
    import fp4_kv_cache_index_gb300 as C
    for idx_layout in (0, 1):
        st = Setup([random_tree(11, 1), chain(2)], [40013, 24577], idx_layout=idx_layout)
        scores = torch.zeros(st.nq, 40080, device="cuda")
        C.csa2_index_scores_tree(st.cache, st.tree, st.q_idx, st.w, scores)
        check_scores(st, scores, 0.0)
        idx = C.csa2_index_topk_tree(st.cache, st.tree, st.q_idx, st.w).cpu().numpy()
        for r, cols in enumerate(st.rows()):
            assert idx[r].tolist() == rule(scores[r, :len(cols)].cpu().numpy(), cols, 512)


# ------------------------------------------------------------------ readout
def window(st, seed, fp8=False, swa_len=None):
    """Committed and drafted window rows of one layer; NaN in every row that
    no draft may read."""
    import fp4_kv_cache_index_gb300 as C
    S = len(st.trees)
    n = swa_len if swa_len is not None else [min(st.W, p) for p in st.pos0]
    win = rn(seed, S, st.W, 512).bfloat16()
    for i in range(S):
        win[i, n[i]:] = float("nan")
    draft = rn(seed + 1, st.nq, 512).bfloat16()
    out = {"win": win, "draft": draft, "len": n, "given": swa_len, "fp8": None}
    if fp8:
        a = [x.view(S, st.W, -1) for x in C.csa2_swa_fp8_quantise(torch.nan_to_num(win))]
        b = C.csa2_swa_fp8_quantise(draft)

        def back(codes, rope, scales):
            s = torch.exp2(scales[..., :7].double() - 127).repeat_interleave(64, -1)
            return torch.cat([codes.view(torch.float8_e4m3fn).double() * s, rope.double()], -1)
        out["win"], out["draft"] = back(*a), back(*b)
        for i in range(S):      # codes 0x7F: NaN
            a[0][i, n[i]:] = 0x7F
            a[1][i, n[i]:] = float("nan")
        out["fp8"] = (tuple(a), tuple(b))
    return out


def readout64(st, idx, q, wd, sink=None, rope=False, base=10000.0):
    """(out, bound, lse) by the formula, 64 bits."""
    first = np.concatenate([[0], np.cumsum([len(p) for p in st.trees])])
    out = torch.zeros(st.nq, st.H, 512, dtype=torch.float64, device="cuda")
    mag = torch.zeros_like(out)
    lse = torch.full((st.nq, st.H), -float("inf"), dtype=torch.float64, device="cuda")
    for r, (i, t) in enumerate(st.at):
        p = path_of(st.trees[i], t)
        keep = [x for x in p][-st.W:] if st.W else []
        n = wd["len"][i] if st.W else 0
        pos = st.pos0[i] + len(p) - 1
        # committed rows at positions pos0 - n .. pos0 - 1, in reach: > pos - W
        com = [j for j in range(n) if st.pos0[i] - n + j > pos - st.W]
        sel = idx[r][idx[r] >= 0].long()
        parts = [st.values()[i][0][sel]]
        if st.W:
            parts += [wd["win"][i][com].double(), wd["draft"][[int(first[i]) + x for x in keep]].double()]
        kv = torch.cat(parts)
        x = q[r].double() @ kv.T * SCALE
        if sink is not None:
            x = torch.cat([x, sink.double()[:, None]], 1)
        if x.shape[1] == 0:
            continue
        lse[r] = torch.logsumexp(x, 1)
        pr = torch.exp(x - lse[r][:, None])[:, :kv.shape[0]]
        out[r], mag[r] = pr @ kv, pr @ kv.abs()
        if rope:
            k = torch.arange(32, device="cuda", dtype=torch.float64)
            ang = -float(pos) * base ** (-k / 32)
            for z in (out[r],):
                a, b = z[:, 448::2].clone(), z[:, 449::2].clone()
                z[:, 448::2] = a * ang.cos() - b * ang.sin()
                z[:, 449::2] = a * ang.sin() + b * ang.cos()
            m = mag[r][:, 448::2] + mag[r][:, 449::2]
            mag[r][:, 448::2] = mag[r][:, 449::2] = m
    return out, mag, lse


def run_readout(st, idx, q, wd, **kw):
    import fp4_kv_cache_index_gb300 as C
    f8 = wd["fp8"] or (None, None)
    return C.csa2_sparse_attn_tree(st.cache, st.tree, q, None if wd["fp8"] else wd["win"],
                                   None if wd["fp8"] else wd["draft"], idx, SCALE,
                                   swa_len=wd["given"], swa_fp8=f8[0], draft_fp8=f8[1], **kw)


def compare_readout(st, idx, wd, sink=None, rope=False, q=None, **kw):
    q = rn(77, st.nq, st.H, 512).bfloat16() if q is None else q
    lse = torch.full((st.nq, st.H), 3.0, device="cuda")
    out = run_readout(st, idx, q, wd, lse=lse, sink=sink, rope_out=rope, **kw)
    ref, mag, ref_lse = readout64(st, idx, q, wd, sink, rope)
    bound = (2 * 2.0 ** -8 + 2.0 ** -9) * mag + 2.0 ** -8 * ref.abs()
    err = (out.double() - ref).abs()
    assert torch.all(err <= bound + 1e-30), float((err / (bound + 1e-30)).max())
    many = (idx >= 0).sum(1) >= 100
    if many.any():
        assert float(err[many].mean()) <= float(bound[many].mean()) / 16
    inf = torch.isinf(ref_lse)
    assert torch.equal(torch.isinf(lse), inf)
    # the sum takes the rounded probabilities: off by at most 2^-8 relative
    assert torch.all((lse.double() - ref_lse)[~inf].abs() <= 2.0 ** -8 + 1e-4)
    return out, lse


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("name", list(CASES))
def test_readout(name, fp8):
    import fp4_kv_cache_index_gb300 as C
    st = setup(name, layout=1 if fp8 else 0)
    idx = C.csa2_index_topk_tree(st.cache, st.tree, st.q_idx, st.w)
    wd = window(st, 300, fp8)
    a = compare_readout(st, idx, wd)
    empty = torch.empty(0, dtype=torch.uint8, device="cuda")
    b = compare_readout(st, idx, wd, workspace=empty)     # one CTA a query
    assert float((a[0].float() - b[0].float()).abs().max()) <= 2.0 ** -5
    assert st.cache.device_error() == 0


@pytest.mark.parametrize("heads, sink, rope, fp8", [(64, True, True, False), (128, False, True, True),
                                                    (128, True, False, False), (64, True, True, True)])
def test_readout_epilogue(heads, sink, rope, fp8):
    import fp4_kv_cache_index_gb300 as C
    st = setup("ragged", heads=heads, layout=1)
    idx = C.csa2_index_topk_tree(st.cache, st.tree, st.q_idx, st.w)
    z = rn(5, heads) * 2 if sink else None
    compare_readout(st, idx, window(st, 310, fp8), sink=z, rope=rope)


@pytest.mark.parametrize("swa", [0, 1, 5, 64, 128])
@pytest.mark.parametrize("fp8", [False, True])
def test_windows_shorter_than_the_path(swa, fp8):
    """The path alone overflows a short window: its deepest rows stay."""
    import fp4_kv_cache_index_gb300 as C
    st = Setup([chain(40), random_tree(64, 3), [-1, 0]], [200, 3, 0], swa=swa)
    idx = C.csa2_index_topk_tree(st.cache, st.tree, st.q_idx, st.w)
    wd = window(st, 320, fp8 and swa > 0)
    compare_readout(st, idx, wd)


def test_given_window_lengths():
    import fp4_kv_cache_index_gb300 as C
    st = Setup([chain(9), random_tree(12, 3), [-1, 0, 0]], [400, 90, 130])
    idx = C.csa2_index_topk_tree(st.cache, st.tree, st.q_idx, st.w)
    for lens in ([0, 0, 0], [128, 90, 1], [7, 33, 127]):
        compare_readout(st, idx, window(st, 330, swa_len=lens))
        compare_readout(st, idx, window(st, 331, fp8=True, swa_len=lens))


def test_every_visible_row_counts_once():
    """Zero queries: all logits are 0, so the output is the mean of the rows
    and lse the log of their number, exactly rounded probabilities (1)."""
    import fp4_kv_cache_index_gb300 as C
    st = Setup([random_tree(30, 9), chain(5)], [500, 60])
    idx = C.csa2_index_topk_tree(st.cache, st.tree, st.q_idx, st.w)
    wd = window(st, 340)
    q = torch.zeros(st.nq, 64, 512, dtype=torch.bfloat16, device="cuda")
    out, lse = compare_readout(st, idx, wd, q=q)
    for r, (i, t) in enumerate(st.at):
        n = int((idx[r] >= 0).sum()) + min(128, wd["len"][i] + len(path_of(st.trees[i], t)))
        assert float((lse[r] - np.log(n)).abs().max()) <= 4e-6
    ref, _, _ = readout64(st, idx, q, wd)
    # sums of 640 exact terms in fp32 and one division: only the output's rounding is left
    assert torch.all((out.double() - ref).abs() <= 2.0 ** -8 * ref.abs() + 2.0 ** -14)


def test_nothing_selected_and_no_window():
    """No candidate at all gives zeros and -inf (or the sink's logit)."""
    import fp4_kv_cache_index_gb300 as C
    st = Setup([[-1, 0]], [0], swa=0, ratio=4)
    idx = C.csa2_index_topk_tree(st.cache, st.tree, st.q_idx, st.w)
    assert torch.all(idx == -1)
    q = rn(1, 2, 64, 512).bfloat16()
    for sink in (None, rn(3, 64)):
        lse = torch.zeros(2, 64, device="cuda")
        out = C.csa2_sparse_attn_tree(st.cache, st.tree, q, None, None, idx, SCALE, lse=lse, sink=sink)
        assert torch.all(out == 0)
        if sink is None:
            assert torch.equal(lse, torch.full_like(lse, -float("inf")))
        else:
            # z goes to log2 units and back: two constants and two products,
            # each rounded to fp32 (2^-24 relative)
            assert torch.all((lse - sink).abs() <= 4 * 2.0 ** -24 * sink.abs() * 1.01)


def test_an_entry_off_the_path_is_skipped_and_reported():
    import fp4_kv_cache_index_gb300 as C
    st = Setup([[-1, 0, 0, 1]], [200])
    idx = C.csa2_index_topk_tree(st.cache, st.tree, st.q_idx, st.w)
    wd = window(st, 350)
    q = rn(1, 4, 64, 512).bfloat16()
    good = run_readout(st, idx, q, wd)
    assert st.cache.device_error() == 0
    bad = idx.clone()
    bad[3, 300] = 202       # draft 2's entry: not an ancestor of draft 3
    bad[0, 301] = 204       # past the sequence
    got = run_readout(st, bad, q, wd)
    assert torch.equal(got, good)
    assert st.cache.device_error() == 7
    assert st.cache.device_error() == 0


def test_layers_in_one_launch_are_the_layers_alone():
    import fp4_kv_cache_index_gb300 as C
    st = Setup([random_tree(50, 9), random_tree(64, 8), chain(30)], [500, 60, 999])
    idx = C.csa2_index_topk_tree(st.cache, st.tree, st.q_idx, st.w)
    ws = [window(st, 400 + 10 * l) for l in range(3)]
    qs = [rn(500 + l, st.nq, 64, 512).bfloat16() for l in range(3)]
    sinks = [rn(600, 64), None, rn(601, 64)]
    outs = C.csa2_sparse_attn_tree_layers(st.cache, st.tree, qs, [w["win"] for w in ws],
                                          [w["draft"] for w in ws], idx, SCALE, sinks=sinks,
                                          rope_out=True)
    for l in range(3):
        one = run_readout(st, idx, qs[l], ws[l], sink=sinks[l], rope_out=True)
        assert torch.equal(one, outs[l])


# ------------------------------------------------------------------ against decode
@pytest.mark.parametrize("ratio, layout, idx_layout, fp8", [(1, 0, 0, False), (2, 1, 1, True),
                                                            (2, 0, 0, True), (1, 1, 1, False)])
def test_same_bits_as_decoding_the_path(ratio, layout, idx_layout, fp8):
    """Each draft's selection and readout are those of the decode calls on a
    cache that holds its path and nothing else, window rows in position order."""
    import fp4_kv_cache_index_gb300 as C
    trees = [random_tree(7, 21), random_tree(10, 22)]
    st = Setup(trees, [1301, 642], ratio=ratio, layout=layout, idx_layout=idx_layout)
    idx = C.csa2_index_topk_tree(st.cache, st.tree, st.q_idx, st.w)
    wd = window(st, 700, fp8)
    q = rn(9, st.nq, 64, 512).bfloat16()
    lse = torch.zeros(st.nq, 64, device="cuda")
    empty = torch.empty(0, dtype=torch.uint8, device="cuda")
    out = run_readout(st, idx, q, wd, lse=lse, workspace=empty)
    first = [0, 7]
    for r, (i, t) in enumerate(st.at):
        cols = st.rows()[r]
        one = C.Cache(st.cfg, [len(cols) + 5])
        C.csa2_append_entries(one, [0], [len(cols)], st.ent[i][cols].contiguous(),
                              st.key[i][cols].contiguous())
        d_idx = C.csa2_index_topk_decode(one, st.q_idx[r:r + 1], st.w[r:r + 1])
        mapped = torch.tensor([cols[j] if j >= 0 else -1 for j in d_idx[0].tolist()])
        assert torch.equal(mapped, idx[r].cpu().long()), (r, i, t)
        p = path_of(trees[i], t)
        keep = 128 - len(p)
        if fp8:
            a, b = wd["fp8"]
            rows = tuple(torch.cat([x[i, 128 - keep:], y[[first[i] + j for j in p]]]).contiguous()
                         for x, y in zip(a, b))
            kw, sw = dict(swa_fp8=rows), None
        else:
            sw = torch.cat([wd["win"][i, 128 - keep:], wd["draft"][[first[i] + j for j in p]]])[None]
            kw = {}
        d_lse = torch.zeros(1, 64, device="cuda")
        d_out = C.csa2_sparse_attn_decode(one, q[r:r + 1], sw, d_idx, SCALE, lse=d_lse,
                                          workspace=empty, **kw)
        assert torch.equal(d_out[0], out[r]) and torch.equal(d_lse[0], lse[r]), (r, i, t)


def test_a_decoding_loop_with_drafts():
    """Norm and rotation, append, selection, readout and acceptance, step after
    step, give the tokens' outputs that plain decoding gives, bit for bit."""
    import fp4_kv_cache_index_gb300 as C
    B, m = 2, 2
    cfg = C.config(ratio=m, layout=1, idx_layout=1)
    spec, plain = C.Cache(cfg, [400] * B), C.Cache(cfg, [400] * B)
    lens = [301, 420]
    ks = [rn(i, lens[i] // m, 512) for i in range(B)]
    ki = [rn(10 + i, lens[i] // m, 128).bfloat16() for i in range(B)]
    for c in (spec, plain):
        for i in range(B):
            C.csa2_append_entries(c, [i], [lens[i] // m], ks[i], ki[i])
    empty = torch.empty(0, dtype=torch.uint8, device="cuda")

    def token(i, pos, salt):
        """Raw projections of a token that depend on what it is."""
        s = 100000 * (i + 1) + 100 * pos + salt
        return {"q": rn(s, 64, 512).bfloat16(), "kv": rn(s + 10 ** 7, 512).bfloat16(),
                "qi": rn(s + 2 * 10 ** 7, 32, 128).bfloat16(), "w": rn(s + 3 * 10 ** 7, 32),
                "ki": rn(s + 4 * 10 ** 7, 128).bfloat16()}

    def normed(toks, pos):
        """Queries (bf16), window rows (bf16), entries' rows (fp32), indexer tensors."""
        st = lambda k: torch.stack([t[k] for t in toks])
        p = torch.tensor(pos, device="cuda")
        kv = st("kv")
        outs = [None, None, None, None]
        xs = [st("q"), kv, st("qi"), st("ki"), kv]
        outs = [torch.empty_like(x) for x in xs[:4]] + [torch.empty(kv.shape, device="cuda")]
        C.csa2_norm_rope(xs, p, outs=outs)
        return outs, st("w")

    def entry(rows):
        return torch.stack(rows).mean(0)      # a stand-in for the compressor

    # window rows and tail rows (for the unfinished block) of the committed text
    hist = []
    for i in range(B):
        toks = [token(i, p, 0) for p in range(lens[i] - 128, lens[i])]
        o, _ = normed(toks, list(range(lens[i] - 128, lens[i])))
        hist.append({"win": [r for r in o[1]], "ent": [r for r in o[4]], "ki": [r for r in o[3]]})
    plain_hist = [{k: list(v) for k, v in h.items()} for h in hist]
    plain_len = list(lens)
    rng = np.random.RandomState(3)
    for step in range(4):
        trees = [random_tree(int(rng.randint(1, 9)), 40 + 10 * step + i) for i in range(B)]
        tree = C.Tree(trees, lens)
        depth = tree.depths
        salt = [[0 if rng.rand() < .5 else int(rng.randint(1, 90)) for _ in t] for t in trees]
        toks = [token(i, lens[i] + depth[i][t], salt[i][t]) for i in range(B) for t in range(len(trees[i]))]
        (q, win, qi, kin, ent), w = normed(toks, tree.positions("cpu").tolist())
        first = [0, len(trees[0])]
        own = tree.owners(m)
        rows, keys = [], []
        for i in range(B):
            for t in own[i]:
                p = path_of(trees[i], t)
                seq_rows = hist[i]["ent"] + [ent[first[i] + a] for a in p]
                rows.append(entry(seq_rows[-m:]))
                keys.append(kin[first[i] + t])
        if rows:
            C.csa2_append_entries(spec, list(range(B)), [len(o) for o in own], torch.stack(rows),
                                  torch.stack(keys))
        swa = torch.stack([torch.stack(h["win"][-128:]) for h in hist])
        idx = C.csa2_index_topk_tree(spec, tree, qi, w)
        out = C.csa2_sparse_attn_tree(spec, tree, q, swa, win, idx, SCALE, rope_out=True,
                                      workspace=empty)
        accepted = [int(rng.randint(-1, len(t))) for t in trees]
        C.csa2_cache_accept_tree(spec, tree, accepted)
        # the accepted tokens, decoded one by one
        for i in range(B):
            p = path_of(trees[i], accepted[i])
            for t in p:
                r = first[i] + t
                pos = plain_len[i]
                h = plain_hist[i]
                h["win"].append(win[r])
                h["ent"].append(ent[r])
                if (pos + 1) % m == 0:
                    C.csa2_append_entries(plain, [i], [1], entry(h["ent"][-m:])[None], kin[r:r + 1])
                d_idx = C.csa2_index_topk_decode(plain, qi[r:r + 1], w[r:r + 1], seq_ids=[i])
                d = C.csa2_sparse_attn_decode(
                    plain, q[r:r + 1], torch.stack(h["win"][-128:])[None].contiguous(), d_idx, SCALE,
                    seq_ids=[i], rope_pos=torch.tensor([pos], device="cuda"), workspace=empty)
                assert torch.equal(d[0], out[r]), (step, i, t)
                plain_len[i] += 1
            hist[i] = {k: list(v) for k, v in plain_hist[i].items()}
            lens[i] = plain_len[i]
            assert spec.length(i) == plain.length(i) == lens[i] // m
    assert spec.device_error() == 0
    a, b = spec.views(), plain.views()
    for i in range(B):
        lo, n = a["entry_offset"][i], spec.length(i)
        for k in ("codes", "scales", "idx_codes", "idx_scales"):
            assert torch.equal(a[k][lo:lo + n], b[k][lo:lo + n])


# ------------------------------------------------------------------ acceptance
@pytest.mark.parametrize("layout, idx_layout", [(0, 0), (1, 1)])
@pytest.mark.parametrize("ratio", [1, 2, 5])
def test_accept_keeps_the_path(layout, idx_layout, ratio):
    import fp4_kv_cache_index_gb300 as C
    trees = [random_tree(64, 1), chain(64), random_tree(9, 2), [], [-1], random_tree(33, 5)]
    pos0 = [200, 64, 0, 30, 9, 101]
    for seed, pick in enumerate(([63, 40, 8, -1, 0, 32], [-1] * 6, [0, 63, 5, -1, -1, 20])):
        st = Setup(trees, pos0, ratio=ratio, layout=layout, idx_layout=idx_layout,
                   seq_ids=[5, 0, 3, 1, 6, 2], extra_seqs=2)
        before = {k: (v.clone() if isinstance(v, torch.Tensor) else v)
                  for k, v in st.cache.views().items()}
        C.csa2_cache_accept_tree(st.cache, st.tree, pick)
        v = st.cache.views()
        touched = torch.zeros(v["codes"].shape[0], dtype=torch.bool, device="cuda")
        for i, s in enumerate(st.seq):
            keep = [e for e, o in enumerate(st.own[i]) if pick[i] >= 0 and o in path_of(trees[i], pick[i])]
            n = st.n_com[i] + len(keep)
            assert st.cache.length(s) == n == int(v["lengths"][s])
            lo = v["entry_offset"][s]
            src = [lo + j for j in range(st.n_com[i])] + [lo + st.n_com[i] + e for e in keep]
            for k in ("codes", "scales", "idx_k", "idx_codes", "idx_scales"):
                if v[k] is not None:
                    assert torch.equal(v[k][lo:lo + n].view(torch.uint8), before[k][src].view(torch.uint8))
            touched[lo + st.n_com[i]:lo + n] = True
        for k in ("codes", "scales"):     # nothing else moved
            assert torch.equal(v[k][~touched], before[k][~touched])


# ------------------------------------------------------------------ calls in earnest
def test_graph_capture_and_another_stream():
    import fp4_kv_cache_index_gb300 as C
    st = Setup([random_tree(20, 9), chain(5)], [2500, 60])
    wd = window(st, 340)
    q = rn(2, st.nq, 64, 512).bfloat16()
    idx = torch.zeros(st.nq, 512, dtype=torch.int32, device="cuda")
    out = torch.zeros_like(q)
    ws = torch.empty(C.csa2_index_workspace_bytes(st.cache, st.nq), dtype=torch.uint8, device="cuda")

    def step():
        C.csa2_index_topk_tree(st.cache, st.tree, st.q_idx, st.w, topk_idx=idx, workspace=ws)
        run_readout(st, idx, q, wd, out=out)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    s.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    st.q_idx.copy_(rn(91, *st.q_idx.shape).bfloat16())
    q.copy_(rn(92, *q.shape).bfloat16())
    g.replay()
    torch.cuda.synchronize()
    got_idx, got = idx.clone(), out.clone()
    step()
    torch.cuda.synchronize()
    assert torch.equal(got_idx, idx) and torch.equal(got, out)
    # on a stream of the caller's, scratch allocated by the call
    st2 = torch.cuda.Stream()
    st2.wait_stream(torch.cuda.current_stream())
    idx2 = C.csa2_index_topk_tree(st.cache, st.tree, st.q_idx, st.w, stream=st2)
    st2.synchronize()
    assert torch.equal(idx2, idx)


def test_calls_from_two_threads():
    """Trees of other widths (two and eight drafts a tile) scored at once from
    two threads, each with its cache, stream and workspace."""
    import threading
    import fp4_kv_cache_index_gb300 as C
    sts = [Setup([chain(2)], [700]), Setup([chain(16)], [900])]
    want = [C.csa2_index_topk_tree(st.cache, st.tree, st.q_idx, st.w) for st in sts]
    torch.cuda.synchronize()
    got, errors = [None, None], []

    def work(i):
        try:
            st = sts[i]
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(200):
                    got[i] = C.csa2_index_topk_tree(st.cache, st.tree, st.q_idx, st.w)
                torch.cuda.current_stream().synchronize()
        except Exception as e:   # noqa: BLE001 - reported below
            errors.append(e)
    ts = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in ts:
        t.start()
    for t in ts:
        t.join()
    assert not errors
    for i in range(2):
        assert torch.equal(got[i], want[i])


def test_outputs_belong_to_the_stream_of_the_call():
    """Memory that the current stream has just given back may still be read by
    its pending work: a call on another stream must not return it."""
    import fp4_kv_cache_index_gb300 as C
    st = Setup([random_tree(20, 9), chain(5)], [2500, 60])
    wd = window(st, 341)
    q = rn(3, st.nq, 64, 512).bfloat16()
    pos = st.tree.positions()
    idx = C.csa2_index_topk_tree(st.cache, st.tree, st.q_idx, st.w)
    here = [lambda s: C.csa2_index_topk_tree(st.cache, st.tree, st.q_idx, st.w, stream=s),
            lambda s: run_readout(st, idx, q, wd, stream=s),
            lambda s: C.csa2_norm_rope([q], pos, stream=s)[0]]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for call in here:
        want = call(None)
        freed = torch.empty_like(want)
        place = freed.data_ptr()
        del freed
        got = call(s)
        s.synchronize()
        assert got.data_ptr() != place
        assert torch.equal(got, want)


def test_repeats_are_the_same_bits():
    import fp4_kv_cache_index_gb300 as C
    st = Setup([random_tree(64, 9), random_tree(64, 10)], [9000, 5000])
    wd = window(st, 340)
    q = rn(2, st.nq, 64, 512).bfloat16()
    idx = C.csa2_index_topk_tree(st.cache, st.tree, st.q_idx, st.w)
    out = run_readout(st, idx, q, wd)
    for _ in range(5):
        assert torch.equal(C.csa2_index_topk_tree(st.cache, st.tree, st.q_idx, st.w), idx)
        assert torch.equal(run_readout(st, idx, q, wd), out)


def test_offsets_past_32_bits():
    """A sequence whose entries start more than 2^31 bytes into the arrays."""
    import fp4_kv_cache_index_gb300 as C
    for idx_layout in (0, 1):
        cfg = C.config(layout=1, idx_layout=idx_layout)
        tree = C.Tree([random_tree(6, 1)], [150], seq_ids=[1])
        st = Setup([random_tree(6, 1)], [150], layout=1, idx_layout=idx_layout)
        big = C.Cache(cfg, [17_000_003, 300])
        C.csa2_append_entries(big, [1], [156], st.ent[0], st.key[0])
        idx = C.csa2_index_topk_tree(big, tree, st.q_idx, st.w)
        assert torch.equal(idx, C.csa2_index_topk_tree(st.cache, st.tree, st.q_idx, st.w))
        wd = window(st, 3)
        q = rn(2, 6, 64, 512).bfloat16()
        out = C.csa2_sparse_attn_tree(big, tree, q, wd["win"], wd["draft"], idx, SCALE)
        assert torch.equal(out, run_readout(st, idx, q, wd))
        C.csa2_cache_accept_tree(big, tree, [5])
        C.csa2_cache_accept_tree(st.cache, st.tree, [5])
        a, b = big.views(), st.cache.views()
        n = st.cache.length(0)
        assert big.length(1) == n
        assert torch.equal(a["codes"][17_000_003:17_000_003 + n], b["codes"][:n])
        del big, a
        torch.cuda.empty_cache()


def test_no_drafts_at_all():
    import fp4_kv_cache_index_gb300 as C
    st = Setup([[], []], [10, 20])
    assert C.csa2_index_topk_tree(st.cache, st.tree, st.q_idx, st.w).shape == (0, 512)
    e = torch.empty(0, 64, 512, dtype=torch.bfloat16, device="cuda")
    wd = window(st, 1)
    assert run_readout(st, torch.empty(0, 512, dtype=torch.int32, device="cuda"), e, wd).shape == e.shape
    C.csa2_cache_accept_tree(st.cache, st.tree, [-1, -1])
    assert [st.cache.length(i) for i in range(2)] == [10, 20]
    none = C.Tree([], [])
    C.csa2_cache_accept_tree(st.cache, none, [])


@pytest.mark.parametrize("idx_layout", [0, 1])
def test_a_wait_that_runs_out_is_reported(idx_layout):
    """The indexer's key loads are withheld: its waits run out, the error word
    says so, and the cache works afterwards."""
    import fp4_kv_cache_index_gb300 as C
    st = Setup([random_tree(9, 2), random_tree(6, 3)], [700, 300], idx_layout=idx_layout)
    good = C.csa2_index_topk_tree(st.cache, st.tree, st.q_idx, st.w)
    scores = torch.full((st.nq, 768), -5.0, device="cuda")
    st.cache.set_wait_limit(200_000)
    st.cache.inject_fault(1)
    C.csa2_index_scores_tree(st.cache, st.tree, st.q_idx, st.w, scores)
    torch.cuda.synchronize()
    assert torch.all(scores == -5.0)
    assert st.cache.device_error() == 6
    st.cache.inject_fault(0)
    st.cache.set_wait_limit(0)
    assert torch.equal(C.csa2_index_topk_tree(st.cache, st.tree, st.q_idx, st.w), good)
    assert st.cache.device_error() == 0


def test_refusals():
    import fp4_kv_cache_index_gb300 as C
    st = Setup([[-1, 0, 0], [-1]], [40, 20])
    c, t, qi, w = st.cache, st.tree, st.q_idx, st.w

    def refused(f, status=None):
        with pytest.raises((C.Csa2Error, ValueError)) as e:
            f()
        if status is not None:
            assert e.value.status == status
    # the cache does not hold what the tree says
    for parents, pos0, seq in (([[-1, 0], [-1]], [40, 20], None), ([[-1, 0, 0], [-1]], [41, 20], None),
                               ([[-1, 0, 0], [-1]], [-1, 20], None), ([[-1, 0, 0], [-1]], [40, 20], [0, 0]),
                               ([[-1, 0, 0], [-1]], [40, 20], [0, 2]), ([[-1, 0, 0], [-1]], [40, 20], [-1, 1]),
                               ([[-1, 0, 0], [-1], []], [40, 20, 0], None)):
        bad = C.Tree(parents, pos0, seq)
        n = bad.n_queries
        refused(lambda: C.csa2_index_topk_tree(c, bad, qi[:n], w[:n]), 1)
        refused(lambda: C.csa2_cache_accept_tree(c, bad, [-1] * bad.n_seqs), 1)
    scores = torch.zeros(4, 44, device="cuda")
    refused(lambda: C.csa2_index_scores_tree(c, t, qi[:3], w, scores))
    refused(lambda: C.csa2_index_scores_tree(c, t, qi, w.double(), scores))
    refused(lambda: C.csa2_index_scores_tree(c, t, qi.cpu(), w, scores))
    refused(lambda: C.csa2_index_scores_tree(c, t, qi, w, scores[:, :40].contiguous()), 3)
    refused(lambda: C.csa2_index_scores_tree(c, t, qi, w, torch.zeros(4, 46, device="cuda")), 1)
    mx = Setup([[-1, 0, 0], [-1]], [40, 20], idx_layout=1)
    hist = torch.zeros(4, 2048, dtype=torch.int32, device="cuda")
    refused(lambda: C.csa2_index_scores_tree(mx.cache, mx.tree, qi, w, scores, key_hist=hist), 2)
    refused(lambda: C.csa2_index_topk_tree(c, t, qi, w, workspace=torch.empty(1 << 20, dtype=torch.uint8)))
    refused(lambda: C.csa2_index_topk_tree(c, t, qi, w, workspace=torch.empty(64, dtype=torch.uint8, device="cuda")), 3)
    idx = C.csa2_index_topk_tree(c, t, qi, w)
    wd = window(st, 5)
    q = rn(1, 4, 64, 512).bfloat16()
    go = lambda **kw: C.csa2_sparse_attn_tree(**{**dict(cache=c, tree=t, q=q, swa_kv=wd["win"], draft_kv=wd["draft"],
                                                        topk_idx=idx, scale=SCALE), **kw})
    go()
    refused(lambda: go(q=q[:3]))
    refused(lambda: go(q=q.float()))
    refused(lambda: go(swa_kv=None))
    refused(lambda: go(draft_kv=None))
    refused(lambda: go(draft_kv=wd["draft"][:3].contiguous()))
    refused(lambda: go(topk_idx=idx[:, :128].contiguous()))
    refused(lambda: go(swa_len=[41, 20]), 1)
    refused(lambda: go(swa_len=[-1, 20]), 1)
    refused(lambda: go(swa_len=[1]))
    refused(lambda: go(rope_out=True, rope_base=float("nan")), 1)
    refused(lambda: go(swa_fp8=C.csa2_swa_fp8_quantise(torch.nan_to_num(wd["win"]))))
    refused(lambda: go(sink=torch.zeros(63, device="cuda")))
    refused(lambda: C.csa2_cache_accept_tree(c, t, [3, 0]), 1)
    refused(lambda: C.csa2_cache_accept_tree(c, t, [-2, 0]), 1)
    refused(lambda: C.csa2_cache_accept_tree(c, t, [0]))
    assert [c.length(i) for i in range(2)] == [43, 21]
    C.csa2_cache_accept_tree(c, t, [2, -1])
    assert [c.length(i) for i in range(2)] == [42, 20]
    refused(lambda: C.csa2_cache_accept_tree(c, t, [2, -1]), 1)      # the step is over


def test_the_readme_step_runs():
    import os
    import re
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    text = open(os.path.join(root, "README.md")).read()
    code = re.findall(r"```python\n(.*?)```", text, re.S)[1]
    assert "csa2_cache_accept_tree" in code
    exec(compile(code, "README.md", "exec"), {})
