"""Norm of every head and rotation of its last channels (csa2_norm_rope)
against the formula in 64 bits (angles in extended precision).

Tolerance, derived: a lane adds 16 squares in turn and five more sums join the
lanes, 22 roundings of 2^-24 under a square root (11); rsqrt is within 2 ulp
(2^-22, so 4); the mean, the square of the scale and two products add one
each: below 32 * 2^-24 = 2^-19 relative.  A rotated value
a cos - b sin adds the sine's and cosine's error (2 ulp, and half a step of
the angle in [-pi, pi], 2^-23) on |a| + |b|.  So |error| <= 2^-18 (|a| + |b|),
plus pos * 2^-51 for the frequency's rounding (53 bits, one rounding of pow),
plus half a step of the output's type: 2^-8 (bf16) or 2^-24 (fp32) relative.
"""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

EPS = 1e-6


def reference(x, pos, weight, rope, base=10000.0, norm=True, eps=EPS):
    """(y, magnitude |a| + |b| of each channel's pair), 64 bits."""
    x = x.detach().cpu().double().numpy()
    if norm:
        with np.errstate(all="ignore"):
            x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    if weight is not None:
        x = x * weight.cpu().double().numpy()
    mag = np.abs(x)
    if rope:
        ld = np.longdouble
        t = np.arange(rope // 2).astype(ld)
        ang = pos.cpu().numpy().astype(ld)[:, None] * np.power(ld(base), -2 * t / ld(rope))
        shape = (len(pos),) + (1,) * (x.ndim - 2) + (rope // 2,)
        c = np.cos(ang).astype(np.float64).reshape(shape)
        s = np.sin(ang).astype(np.float64).reshape(shape)
        a, b = x[..., -rope::2].copy(), x[..., -rope + 1::2].copy()
        x = x.copy()
        with np.errstate(invalid="ignore"):
            x[..., -rope::2], x[..., -rope + 1::2] = a * c - b * s, a * s + b * c
        mag[..., -rope::2] = mag[..., -rope + 1::2] = np.abs(a) + np.abs(b)
    return x, mag


def check(y, x, pos, weight, rope, base=10000.0, norm=True, eps=EPS):
    ref, mag = reference(x, pos, weight, rope, base, norm, eps)
    half = 2.0 ** -8 if y.dtype == torch.bfloat16 else 2.0 ** -24
    got = y.detach().cpu().double().numpy()
    far = float(pos.abs().max()) if pos is not None and pos.numel() else 0.0
    tol = half * np.abs(ref) + (2.0 ** -18 + far * 2.0 ** -51) * mag + 1e-38
    fine = np.isfinite(ref)
    assert np.array_equal(np.isnan(ref), np.isnan(got))
    assert np.all(np.abs(got - ref)[fine] <= tol[fine]), np.max((np.abs(got - ref) / tol)[fine])


def rand(shape, dtype=torch.bfloat16, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * 3).to(dtype)


def positions(n, seed=1, hi=1 << 20):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randint(0, hi, (n,), generator=g, device="cuda")


@pytest.mark.parametrize("dim, rope", [(512, 64), (512, 0), (512, 8), (512, 128), (256, 128),
                                       (128, 64), (128, 128), (64, 64), (64, 24)])
@pytest.mark.parametrize("tokens, heads", [(1, 1), (1, 64), (3, 5), (17, 32), (130, 1), (5, 128)])
def test_against_64_bits(dim, rope, tokens, heads):
    import fp4_kv_cache_index_gb300 as C
    pos = positions(tokens)
    w = 1 + 0.2 * rand((dim,), torch.float32, 5)
    for i, (xt, yt) in enumerate([(torch.bfloat16, torch.bfloat16), (torch.bfloat16, torch.float32),
                                  (torch.float32, torch.bfloat16), (torch.float32, torch.float32)]):
        x = rand((tokens, heads, dim), xt, 10 + i)
        out = torch.empty(x.shape, dtype=yt, device="cuda")
        weight = w if i % 2 == 0 else None
        y, = C.csa2_norm_rope([x], pos, weights=[weight], outs=[out], rope_dim=rope)
        assert y.data_ptr() == out.data_ptr()
        check(out, x, pos, weight, rope)


def test_several_tensors_of_a_step_in_one_launch():
    """Queries, KV rows out of the same projection, indexer queries and keys:
    strides, types, norms and positions of their own."""
    import fp4_kv_cache_index_gb300 as C
    n, H = 37, 64
    row = rand((n, H + 1, 512), seed=2)
    q, kv = row[:, :H], row[:, H:]
    qi, ki = rand((n, 32, 128), seed=3), rand((11, 128), torch.float32, 4)
    pos, pos_k = positions(n), positions(11, 7)
    w = [1 + 0.2 * rand((d,), torch.float32, 20 + i) for i, d in enumerate((512, 512, 128, 128))]
    outs = [torch.empty(n, H, 512, dtype=torch.bfloat16, device="cuda"),
            torch.empty(n, 1, 512, device="cuda"), torch.empty_like(qi),
            torch.empty(11, 128, dtype=torch.bfloat16, device="cuda")]
    keep = row.clone()
    C.csa2_norm_rope([q, kv, qi, ki], [pos, pos, pos, pos_k], weights=[w[0], w[1], None, w[3]],
                     outs=outs, norms=[True, True, False, True], rope_dim=[64, 64, 64, 32])
    assert torch.equal(row, keep)
    check(outs[0], q, pos, w[0], 64)
    check(outs[1], kv, pos, w[1], 64)
    check(outs[2], qi, pos, None, 64, norm=False)
    check(outs[3], ki, pos_k, w[3], 32)
    # each alone gives the same bits
    for i, (x, p, r) in enumerate([(q, pos, 64), (kv, pos, 64), (qi, pos, 64), (ki, pos_k, 32)]):
        alone, = C.csa2_norm_rope([x], p, weights=[None if i == 2 else w[i]],
                                  outs=[torch.empty_like(outs[i])], norms=[i != 2], rope_dim=r)
        assert torch.equal(alone, outs[i])


def test_strided_output_leaves_the_rest_alone_and_in_place():
    import fp4_kv_cache_index_gb300 as C
    n = 9
    x = rand((n, 6, 128), seed=8)
    pos = positions(n)
    wide = torch.full((n + 2, 10, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    view = wide[1:n + 1, 2:8]
    C.csa2_norm_rope([x], pos, outs=[view])
    check(view, x, pos, None, 64)
    rest = wide.clone()
    rest[1:n + 1, 2:8] = 7.0
    assert torch.all(rest == 7.0)
    y, = C.csa2_norm_rope([x], pos, outs=[torch.empty_like(x)])
    C.csa2_norm_rope([x], pos, outs=[x])
    assert torch.equal(x, y)
    # tokens in another order through a transposed view: heads before tokens
    xt = rand((6, n, 128), seed=9)
    y, = C.csa2_norm_rope([xt.transpose(0, 1)], pos, outs=[torch.empty(n, 6, 128, dtype=xt.dtype, device="cuda")])
    check(y, xt.transpose(0, 1), pos, None, 64)


def test_no_tokens_and_no_heads():
    import fp4_kv_cache_index_gb300 as C
    e = torch.empty(0, 4, 128, dtype=torch.bfloat16, device="cuda")
    z = torch.empty(3, 0, 128, dtype=torch.bfloat16, device="cuda")
    x = rand((3, 2, 128))
    none = torch.empty(0, dtype=torch.int64, device="cuda")
    pos = positions(3)
    ys = C.csa2_norm_rope([e, z, x], [none, pos, pos])
    assert ys[0].shape == e.shape and ys[1].shape == z.shape
    check(ys[2], x, pos, None, 64)
    assert C.csa2_norm_rope([], pos) == []


def test_zeros_infinities_nan_and_extremes():
    """Zero rows stay zero, a NaN or an infinity stays in its own head, and
    magnitudes whose squares leave fp32 are normed like any other."""
    import fp4_kv_cache_index_gb300 as C
    x = rand((2, 12, 512), torch.float32, 3)
    x[0, 0] = 0
    x[0, 1, 5] = float("nan")
    x[0, 2, 500] = float("inf")
    x[0, 3] *= 1e37
    x[0, 4] *= 1e18         # the sum of squares overflows, no square does
    x[0, 5] *= 1e-30
    x[0, 6] = 0
    x[0, 6, 77] = 3e38
    x[0, 7] = 3.0e38
    x[0, 8] = 1e-44
    pos = torch.tensor([0, 123457], device="cuda")
    for out in (torch.empty_like(x), torch.empty(x.shape, dtype=torch.bfloat16, device="cuda")):
        C.csa2_norm_rope([x], pos, outs=[out])
        live = [h for h in range(12) if h not in (1, 2)]
        check(out[:, live], x[:, live], pos, None, 64)
        assert torch.all(out[0, 0] == 0)
        assert torch.isnan(out[0, 1]).all()      # the mean of the head is NaN
        # x / inf = 0 for finite channels, inf / inf = NaN; the rotation spreads it over its pair
        bad = torch.isnan(out[0, 2])
        assert bad[500] and bad[501] and bad.sum() == 2
        assert torch.all(out[0, 2][~bad] == 0)


@pytest.mark.parametrize("where", [0, 1, (1 << 20) + 1, (1 << 31) + 12345, -1, -((1 << 24) + 3)])
def test_far_positions(where):
    import fp4_kv_cache_index_gb300 as C
    n = 40
    x = rand((n, 2, 512), torch.float32, 6)
    pos = torch.arange(where, where + n, device="cuda")
    for base in (10000.0, 500000.0, 1.0):
        y, = C.csa2_norm_rope([x], pos, rope_base=base, rope_dim=64)
        check(y, x, pos, None, 64, base)


def test_rotation_is_undone_by_the_opposite_position():
    import fp4_kv_cache_index_gb300 as C
    x = rand((21, 4, 512), torch.float32, 6)
    pos = positions(21)
    y, = C.csa2_norm_rope([x], pos, norms=[False])
    z, = C.csa2_norm_rope([y], -pos, norms=[False])
    # two rotations: at most 2 * 2^-18 of the pair's magnitude (below 2 |x|max)
    assert float((z - x).abs().max()) <= 2 ** -16 * float(x.abs().max())


def test_captured_and_replayed_on_another_stream():
    import fp4_kv_cache_index_gb300 as C
    x, pos = rand((50, 8, 512), seed=4), positions(50)
    out = torch.zeros_like(x)
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        C.csa2_norm_rope([x], pos, outs=[out])
    s.synchronize()
    first = out.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        C.csa2_norm_rope([x], pos, outs=[out])
    x.copy_(rand((50, 8, 512), seed=5))
    pos.add_(3)
    g.replay()
    torch.cuda.synchronize()
    check(out, x, pos, None, 64)
    assert not torch.equal(out, first)


def test_refusals():
    import fp4_kv_cache_index_gb300 as C
    x, pos = rand((4, 2, 128)), positions(4)
    with pytest.raises(ValueError):
        C.csa2_norm_rope([x.half()], pos)
    with pytest.raises(ValueError):
        C.csa2_norm_rope([x.cpu()], pos)
    with pytest.raises(ValueError):
        C.csa2_norm_rope([x], pos.int())
    with pytest.raises(ValueError):
        C.csa2_norm_rope([x], pos[:3])
    with pytest.raises(ValueError):
        C.csa2_norm_rope([x], pos, outs=[torch.empty_like(x[:3])])
    with pytest.raises(ValueError):
        C.csa2_norm_rope([x], pos, weights=[torch.ones(64, device="cuda")])
    with pytest.raises(ValueError):
        C.csa2_norm_rope([x[..., ::2]], pos)
    with pytest.raises(ValueError):
        C.csa2_norm_rope([x] * 9, pos)
    with pytest.raises(C.Csa2Error):      # heads 8 bytes off a 16-byte boundary
        C.csa2_norm_rope([rand((4, 132))[:, 4:]], pos)
    with pytest.raises(C.Csa2Error):
        C.csa2_norm_rope([rand((4, 2, 96))], pos)
    with pytest.raises(C.Csa2Error):
        C.csa2_norm_rope([x], pos, eps=0.0)
    with pytest.raises(C.Csa2Error):      # every token of the output on one place
        C.csa2_norm_rope([x], pos, outs=[rand((1, 2, 128)).expand(4, 2, 128)])
    with pytest.raises(C.Csa2Error):
        C.csa2_norm_rope([x], pos, eps=2.0)


def test_the_ends_of_the_ranges():
    """eps 1 beside squares beyond fp32 and beside zeros; the smallest eps; an
    input that broadcasts one token."""
    import fp4_kv_cache_index_gb300 as C
    x = rand((4, 3, 256), torch.float32, 8)
    x[1] *= 1e30
    x[2] = 0
    x[3] *= 1e-12
    pos = positions(4)
    for eps in (1.0, 1e-30):
        y, = C.csa2_norm_rope([x], pos, eps=eps)
        check(y, x, pos, None, 64, eps=eps)
    one = rand((1, 3, 256)).expand(4, 3, 256)
    y, = C.csa2_norm_rope([one], pos, outs=[torch.empty(4, 3, 256, dtype=torch.bfloat16, device="cuda")])
    check(y, one, pos, None, 64)


def test_calls_from_two_threads():
    """Launches of different table sizes issued at once from two threads, each
    on its own stream."""
    import threading
    import fp4_kv_cache_index_gb300 as C
    xs = [rand((96, 1, 64), seed=1), rand((2, 64, 512), seed=2)]
    ps = [positions(96, 3), positions(2, 4)]
    torch.cuda.synchronize()
    outs, errors = [[], []], []

    def work(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(300):
                    outs[i] = C.csa2_norm_rope([xs[i]], ps[i])
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
        check(outs[i][0], xs[i], ps[i], None, 64)
