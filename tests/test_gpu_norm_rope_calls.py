"""Calls of csa2_norm_rope that its documentation allows: single outputs left
to the call, and no positions where nothing is rotated."""
import pytest
import torch

from tests.test_gpu_norm_rope import check, positions, rand

pytestmark = pytest.mark.gpu


def test_single_outputs_left_to_the_call():
    import fp4_kv_cache_index_gb300 as C
    xs = [rand((5, 4, 128), seed=1), rand((5, 64), torch.float32, 2), rand((5, 2, 512), seed=3)]
    pos = positions(5)
    given = torch.empty(5, 64, dtype=torch.bfloat16, device="cuda")
    ys = C.csa2_norm_rope(xs, pos, outs=[None, given, None], rope_dim=64)
    assert ys[1] is given
    for x, y in zip(xs, ys):
        assert y.shape == x.shape
        check(y, x, pos, None, 64)
    assert [y.dtype for y in ys] == [torch.bfloat16, torch.bfloat16, torch.bfloat16]
    alone = C.csa2_norm_rope(xs, pos, rope_dim=64)
    assert torch.equal(alone[0], ys[0]) and torch.equal(alone[2], ys[2])
    # made on the stream of the call
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    other = C.csa2_norm_rope(xs, pos, outs=[None] * 3, stream=s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(other, alone))


def test_no_positions_where_nothing_is_rotated():
    import fp4_kv_cache_index_gb300 as C
    x, z, pos = rand((7, 3, 256), seed=4), rand((7, 128), seed=5), positions(7)
    y, = C.csa2_norm_rope([x], None, rope_dim=0)
    check(y, x, None, None, 0)
    a, b = C.csa2_norm_rope([x, z], [None, pos], rope_dim=[0, 64])
    check(a, x, None, None, 0)
    check(b, z, pos, None, 64)
    for bad in (lambda: C.csa2_norm_rope([x], None), lambda: C.csa2_norm_rope([x, z], [pos, None])):
        with pytest.raises(ValueError):
            bad()
