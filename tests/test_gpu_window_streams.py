"""Verification and window attention in turn on one stream leave SMs to another
stream's kernels: their launches overlap at a kernel's end only."""
import pytest
import torch

from tests.test_gpu_verify import gen, make
from tests.test_gpu_window import C, SCALE, dev64, make_q, make_rows

pytestmark = pytest.mark.gpu


def captured(f):
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        f()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        f()
    return s, g


def test_another_streams_kernels_do_not_wait_for_the_end():
    """Short kernels that alone take less than a tenth of the other stream's time end
    well before it (in a fifth of its time)."""
    c = C()
    parents = [[t - 1 for t in range(1 + i % 8)] for i in range(64)]
    d = make(parents, 131072, torch.bfloat16, 5)
    d["temperature"].fill_(0.8)
    tree = c.Tree(parents, [0] * 64)
    acc, tok = (torch.empty(64, dtype=torch.int32, device="cuda") for _ in range(2))
    win = c.Window(128)
    c.csa2_window_append(win, make_rows(128 * 128, 3), dev64([0] * 128), n_rows=[128] * 128)
    q, pos = make_q(128, 64, 4), dev64([127] * 128)
    out = torch.empty_like(q)
    x = torch.randn(1 << 22, generator=gen(1), device="cuda")
    y = torch.empty_like(x)

    def steps():
        for _ in range(20):
            c.csa2_verify_tree(tree, d["tokens"], d["logits"], d["temperature"], d["uniform"],
                               d["noise"], d["root_logits"], d["draft_logits"], d["draft_root"], acc, tok)
            c.csa2_window_attn_decode(win, q, pos, SCALE, out=out)

    def short():
        for _ in range(40):
            torch.add(x, 1.0, out=y)
    (s1, g1), (s2, g2) = captured(steps), captured(short)
    for _ in range(3):
        start, end1, end2 = (torch.cuda.Event(enable_timing=True) for _ in range(3))
        with torch.cuda.stream(s1):
            start.record(s1)
            g1.replay()
            end1.record(s1)
        with torch.cuda.stream(s2):
            g2.replay()
            end2.record(s2)
        torch.cuda.synchronize()
        assert start.elapsed_time(end2) < 0.6 * start.elapsed_time(end1)
