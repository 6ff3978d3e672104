"""What a captured call takes anew when it is replayed, and what it keeps: append,
read and decode find positions in device memory, a tree's call has the
positions, sequences and parents of its capture."""
import pytest
import torch

from tests.test_gpu_window import C, SCALE, dev64, make_q, make_rows

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fp8", [True, False])
def test_a_replayed_tree_has_the_positions_of_its_capture(fp8):
    c = C()
    win = c.Window(2, swa=64, n_first=2, fp8=fp8)
    c.csa2_window_append(win, make_rows(200, 1), dev64([0, 0]), n_rows=[100, 100])
    tree = c.Tree([[-1, 0, 0], [-1]], [100, 100])
    q, kv = make_q(4, 64, 2), make_rows(4, 3)
    form = c.csa2_swa_fp8_quantise(kv) if fp8 else kv
    accepted = torch.tensor([1, 0], dtype=torch.int32, device="cuda")
    want = c.csa2_window_attn_tree(win, tree, q, form, SCALE).clone()
    out = torch.zeros_like(want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.csa2_window_attn_tree(win, tree, q, form, SCALE, out=out)
        c.csa2_window_accept_tree(win, tree, form, accepted)
    g.replay()
    assert torch.equal(out, want)
    pos = win.pos.view(-1)[:128].view(2, 64)
    assert pos[0, 100 % 64] == 100 and pos[0, 101 % 64] == 101 and pos[1, 100 % 64] == 100
    # later rows do not move the captured call: it sees what is held below 100 (a row
    # that has taken an older one's place is none) and writes at 100 again
    c.csa2_window_append(win, make_rows(2, 5), dev64([102, 101]))
    direct = c.csa2_window_attn_tree(win, tree, q, form, SCALE)
    out.zero_()
    g.replay()
    assert torch.equal(out, direct)
    assert pos[0, 100 % 64] == 100 and pos[0, 101 % 64] == 101 and pos[0, 102 % 64] == 102
    assert win.device_error() == 0
