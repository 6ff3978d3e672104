"""Bounded waits of the window layers' attention: with the queries of a CTA's
n-th item and the ones behind it withheld every wait runs out, the call ends, the
error word says so, and the next call is right.  (No copy and no MMA is in
flight then.)"""
import pytest
import torch

from tests.test_gpu_window import C, SCALE, dev64, make_q, make_rows, random_tree

pytestmark = pytest.mark.gpu

TIMEOUT = 6       # CSA2_ERR_TIMEOUT
LIMIT = 200_000   # cycles: 0.1 ms


def filled(n_seqs, fp8, seed):
    win = C().Window(n_seqs, swa=128, n_first=4, fp8=fp8)
    rows = make_rows(150 * n_seqs, seed)
    C().csa2_window_append(win, rows, dev64([0] * n_seqs), n_rows=[150] * n_seqs)
    return win


def runs_out(win, call, n):
    """`call` with everything loaded, with queries withheld, and again."""
    want = call().clone()
    assert win.device_error() == 0
    win.set_wait_limit(LIMIT)
    win.inject_fault(n)
    call()
    torch.cuda.synchronize()                  # the kernel ended by itself
    assert win.device_error() == TIMEOUT
    assert win.device_error() == 0            # read and cleared
    win.inject_fault(0)
    win.set_wait_limit(0)
    assert torch.equal(call(), want)
    assert win.device_error() == 0


@pytest.mark.parametrize("fp8", [True, False])
@pytest.mark.parametrize("heads", [64, 128])
@pytest.mark.parametrize("nq,n", [(1, 1), (60, 1), (130, 1), (600, 1), (600, 2), (600, 3)])
def test_decode(fp8, heads, nq, n):
    """Four CTAs an item, two, one, and four items a CTA."""
    win = filled(50, fp8, 3)
    q, pos = make_q(nq, heads, 5), dev64([149 - i % 7 for i in range(nq)])
    ids = [i % 50 for i in range(nq)]
    runs_out(win, lambda: C().csa2_window_attn_decode(win, q, pos, SCALE, seq_ids=ids), n)


@pytest.mark.parametrize("fp8", [True, False])
@pytest.mark.parametrize("heads", [64, 128])
@pytest.mark.parametrize("trees,drafts,n", [(1, 3, 1), (30, 3, 1), (40, 32, 1), (40, 32, 2), (40, 32, 3),
                                            (300, 4, 2), (700, 2, 3)])
def test_trees(fp8, heads, trees, drafts, n):
    """Items of the same tree in a CTA, of several trees, and both."""
    win = filled(trees, fp8, 7)
    tree = C().Tree([random_tree(drafts, i) if heads == 128 or i % 2 else [-1] * drafts
                     for i in range(trees)], [150] * trees)
    q, kv = make_q(tree.n_queries, heads, 9), make_rows(tree.n_queries, 11)
    rows = C().csa2_swa_fp8_quantise(kv) if fp8 else kv
    runs_out(win, lambda: C().csa2_window_attn_tree(win, tree, q, rows, SCALE), n)


@pytest.mark.parametrize("heads,nq,n", [(64, 1, 1), (64, 91, 1), (64, 1301, 1), (64, 1301, 2),
                                        (64, 1301, 3), (64, 1301, 4), (128, 700, 1), (128, 700, 2),
                                        (128, 700, 4)])
def test_chunks(heads, nq, n):
    """Items that keep their rows, and such that take a new block."""
    win = filled(1, True, 13)
    rows, q = make_rows(nq + 150, 15), make_q(nq, heads, 17)

    def call():
        return C().csa2_window_attn_prefill(q, 150, rows, 0, SCALE, n_first=4, error=win.error,
                                            wait_cycles=win.waits[0], withhold=win.waits[1])
    runs_out(win, call, n)


def test_limits_are_checked():
    win = filled(1, True, 19)
    for f in (win.set_wait_limit, win.inject_fault):
        with pytest.raises(ValueError):
            f(-1)
    q, rows = make_q(2, 64, 1), make_rows(2, 2)
    for bad in (dict(wait_cycles=-1), dict(withhold=-1)):
        with pytest.raises(RuntimeError):
            C().csa2_window_attn_prefill(q, 0, rows, 0, SCALE, **bad)
