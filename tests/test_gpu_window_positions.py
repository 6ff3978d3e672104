"""The ends of the range of positions: the lowest one sees nothing, whatever
the cache holds."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fp8", [True, False])
@pytest.mark.parametrize("swa", [128, 5])
def test_the_lowest_position_sees_nothing(fp8, swa):
    """Rows at the highest positions are not the ones before the lowest."""
    import fp4_kv_cache_index_gb300 as C
    win = C.Window(2, swa=swa, n_first=2, fp8=fp8)
    rows = torch.ones(2 * swa, 512, dtype=torch.bfloat16, device="cuda")
    at = torch.tensor([2 ** 63 - swa, 0], dtype=torch.int64, device="cuda")
    C.csa2_window_append(win, rows, at, n_rows=[swa, swa])
    q = torch.ones(2, 64, 512, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(2, 64, device="cuda")
    for low in (-2 ** 63, -2 ** 63 + 1, -2 ** 63 + swa, -1):
        pos = torch.full((2,), low, dtype=torch.int64, device="cuda")
        out = C.csa2_window_attn_decode(win, q, pos, 0.01, lse=lse)
        assert (out == 0).all() and (lse == -torch.inf).all(), low
    pos = torch.tensor([2 ** 63 - 1, swa - 1], dtype=torch.int64, device="cuda")
    out = C.csa2_window_attn_decode(win, q, pos, 0.01, lse=lse)
    assert (out == 1).all() and torch.isfinite(lse).all()
    assert win.device_error() == 0
