"""Rows with NaN in a 64-channel block, written to a cache in 8 bits: codes and
scales are those of csa2_swa_fp8_quantise, which leaves NaN out of the block's
largest magnitude."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n", [1, 40, 33000])
def test_blocks_with_nan_are_rounded_as_the_quantiser_rounds_them(n):
    import fp4_kv_cache_index_gb300 as C
    g = torch.Generator(device="cuda").manual_seed(n)
    rows = torch.randn(n, 512, generator=g, device="cuda").bfloat16()
    for r in range(min(n, 40)):
        b = 64 * (r % 7)
        row = rows[r]
        row[b:b + 64] *= 2.0 ** (r - 20)
        k = r % 8
        if k == 0:
            row[b:b + 64:2] = math.nan                 # all even channels
        elif k == 1:
            row[b + 1:b + 64:2] = math.nan             # all odd ones
        elif k == 2:
            row[b:b + 64] = math.nan
        elif k == 3:
            row[b:b + 64:2] = -math.nan
            row[b + 1] = math.inf
        elif k == 4:
            row[b:b + 63] = math.nan
        elif k == 5:
            row[b + 8:b + 16:2] = math.nan             # all even ones of a lane
        elif k == 6:
            row[b:b + 64:2] = math.nan
            row[b + 1:b + 64:2] = 0.0
        else:
            row[b + 3] = math.nan
    codes, rope, scales = C.csa2_swa_fp8_quantise(rows)
    win = C.Window(1, swa=128, fp8=True)
    rounded = torch.empty_like(rows)
    C.csa2_window_append(win, rows, torch.zeros(1, dtype=torch.int64, device="cuda"), n_rows=[n],
                         rounded=rounded)
    back = C.csa2_window_read(win, torch.full((1,), n, dtype=torch.int64, device="cuda"),
                              n_rows=min(n, 128), fp8=True)
    for got, want in zip(back, (codes, rope.view(n, 64), scales)):
        a = got.view(torch.uint8) if got.dtype == torch.uint8 else got.view(torch.int16)
        b = want.view(torch.uint8) if want.dtype == torch.uint8 else want.view(torch.int16)
        assert torch.equal(a, b[-min(n, 128):].view(a.shape))
    # the rounded rows: code times power of two, NaN where the code is one
    x = codes.view(torch.float8_e4m3fn).float().view(n, 7, 64)
    s = torch.ldexp(torch.ones((), device="cuda"), scales[:, :7].int() - 127)
    want = (x * s[:, :, None]).view(n, 448).bfloat16()
    assert torch.equal(rounded[:, :448].isnan(), want.isnan())
    assert torch.equal(rounded[:, :448].nan_to_num(1.5), want.nan_to_num(1.5))
