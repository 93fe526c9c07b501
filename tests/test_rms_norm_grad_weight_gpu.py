"""The norm's weight gradient counts every row once (GPU), at any number of rows: with h of ones and minus ones and whole g, every
sum on the way is a whole number below 2^24, so the result is exact and a row too few or too many shows."""
import numpy as np
import pytest
import torch

import xnor_popcount_gemm_gb300 as bt

pytestmark = pytest.mark.gpu


# rows to lanes, one, two and four a warp, and tails of each; rows through the ring, aligned and not, for every number of columns a
# thread has; rows that are read twice
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,N", [(1, 8), (2431, 8), (2433, 8), (5003, 32), (9000, 31), (30001, 64), (2561, 72), (5003, 128), (2434, 127), (2561, 256), (40001, 512),
                                 (2600, 777), (9001, 1000), (9001, 1024), (305, 1024), (3001, 1032), (5001, 2048), (3001, 2047), (4999, 4096), (303, 4096), (607, 4093),
                                 (2000, 8192), (601, 8191), (777, 16384), (311, 16383), (999, 17000), (500, 17001), (97, 32768)])
def test_every_row_counts_once(T, N, dtype):
    # the mean of the squares, N / N, and its root are 1 in fp32
    assert np.float32(np.float64(N) * np.float64(np.float32(1.0 / N))) == 1.0
    gen = torch.Generator(device="cuda").manual_seed(T + N)
    h = torch.randint(0, 2, (T, N), generator=gen, device="cuda") * 2 - 1
    g = torch.randint(1, 8, (T, N), generator=gen, device="cuda")
    want = (g * h).sum(dim=0)
    assert 7 * T < 1 << 24
    g, h = g.to(dtype), h.to(dtype)
    for gs in (None, torch.zeros(T, N, dtype=dtype, device="cuda")):
        gx, gw = bt.bt_rms_norm_backward(g, h, None, 0.0, grad_sum=gs)
        assert torch.equal(gw, want.float())
