"""RMS norm over the whole range of fp32 values (GPU): the fp32 value under the result's rounding is the nearest one but for
about one in 2^24, wherever a row's values lie."""
import pytest
import torch

import xnor_popcount_gemm_gb300 as bt

pytestmark = pytest.mark.gpu

# powers of two that rows lie around: every eighth, and those where sums and their inverses come next to the ends of fp32's range
SIZES = sorted({*range(-144, 128, 8), *range(-48, -36), *range(45, 66)})


@pytest.mark.parametrize("N", [64, 100, 4096, 40000])
def test_every_size_of_values(N):
    gen = torch.Generator().manual_seed(N)
    T = max(1, (1 << 18) // N)
    base = torch.randn(T, N, generator=gen, dtype=torch.float64).cuda()
    off = 0
    for e in SIZES:
        x = (base * 2.0 ** e * 0.3).float()
        x64 = x.double()
        y, _, _ = bt.bt_rms_norm(x, None, 0.0)
        want = (x64 / torch.sqrt(x64.square().mean(dim=1, keepdim=True))).float()
        wrong = y != want
        off += int(wrong.sum())
        assert bool(((y - want).abs()[wrong] <= want.abs()[wrong] * torch.finfo(torch.float32).eps).all())
    # one in 2^24 of these values is one or two a width; four times that and one more are allowed
    n = len(SIZES) * T * N
    assert off <= 1 + 4 * n // (1 << 24), (off, n)
