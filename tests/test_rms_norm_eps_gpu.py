"""RMS norm and its backward with an eps that fp32 holds with few digits or not at all (GPU), against 64 bits."""
import pytest
import torch

import xnor_popcount_gemm_gb300 as bt

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16
# one eight to a warp's lanes, a CTA, odd widths, wider than registers and the backward's ring
SHAPES = [(2500, 64), (5, 256), (5, 101), (3, 4096), (2, 20000), (2, 33001)]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("T,N", SHAPES)
@pytest.mark.parametrize("eps", [1e-50, 1e-44, 1e-42, 3e-40])
def test_small_eps(T, N, dtype, eps):
    gen = torch.Generator().manual_seed(N)
    # rows about sqrt(eps) where their type has normal numbers there, a row of zeros, an ordinary one
    size = max(eps ** 0.5, 1e-25)
    x = (torch.randn(T, N, generator=gen, dtype=torch.float64) * size).to(dtype)
    x[0] = 0
    if T > 3:
        x[2] = torch.randn(N, generator=gen).to(dtype)
    x = x.cuda()
    g = (torch.randn(T, N, generator=gen) * 1e-3 * size).to(dtype).cuda()
    x64, g64 = x.double(), g.double()
    inv = 1.0 / torch.sqrt(x64.square().mean(dim=1, keepdim=True) + eps)
    y, _, _ = bt.bt_rms_norm(x, None, eps)
    want = x64 * inv
    half = torch.finfo(dtype).eps / 2
    # the fp32 value is the nearest or the one beside it, then one rounding
    assert bool(((y.double() - want).abs() <= want.abs() * (half + 2.0 ** -23)).all())
    assert int(y[0].count_nonzero()) == 0
    gx, gw = bt.bt_rms_norm_backward(g, x, None, eps)
    n = x64 * inv
    gn = g64 * n
    want = inv * (g64 - n * gn.mean(dim=1, keepdim=True))
    # a row's sums: a thread's part one after the other (at most 140 values), a tree above it; a few roundings a value
    c = 160 * 2.0 ** -24
    bound = c * inv * (g64.abs() + n.abs() * gn.abs().mean(dim=1, keepdim=True)) + want.abs() * (half + 2.0 ** -23)
    assert bool(((gx.double() - want).abs() <= bound + torch.finfo(dtype).smallest_normal).all())
    # rows one after the other, n itself to a few roundings and its row's sum
    assert bool(((gw.double() - gn.sum(dim=0)).abs() <= (T + 160) * 2.0 ** -24 * gn.abs().sum(dim=0) + 1e-37).all())


def test_codes_of_zeros_and_the_smallest_eps():
    x = torch.zeros(4, 96, device="cuda")
    for eps in (5e-324, 1e-310, 1e-46):
        y, _, q = bt.bt_rms_norm(x, None, eps, code=bt.BT_CODE_E2M1)
        assert int(y.count_nonzero()) == 0 and int(bt.bt_mx_dequantize(q).count_nonzero()) == 0
