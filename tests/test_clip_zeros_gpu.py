"""Clipping gradients that are all zero (GPU): they stay as they are, also where max_norm and eps leave 0 / 0."""
import pytest
import torch

import xnor_popcount_gemm_gb300 as bt

pytestmark = pytest.mark.gpu
F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("sizes", [[1], [7, 0, 5000], [33] * 70])      # (70: more than the small table of tensors holds)
@pytest.mark.parametrize("max_norm,eps", [(0.0, 0.0), (0.0, 1e-6), (1.0, 0.0), (1.0, 1e-6)])
def test_zeros_stay(sizes, dtype, max_norm, eps):
    ts = [torch.zeros(n, device="cuda", dtype=dtype) for n in sizes]
    ts[-1][::2] = -0.0
    kept = [t.clone() for t in ts]
    norm = bt.bt_clip_grads(ts, max_norm, eps)
    assert float(norm) == 0.0
    for t, k in zip(ts, kept):
        assert torch.equal(t, k) and torch.equal(torch.signbit(t), torch.signbit(k))


def test_the_smallest_value_is_not_zero():
    t = [torch.zeros(5000, device="cuda"), torch.zeros(3, device="cuda")]
    t[1][1] = 2.0 ** -149
    assert float(bt.bt_clip_grads(t, 0.0, 0.0)) == 2.0 ** -149
    assert int(t[1].count_nonzero()) == 0 and bool(torch.isfinite(t[1]).all())
