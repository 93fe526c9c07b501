"""RMS norm and its backward written over their own operands (GPU), with as many rows as every kind of kernel takes several a
CTA of: bit for bit what they give elsewhere."""
import pytest
import torch

import xnor_popcount_gemm_gb300 as bt

pytestmark = pytest.mark.gpu
F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16


def _rows(seed, T, N, dtype):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(T, N, generator=gen, device="cuda") * torch.exp(torch.randn(T, 1, generator=gen, device="cuda"))).to(dtype)


# lanes of a warp, a CTA with one, two and four eights a thread, odd widths, wider than registers
@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("T,N", [(20000, 64), (9000, 128), (5000, 512), (400, 2048), (2000, 4096), (2000, 4093), (2500, 65), (300, 16385), (200, 33001)])
def test_norm(T, N, dtype):
    x, r, w = _rows(1, T, N, dtype), _rows(2, T, N, dtype), _rows(3, 1, N, dtype)[0]
    y, h, q = bt.bt_rms_norm(x, w, residual=r, code=bt.BT_CODE_E2M1)
    alone = bt.bt_rms_norm(x, w)[0]
    codes = bt.bt_mx_dequantize(q)
    # the sum over the residual and the result over x, the sum over x, the result over x without a sum
    a, b = x.clone(), r.clone()
    _, _, p = bt.bt_rms_norm(a, w, residual=b, sum=b, out=a, code=bt.BT_CODE_E2M1)
    assert torch.equal(b, h) and torch.equal(a, y) and torch.equal(bt.bt_mx_dequantize(p), codes)
    a, b = x.clone(), r.clone()
    o, _, _ = bt.bt_rms_norm(a, w, residual=b, sum=a)
    assert torch.equal(a, h) and torch.equal(o, y) and torch.equal(b, r)
    a = x.clone()
    bt.bt_rms_norm(a, w, out=a)
    assert torch.equal(a, alone)
    # the result over the residual, the sum not wanted (which the binding always is)
    b = r.clone()
    t = {F32: bt.BT_F32, BF16: bt.BT_BF16, F16: bt.BT_F16}[dtype]
    s = torch.cuda.current_stream().cuda_stream
    assert bt._c_rms(x.data_ptr(), t, N, b.data_ptr(), N, w.data_ptr(), t, T, N, 1e-6, None, 0, b.data_ptr(), N, 0, None, None, s) == 0
    assert torch.equal(b, y)


# lanes of a warp, the ring with several rows a CTA (aligned and not, every number of columns a thread), two passes over wide rows
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("T,N", [(20000, 64), (9000, 200), (5000, 255), (9000, 512), (2600, 1000), (2600, 1001), (1300, 2048), (1300, 4096), (1300, 4093),
                                 (700, 8192), (700, 8191), (400, 16384), (400, 16383), (300, 17000), (300, 20001)])
def test_backward(T, N, dtype):
    g, h, gs, w = _rows(1, T, N, dtype), _rows(2, T, N, dtype), _rows(3, T, N, dtype), _rows(4, 1, N, dtype)[0]
    gx, gw = bt.bt_rms_norm_backward(g, h, w, grad_sum=gs)
    for which in range(3):
        t = [g.clone(), h.clone(), gs.clone()]
        a, b = bt.bt_rms_norm_backward(t[0], t[1], w, grad_sum=t[2], grad_x=t[which])
        assert a is t[which] and torch.equal(a, gx) and torch.equal(b, gw)
        assert all(torch.equal(p, q) for i, (p, q) in enumerate(zip(t, (g, h, gs))) if i != which)
    assert bt.bt_device_status() == 0
