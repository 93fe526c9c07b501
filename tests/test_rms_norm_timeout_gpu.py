"""The norm's backward with waits that run out (GPU): reported once, what is on its way still lands, the next call is right.

With a limit of 1 ns a warp that meets a row still on its way gives up at once. Every kind of row that goes through the ring:
several CTAs an SM, two, one, a thread's columns read a second time, aligned and not, one row a CTA and many."""
import pytest
import torch

import xnor_popcount_gemm_gb300 as bt

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,N", [(1, 64), (5000, 1000), (3000, 777), (4000, 2048), (700, 4093), (2000, 4096), (900, 8192), (900, 8191), (600, 16384)])
def test_a_wait_that_runs_out_is_reported(T, N):
    gen = torch.Generator().manual_seed(N)
    g, h, gs = (torch.randn(T, N, generator=gen).to(torch.bfloat16).cuda() for _ in range(3))
    w = torch.rand(N, generator=gen).cuda()
    want = bt.bt_rms_norm_backward(g, h, w, grad_sum=gs)
    assert bt.bt_device_status() == 0
    buf = torch.full((T + 4, N), 7.0, dtype=torch.bfloat16, device="cuda")
    bt.bt_set_wait_timeout(1)
    try:
        for _ in range(3):
            bt.bt_rms_norm_backward(g, h, w, grad_sum=gs, grad_x=buf[:T])
        status = bt.bt_device_status()
    finally:
        bt.bt_set_wait_timeout(0)
    # (the clock that waits are measured by ticks once in a while: the copies of one short row may land before it does. Then
    # no wait ran out, and the result is whole)
    assert status == bt.BT_ERR_TIMEOUT or (T == 1 and status == 0 and torch.equal(buf[:T], want[0]))
    assert bt.bt_device_status() == 0
    assert bool((buf[T:] == 7.0).all())
    got = bt.bt_rms_norm_backward(g, h, w, grad_sum=gs)
    assert all(torch.equal(a, b) for a, b in zip(got, want)) and bt.bt_device_status() == 0
