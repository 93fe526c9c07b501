"""GPU: numbers of the adapters that random inputs do not show (bt_adapter_linear,
bt_adapter_linear_backward): ranks that cancel."""
import pytest
import torch

import xnor_popcount_gemm_gb300 as bt

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(autouse=True)
def _device_clean():
    yield
    assert bt.bt_device_status() == 0


@pytest.fixture(params=["small", "large"])
def path(request, monkeypatch):
    """Either forward, whatever the rule on sizes says."""
    monkeypatch.setenv("BT_ADAPTER_PATH", request.param)
    return request.param


def _bf16_parts(v):
    """fp32 values as three bf16 ones that sum to them exactly."""
    parts = []
    for _ in range(3):
        parts.append(v.bfloat16())
        v = v - parts[-1].float()
    assert not v.any()
    return parts


def _near_pairs(L, seed):
    """Two fp32 values of 24 bits in [1, 2) for every adapter, 2^-16 to 2^-15 apart."""
    gen = torch.Generator().manual_seed(seed)
    one = 1 + torch.rand(L, generator=gen) * 0.99
    return one, one + (1 + torch.rand(L, generator=gen)) * 2.0 ** -16


def test_ranks_that_cancel_show_no_rounding_of_u(path):
    """u_0 and u_1 agree in 15 bits and are subtracted. Each is a sum of three terms, which drops 2^-23 of it at most a
    term, and its three bf16 values leave nothing: 2 x 3 x 2^-23 x 2 in all, and the result's own rounding. (Two bf16
    values of each would be 2^-18 off on average.)"""
    L, T, K, N, R = 64, 128, 64, 48, 16
    one, two = _near_pairs(L, 1)
    x = torch.zeros(T, K)
    x[:, :3] = 1
    a, b = torch.zeros(L, R, K), torch.zeros(L, N, R)
    a[:, 0, :3] = torch.stack([p.float() for p in _bf16_parts(one)], 1)
    a[:, 1, :3] = torch.stack([p.float() for p in _bf16_parts(two)], 1)
    b[:, :, 0], b[:, :, 1] = 1, -1
    ids = torch.arange(T) % L
    plan = bt.bt_adapter_plan(ids, L, device=DEV)
    x, a, b, s = (t.to(DEV) for t in (x.bfloat16(), a.bfloat16(), b.bfloat16(), torch.ones(L)))
    want = (one.double() - two.double())[ids][:, None]
    for out_dtype in (torch.bfloat16, torch.float32):
        got = bt.bt_adapter_linear(x, a, b, s, plan, out_dtype=out_dtype).cpu().double()
        step = 2.0 ** -8 if out_dtype == torch.bfloat16 else 2.0 ** -23
        assert ((got - want).abs() <= 12 * 2.0 ** -23 + step * want.abs()).all(), (got - want).abs().max()


def test_ranks_that_cancel_show_no_rounding_of_du():
    """The same of dU and grad_x."""
    L, T, K, N, R = 64, 128, 40, 64, 16
    one, two = _near_pairs(L, 2)
    g = torch.zeros(T, N)
    g[:, :3] = 1
    a, b = torch.zeros(L, R, K), torch.zeros(L, N, R)
    b[:, :3, 0] = torch.stack([p.float() for p in _bf16_parts(one)], 1)
    b[:, :3, 1] = torch.stack([p.float() for p in _bf16_parts(two)], 1)
    a[:, 0], a[:, 1] = 1, -1
    ids = torch.arange(T) % L
    plan = bt.bt_adapter_plan(ids, L, device=DEV)
    x = torch.zeros(T, K)
    x, g, a, b = (t.bfloat16().to(DEV) for t in (x, g, a, b))
    u = torch.zeros(T, R, device=DEV)
    got = bt.bt_adapter_linear_backward(x, g, u, a, b, torch.ones(L, device=DEV), plan)[0].cpu().double()
    want = (one.double() - two.double())[ids][:, None]
    assert ((got - want).abs() <= 12 * 2.0 ** -23 + 2.0 ** -8 * want.abs()).all(), (got - want).abs().max()
