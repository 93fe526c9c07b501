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


def _signs(L, C, R, dtype):
    """[L, C, R]: ranks of one sign for every c, which alternates."""
    gen = torch.Generator().manual_seed(3)
    return ((torch.rand(L, C, R, generator=gen) + 0.5) * (1 - 2 * (torch.arange(C) % 2))[:, None]).to(dtype)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("R", [1, 3, 8, 16, 24, 40, 100])
@pytest.mark.parametrize("T", [4, 70])
def test_an_infinity_goes_as_far_as_the_formula_says(T, R, dtype, path):
    """An infinity in x makes u of its token infinite, and its results +inf or -inf with the sign of B's row; a rank that
    is no 16, 32, 64 or 128 adds nothing of its padding."""
    K, N = 72, 41
    gen = torch.Generator().manual_seed(4)
    x, a, b = torch.randn(T, K, generator=gen).to(dtype), torch.rand(1, R, K, generator=gen).to(dtype) + 0.5, _signs(1, N, R, dtype)
    x[2, 9] = float("inf")
    plan = bt.bt_adapter_plan([0] * T, 1, device=DEV)
    u = torch.empty(T, R, device=DEV)
    for out_dtype in (dtype, torch.float32):
        out = bt.bt_adapter_linear(*(t.to(DEV) for t in (x, a, b)), torch.ones(1, device=DEV), plan, out_dtype=out_dtype, u=u).cpu()
        want = (x.double() @ a[0].double().t()) @ b[0].double().t()
        assert torch.equal(out[2].double(), want[2]) and want[2].isinf().all()
        assert torch.cat([out[:2], out[3:]]).isfinite().all() and (u[2] == float("inf")).all()


@pytest.mark.parametrize("R", [1, 3, 8, 16, 24, 40, 100])
def test_an_infinity_in_the_backward(R):
    """The same of g, dU, grad_x and grad_a."""
    T, K, N = 70, 72, 41
    gen = torch.Generator().manual_seed(5)
    x, g = torch.randn(T, K, generator=gen).bfloat16(), torch.randn(T, N, generator=gen).bfloat16()
    a, b = _signs(1, K, R, torch.bfloat16).transpose(1, 2).contiguous(), torch.rand(1, N, R, generator=gen).bfloat16() + 0.5
    x[2][x[2] == 0] = 1.0
    g[2, 7] = float("inf")
    plan = bt.bt_adapter_plan([0] * T, 1, device=DEV)
    u = torch.randn(T, R, generator=gen)
    gx, ga, gb = bt.bt_adapter_linear_backward(*(t.to(DEV) for t in (x, g, u, a, b, torch.ones(1))), plan)
    du = g.double() @ b[0].double()
    assert torch.equal(gx[2].cpu().double(), (du @ a[0].double())[2]) and gx[2].isinf().all()
    assert torch.cat([gx[:2], gx[3:]]).isfinite().all()
    assert torch.equal(ga[0].cpu().double(), du.t() @ x.double())              # infinite all over, by x's sign
    assert not gb[0, 7].isfinite().any() and torch.cat([gb[0, :7], gb[0, 8:]]).isfinite().all()


@pytest.mark.parametrize("K", [5, 8])
def test_as_many_adapters_as_a_plan_takes(K, monkeypatch):
    """65536 adapters of rank 1, most of them without a token, widths that are a multiple of 4 and one that is not."""
    monkeypatch.setenv("BT_ADAPTER_PATH", "large")
    L, T, N, R = 65536, 1400, 6, 1
    gen = torch.Generator().manual_seed(6)
    ids = torch.randint(0, L, (T,), generator=gen)
    ids[:600], ids[600] = L - 1, 0                   # one whose tokens are split
    x, a, b = (torch.randn(*s, generator=gen).bfloat16() for s in ((T, K), (L, R, K), (L, N, R)))
    g = torch.randn(T, N, generator=gen).bfloat16()
    d = [t.to(DEV) for t in (x, a, b, torch.ones(L))]
    plan = bt.bt_adapter_plan(ids, L, device=DEV)
    u = torch.empty(T, R, device=DEV)
    out = bt.bt_adapter_linear(*d, plan, out_dtype=torch.float32, u=u).cpu().double()
    xd, ad, bd, gd = x.double(), a.double()[ids], b.double()[ids], g.double()
    ud = torch.einsum("tk,trk->tr", xd, ad)
    size = torch.einsum("tk,trk->tr", xd.abs(), ad.abs())
    assert ((out - torch.einsum("tr,tnr->tn", ud, bd)).abs() <= (K + 2) * 2.0 ** -22 * torch.einsum("tr,tnr->tn", size, bd.abs())).all()
    nan = float("nan")
    gx, ga, gb = bt.bt_adapter_linear_backward(d[0], g.to(DEV), u, *d[1:], plan, grad_a=torch.full(a.shape, nan, device=DEV),
                                               grad_b=torch.full(b.shape, nan, device=DEV))
    du, dsize = torch.einsum("tn,tnr->tr", gd, bd), torch.einsum("tn,tnr->tr", gd.abs(), bd.abs())
    wx, sx = torch.einsum("tr,trk->tk", du, ad), torch.einsum("tr,trk->tk", dsize, ad.abs())
    assert ((gx.cpu().double() - wx).abs() <= 2.0 ** -8 * wx.abs() + (N + 2) * 2.0 ** -22 * sx).all()
    for got, left, mag, right in ((ga, du, dsize, xd), (gb.transpose(1, 2), ud, size, gd)):
        want, bound = (torch.zeros(L, R, right.shape[1]).double().index_add_(0, ids, l[:, :, None] * r[:, None])
                       for l, r in ((left, right), (mag, right.abs())))
        assert ((got.cpu().double() - want).abs() <= 600 * 2.0 ** -22 * bound).all()


def test_a_wait_that_runs_out_is_reported(monkeypatch):
    """With a limit of 1 ns the first wait for a copy or a product in flight gives up: TIMEOUT, once; what is in flight
    still lands, and the next call is as always. (It may have landed by the first look: several calls, the first that did
    not will do.)"""
    monkeypatch.setenv("BT_ADAPTER_PATH", "large")
    T, K, N, R, L = 600, 2048, 1024, 32, 3
    gen = torch.Generator().manual_seed(7)
    x, g = (torch.randn(T, c, generator=gen).bfloat16().to(DEV) for c in (K, N))
    a, b = (torch.randn(*s, generator=gen).bfloat16().to(DEV) for s in ((L, R, K), (L, N, R)))
    scale, plan, u = torch.ones(L, device=DEV), bt.bt_adapter_plan(torch.arange(T) % L, L, device=DEV), torch.empty(T, R, device=DEV)

    def forward():
        return [bt.bt_adapter_linear(x, a, b, scale, plan, u=u)]

    def backward():
        return list(bt.bt_adapter_linear_backward(x, g, u, a, b, scale, plan))

    for call in (forward, backward):
        want = call()
        assert bt.bt_device_status() == 0
        seen = []
        bt.bt_set_wait_timeout(1)
        try:
            while bt.BT_ERR_TIMEOUT not in seen and len(seen) < 200:
                call()
                seen.append(bt.bt_device_status())
        finally:
            bt.bt_set_wait_timeout(0)
        assert set(seen) <= {0, bt.BT_ERR_TIMEOUT} and seen[-1] == bt.BT_ERR_TIMEOUT
        assert bt.bt_device_status() == 0
        assert all(torch.equal(p, q) for p, q in zip(call(), want))


@pytest.mark.parametrize("T", [4, 70])
def test_an_infinite_rank_beside_large_ones_in_half_precision(T, path):
    """u_0 = inf beside u_1 = -1e5 and u_2 = -3e5, beyond half precision's range: the results are +inf, not NaN."""
    K, N, R = 32, 24, 16
    x, a, b = torch.ones(T, K).half(), torch.zeros(1, R, K).half(), torch.ones(1, N, R).half()
    a[0, 0, 3] = float("inf")
    a[0, 1], a[0, 2] = -1e5 / K, -3e5 / K
    plan = bt.bt_adapter_plan([0] * T, 1, device=DEV)
    d = [t.to(DEV) for t in (x, a, b, torch.ones(1))]
    for out_dtype in (torch.float16, torch.float32):
        assert (bt.bt_adapter_linear(*d, plan, out_dtype=out_dtype) == float("inf")).all()
    a[0, 0, 3] = 0
    out = bt.bt_adapter_linear(d[0], a.to(DEV), *d[2:], plan, out_dtype=torch.float32)
    want = (x.double() @ a[0].double().t()).sum(1)[:, None]
    assert ((out.cpu().double() - want).abs() <= K * 2.0 ** -22 * want.abs()).all()
