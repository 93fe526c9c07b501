"""GPU parity of the low-rank adapters (bt_adapter_linear,
bt_adapter_linear_backward) against the formulas in 64 bits on the CPU.

Tolerances. A sum of n products of 16-bit values, exact in fp32, lies within
n 2^-23 sum|terms| of the exact sum (the classical bound n u sum|terms|,
u = 2^-24, doubled). u and dU enter the second product as two 16-bit values,
within 2^-16 of themselves. So, with |.| sums of magnitudes:
  u, dU:   K (N) 2^-23 |x||A|, |g||B| s
  out, dX: s (|B| err(u) + (R 2^-23 + 2^-16) |u||B|) + one step of the result's type
  dA, dB:  |x| err(dU) + (n 2^-23 + 2^-16) |dU||x|, n the adapter's tokens.
"""
import pytest
import torch

import xnor_popcount_gemm_gb300 as bt

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
STEP = {torch.float32: 2.0 ** -23, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -10}
TINY = {torch.float32: 0.0, torch.bfloat16: 0.0, torch.float16: 2.0 ** -24}


@pytest.fixture(autouse=True)
def _device_clean():
    yield
    assert bt.bt_device_status() == 0


@pytest.fixture(params=["small", "large"])
def path(request, monkeypatch):
    """Either forward, whatever the rule on sizes says."""
    monkeypatch.setenv("BT_ADAPTER_PATH", request.param)
    return request.param


def _ids(T, L, kind, seed):
    gen = torch.Generator().manual_seed(seed)
    if kind == "runs":
        ids = torch.randint(0, L, (max(1, T // 50 + 1),), generator=gen).repeat_interleave(50)[:T]
        return torch.cat([ids, ids.new_full((T - ids.numel(),), 0)])
    ids = torch.randint(0, L, (T,), generator=gen)
    if kind == "some":
        ids[torch.rand(T, generator=gen) < 0.3] = -1
    if kind == "skew":                                       # one adapter with most tokens
        ids[torch.rand(T, generator=gen) < 0.8] = L - 1
    return ids


def _inputs(T, K, N, R, L, dtype, seed=0):
    gen = torch.Generator().manual_seed(seed)
    n = lambda *s, std=1.0: (torch.randn(*s, generator=gen) * std).to(dtype)  # noqa: E731
    return n(T, K), n(L, R, K, std=K ** -0.5), n(L, N, R, std=R ** -0.5), torch.rand(L, generator=gen) + 0.5


def _forward(x, a, b, s, ids, base):
    """(out, out's bound before rounding, u, u's bound) in 64 bits."""
    x, a, b, s = x.double(), a.double(), b.double(), s.double()
    T, K, R, N = x.shape[0], x.shape[1], a.shape[1], b.shape[1]
    y = torch.zeros(T, N).double() if base is None else base.double().clone()
    e, u, ue = torch.zeros(T, N).double(), torch.zeros(T, R).double(), torch.zeros(T, R).double()
    for i in ids.unique().tolist():
        if i < 0:
            continue
        r = ids == i
        u[r] = x[r] @ a[i].t()
        ue[r] = K * 2.0 ** -23 * (x[r].abs() @ a[i].abs().t())
        y[r] += s[i] * (u[r] @ b[i].t())
        e[r] = s[i] * (ue[r] @ b[i].abs().t() + (R * 2.0 ** -23 + 2.0 ** -16) * (u[r].abs() @ b[i].abs().t()))
    return y, e, u, ue


def _near(got, want, bound, what):
    got = got.cpu()
    bound = bound + STEP[got.dtype] * want.abs() + TINY[got.dtype]
    bad = ~((got.double() - want).abs() <= bound)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} off, first {bad.nonzero()[0].tolist()}: " \
        f"{got[tuple(bad.nonzero()[0])]} for {want[tuple(bad.nonzero()[0])]}, bound {bound[tuple(bad.nonzero()[0])]}"


def _check_forward(x, a, b, s, ids, base, out_dtype, **kw):
    y, e, u, ue = _forward(x, a, b, s, ids, base)
    plan = bt.bt_adapter_plan(ids, a.shape[0], device=DEV)
    d = [t.to(DEV) for t in (x, a, b, s)]
    bd = None if base is None else base.to(DEV)
    ug = torch.full((x.shape[0], a.shape[1]), 9.0, device=DEV)
    out = bt.bt_adapter_linear(*d, plan, base=bd, out_dtype=out_dtype, u=ug, **kw)
    assert out.dtype == out_dtype
    _near(out, y, e, "out")
    _near(ug, u, ue, "u")
    again = bt.bt_adapter_linear(*d, plan, base=bd, out_dtype=out_dtype)
    assert torch.equal(out, again)
    return out


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("T,K,N,R,L,kind", [
    (1, 64, 64, 8, 1, "all"), (1, 8, 8, 1, 2, "all"), (1, 1, 1, 1, 1, "all"), (2, 96, 40, 16, 2, "all"),
    (7, 65, 33, 3, 3, "some"), (16, 128, 256, 16, 1, "all"), (17, 128, 256, 16, 1, "all"), (33, 130, 70, 24, 1, "all"),
    (64, 256, 512, 32, 48, "some"), (64, 516, 515, 33, 5, "some"), (100, 512, 264, 64, 2, "runs"),
    (129, 260, 128, 128, 2, "some"), (300, 67, 129, 100, 3, "skew"), (500, 192, 200, 40, 4, "skew"),
    (257, 1024, 96, 16, 1, "runs"), (40, 2048, 1100, 64, 40, "some"),
])
def test_forward(T, K, N, R, L, kind, dtype, path):
    x, a, b, s = _inputs(T, K, N, R, L, dtype, seed=T + K)
    ids = _ids(T, L, kind, T)
    gen = torch.Generator().manual_seed(1)
    base = torch.randn(T, N, generator=gen)
    _check_forward(x, a, b, s, ids, base.to(dtype), dtype)
    _check_forward(x, a, b, s, ids, base, torch.float32)
    _check_forward(x, a, b, s, ids, base, dtype)
    _check_forward(x, a, b, s, ids, None, torch.float32)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("T,R,kind", [(1, 16, "all"), (24, 24, "all"), (40, 64, "some"), (300, 8, "runs"), (300, 100, "skew")])
def test_fp32_results_are_not_rounded_between_the_products(T, R, kind, dtype, path):
    """In the 2-norm. u: 512 terms in sums of at most 8 steps that drop less than 2^-23 of a sum each, 4e-7 of it on
    average if all dropped half of that; the second product as much at most in as many steps; u's values in the second
    product 2^-22 and less. They are independent: 8e-7 together. (Two bf16 values of u alone: 2^-18 at most, 1.2e-6.)"""
    x, a, b, s = _inputs(T, 512, 384, R, 3, dtype, seed=R)
    ids = _ids(T, 3, kind, 5)
    want = _forward(x, a, b, s, ids, None)[0]
    plan = bt.bt_adapter_plan(ids, 3)
    got = bt.bt_adapter_linear(*(v.to(DEV) for v in (x, a, b, s)), plan, out_dtype=torch.float32).double().cpu()
    assert (got - want).norm() <= 8e-7 * want.norm()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("T", [3, 200])
def test_strides_in_place_and_views(T, dtype, path):
    K, N, R, L = 72, 104, 16, 3
    x, a, b, s = _inputs(T, K, N, R, L, dtype, seed=3)
    ids = _ids(T, L, "some", 4)
    base = torch.randn(T, N, generator=torch.Generator().manual_seed(2)).to(dtype)
    plan = bt.bt_adapter_plan(ids, L, device=DEV)
    want = _check_forward(x, a, b, s, ids, base, dtype)
    d = [t.to(DEV) for t in (a, b, s)]
    for skew, pitch in ((0, 8), (1, 3), (4, 4), (2, 6)):
        xb = torch.full((T, K + pitch), 77.0, dtype=dtype, device=DEV)
        xv = xb[:, skew:skew + K] if skew + K <= K + pitch else xb[:, :K]
        xv.copy_(x.to(DEV))
        yb = torch.full((T, N + pitch + skew), 55.0, dtype=dtype, device=DEV)
        yv = yb[:, skew:skew + N]
        yv.copy_(base.to(DEV))
        out = bt.bt_adapter_linear(xv, *d, plan, base=yv, out=yv)             # onto the projection's result
        assert out.data_ptr() == yv.data_ptr() and torch.equal(yv, want)
        assert (yb[:, :skew] == 55).all() and (yb[:, skew + N:] == 55).all()
        apart = torch.full((T, N + 5), 33.0, dtype=dtype, device=DEV)
        bt.bt_adapter_linear(xv, *d, plan, base=base.to(DEV), out=apart[:, :N])
        assert torch.equal(apart[:, :N], want) and (apart[:, N:] == 33).all()


def test_nobody_has_an_adapter(path):
    x, a, b, s = _inputs(9, 64, 48, 8, 2, torch.bfloat16)
    ids = torch.full((9,), -1)
    base = torch.randn(9, 48)
    plan = bt.bt_adapter_plan(ids, 2, device=DEV)
    u = torch.ones(9, 8, device=DEV)
    out = bt.bt_adapter_linear(x.to(DEV), a.to(DEV), b.to(DEV), s.to(DEV), plan, base=base.to(DEV), out_dtype=torch.bfloat16, u=u)
    assert torch.equal(out.cpu(), base.to(torch.bfloat16)) and not u.any()
    g = torch.randn(9, 48).bfloat16().to(DEV)
    gx, ga, gb = bt.bt_adapter_linear_backward(x.to(DEV), g, u, a.to(DEV), b.to(DEV), s.to(DEV), plan)
    assert not gx.any() and not ga.any() and not gb.any()


def test_no_tokens():
    a, b, s = (t.to(DEV) for t in _inputs(1, 16, 24, 4, 2, torch.bfloat16)[1:])
    plan = bt.bt_adapter_plan([], 2, device=DEV)
    x = torch.empty(0, 16, dtype=torch.bfloat16, device=DEV)
    assert bt.bt_adapter_linear(x, a, b, s, plan).shape == (0, 24)
    nan = float("nan")
    gx, ga, gb = bt.bt_adapter_linear_backward(x, torch.empty(0, 24, dtype=torch.bfloat16, device=DEV), torch.empty(0, 4, device=DEV),
                                               a, b, s, plan, grad_a=torch.full((2, 4, 16), nan, device=DEV),
                                               grad_b=torch.full((2, 24, 4), nan, device=DEV))
    assert gx.shape == (0, 16) and not ga.any() and not gb.any()


@pytest.mark.parametrize("T", [4, 70])
def test_nan_and_infinity_stay_in_their_rows(T, path):
    x, a, b, s = _inputs(T, 128, 72, 16, 1, torch.bfloat16, seed=5)
    ids = torch.zeros(T, dtype=torch.int64)
    clean = _check_forward(x, a, b, s, ids, None, torch.float32)
    x[1, 5], x[2, 9] = float("nan"), float("inf")
    plan = bt.bt_adapter_plan(ids, 1, device=DEV)
    out = bt.bt_adapter_linear(x.to(DEV), a.to(DEV), b.to(DEV), s.to(DEV), plan, out_dtype=torch.float32)
    assert out[1].isnan().all() and not out[2].isfinite().any()
    keep = [t for t in range(T) if t not in (1, 2)]
    assert torch.equal(out[keep], clean[keep])


@pytest.mark.parametrize("T", [3, 80])
def test_half_precision_reaches_beyond_its_range_inside(T, path):
    """u beyond 65504 and far below 2^-24 in half precision: u is fp32 and enters the second product by rows."""
    K, N, R = 256, 64, 8
    x, a, b, s = _inputs(T, K, N, R, 1, torch.float16, seed=6)
    x[0] = 300.0
    a[0, 0] = 8.0                                            # u[0, 0] = 614400
    x[1] = x[1] * 2.0 ** -12
    a[0, 1:] *= 2.0 ** -6
    b *= 2.0 ** -6
    _check_forward(x, a, b, s, torch.zeros(T, dtype=torch.int64), None, torch.float32)


def _backward(x, g, u, a, b, s, ids, gbase):
    """((gx, bound), (ga, bound), (gb, bound)) in 64 bits."""
    x, g, u, a, b, s = (t.double() for t in (x, g, u, a, b, s))
    R, N = a.shape[1], b.shape[1]
    gx = torch.zeros_like(x) if gbase is None else gbase.double().clone()
    gxe, ga, gae, gb, gbe = (torch.zeros_like(t) for t in (x, a, a, b, b))
    for i in ids.unique().tolist():
        if i < 0:
            continue
        r = ids == i
        n = int(r.sum())
        du = s[i] * g[r] @ b[i]
        due = N * 2.0 ** -23 * s[i] * (g[r].abs() @ b[i].abs())
        gx[r] += du @ a[i]
        gxe[r] = due @ a[i].abs() + (R * 2.0 ** -23 + 2.0 ** -16) * (du.abs() @ a[i].abs())
        ga[i] = du.t() @ x[r]
        gae[i] = due.t() @ x[r].abs() + (n * 2.0 ** -23 + 2.0 ** -16) * (du.abs().t() @ x[r].abs())
        gb[i] = s[i] * (g[r].t() @ u[r])
        gbe[i] = (n * 2.0 ** -23 + 2.0 ** -16) * s[i] * (g[r].abs().t() @ u[r].abs())
    return (gx, gxe), (ga, gae), (gb, gbe)


@pytest.mark.parametrize("T,K,N,R,L,kind", [
    (1, 64, 64, 8, 1, "all"), (1, 1, 1, 1, 1, "all"), (3, 33, 17, 2, 2, "some"), (20, 128, 136, 16, 3, "some"),
    (130, 257, 255, 24, 2, "skew"), (300, 130, 514, 33, 5, "some"), (700, 192, 64, 64, 2, "skew"),
    (1100, 72, 200, 128, 1, "all"), (1500, 100, 93, 24, 3, "runs"), (2000, 64, 320, 16, 8, "skew"), (64, 512, 256, 8, 2, "runs"),
])
def test_backward(T, K, N, R, L, kind):
    x, a, b, s = _inputs(T, K, N, R, L, torch.bfloat16, seed=T)
    ids = _ids(T, L, kind, T)
    gen = torch.Generator().manual_seed(T + 1)
    g = torch.randn(T, N, generator=gen).bfloat16()
    gbase = torch.randn(T, K, generator=gen).bfloat16()
    u = _forward(x, a, b, s, ids, None)[2].float()
    plan = bt.bt_adapter_plan(ids, L, device=DEV)
    d = [t.to(DEV) for t in (x, g, u, a, b, s)]
    for base in (None, gbase):
        want = _backward(x, g, u, a, b, s, ids, base)
        nan = float("nan")
        got = bt.bt_adapter_linear_backward(*d, plan, grad_base=None if base is None else base.to(DEV),
                                            grad_a=torch.full(a.shape, nan, device=DEV),
                                            grad_b=torch.full(b.shape, nan, device=DEV))
        for name, o, (w, e) in zip(("grad_x", "grad_a", "grad_b"), got, want):
            _near(o, w, e, name)
        again = bt.bt_adapter_linear_backward(*d, plan, grad_base=None if base is None else base.to(DEV))
        assert all(torch.equal(p, q) for p, q in zip(got, again))            # sums in a fixed order
    # in place on the projection's own gradient, strided operands
    wide = torch.full((T, K + 3), 5.0, dtype=torch.bfloat16, device=DEV)
    wide[:, 1:1 + K] = gbase.to(DEV)
    gw = torch.zeros(T, N + 1, dtype=torch.bfloat16, device=DEV)
    gw[:, :N] = d[1]
    gx, ga, gb = bt.bt_adapter_linear_backward(d[0], gw[:, :N], *d[2:], plan, grad_base=wide[:, 1:1 + K], grad_x=wide[:, 1:1 + K])
    for name, o, (w, e) in zip(("grad_x", "grad_a", "grad_b"), (gx, ga, gb), want):
        _near(o, w, e, name)
    assert (wide[:, 0] == 5).all() and (wide[:, 1 + K:] == 5).all()


def test_gradients_against_differences():
    """The forward is linear in each of x, A and B alone, so a difference of any length is its derivative up to the
    rounding of the two results: 2^-16 (out's operands) and K 2^-23 of their magnitudes, summed over g."""
    T, K, N, R, L = 6, 24, 16, 4, 2
    x, a, b, s = _inputs(T, K, N, R, L, torch.bfloat16, seed=9)
    ids = torch.tensor([0, 1, 0, -1, 1, 0])
    g = torch.randn(T, N, generator=torch.Generator().manual_seed(10)).bfloat16()
    plan = bt.bt_adapter_plan(ids, L, device=DEV)
    u = torch.empty(T, R, device=DEV)

    def loss(x, a, b):
        y = bt.bt_adapter_linear(x.to(DEV), a.to(DEV), b.to(DEV), s.to(DEV), plan, out_dtype=torch.float32, u=u).cpu().double()
        size = _forward(x.abs(), a.abs(), b.abs(), s, ids, None)[0]
        return float((g.double() * y).sum()), float((g.double().abs() * size).sum()) * (2.0 ** -16 + (K + R) * 2.0 ** -22)

    loss(x, a, b)
    grads = bt.bt_adapter_linear_backward(*(t.to(DEV) for t in (x, g)), u, a.to(DEV), b.to(DEV), s.to(DEV), plan)
    for which, (t, gt) in enumerate(zip((x, a, b), grads)):
        for at in ((0, 3), (5, K - 1)) if which == 0 else ((0, 1, 2), (1, R - 1, 3) if which == 1 else (1, 3, R - 1)):
            p, q = t.clone(), t.clone()
            p[at], q[at] = 1.0, -1.0
            args = [x, a, b]
            hi, lo = ([*args[:which], v, *args[which + 1:]] for v in (p, q))
            (fh, eh), (fl, el) = loss(*hi), loss(*lo)
            d, got = (fh - fl) / 2, float(gt[at])
            assert abs(d - got) <= (eh + el) / 2 + 2.0 ** -8 * abs(got), (which, at, d, got)


def test_another_stream_and_a_graph(path):
    T, K, N, R, L = 200, 256, 264, 16, 3
    x, a, b, s = (t.to(DEV) for t in _inputs(T, K, N, R, L, torch.bfloat16, seed=11))
    ids = _ids(T, L, "some", 12)
    plan = bt.bt_adapter_plan(ids, L, device=DEV)
    want = bt.bt_adapter_linear(x, a, b, s, plan)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    got = bt.bt_adapter_linear(x, a, b, s, plan, stream=st)
    st.synchronize()
    assert torch.equal(got, want)
    out, u = torch.zeros_like(want), torch.zeros(T, R, device=DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        bt.bt_adapter_linear(x, a, b, s, plan, out=out, u=u)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)


def test_offsets_beyond_32_bits(path):
    T, K, N, R = 70000, 32768, 64, 8                          # x holds 2.3e9 elements
    x = torch.zeros(T, K, dtype=torch.bfloat16, device=DEV)
    xs, a, b, s = _inputs(2, K, N, R, 2, torch.bfloat16, seed=13)
    x[-2:] = xs.to(DEV)
    for kind in ("few", "many"):
        ids = torch.full((T,), -1)
        ids[-2:] = torch.tensor([1, 0])
        if kind == "many":
            ids[-200:-2] = 1
        y, e, u, ue = _forward(xs, a, b, s, ids[-2:], None)
        plan = bt.bt_adapter_plan(ids, 2, device=DEV)
        ug = torch.empty(T, R, device=DEV)
        out = bt.bt_adapter_linear(x, a.to(DEV), b.to(DEV), s.to(DEV), plan, out_dtype=torch.float32, u=ug)
        _near(out[-2:], y, e, "out")
        _near(ug[-2:], u, ue, "u")
        assert not out[:-2].any()
        g = torch.zeros(T, N, dtype=torch.bfloat16, device=DEV)
        g[-2:] = torch.randn(2, N, generator=torch.Generator().manual_seed(14)).bfloat16().to(DEV)
        want = _backward(xs, g[-2:].cpu(), u.float(), a, b, s, ids[-2:], None)
        ug[-2:] = u.float().to(DEV)
        got = bt.bt_adapter_linear_backward(x, g, ug, a.to(DEV), b.to(DEV), s.to(DEV), plan)
        _near(got[0][-2:], *want[0], "grad_x")
        assert not got[0][:-2].any()
        _near(got[1], *want[1], "grad_a")
        _near(got[2], *want[2], "grad_b")
