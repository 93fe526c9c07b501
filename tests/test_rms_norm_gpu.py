"""RMS norm with the residual's addition and microscaled results, and its backward, against 64 bits (GPU)."""
import math

import pytest
import torch

import xnor_popcount_gemm_gb300 as bt

pytestmark = pytest.mark.gpu
E4M3, E2M1 = bt.BT_CODE_E4M3, bt.BT_CODE_E2M1
F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
# widths: one, below and above a block, aligned and not, several loads a thread, wider than a CTA's registers
WIDTHS = [1, 8, 31, 32, 33, 100, 256, 1000, 4093, 4096, 8200, 11008, 16385, 20000, 33000, 70000]


def rows(seed, T, N, dtype, spread=1.0):
    gen = torch.Generator().manual_seed(seed)
    x = torch.randn(T, N, generator=gen) * torch.exp(spread * torch.randn(T, 1, generator=gen))
    x *= torch.where(torch.rand(N, generator=gen) < 0.02, 25.0, 1.0)
    return x.to(dtype).cuda()


def exact(h, w, eps):
    h = h.double()
    return h / torch.sqrt(h.square().mean(dim=1, keepdim=True) + eps) * (1.0 if w is None else w.double())


def check_rounding(y, y64):
    """The fp32 value is the nearest one but for a few in 2^24, which are one step off: then the 16-bit one hardly ever is."""
    want = y64.float().to(y.dtype)
    off = y != want
    assert int(off.sum()) <= 1 + y.numel() // (1 << 20), int(off.sum())
    assert bool(((y.double() - want.double()).abs()[off] <= want.double().abs()[off] * torch.finfo(y.dtype).eps).all())


def same_operand(a, b):
    n = a.codes.shape[1] // (16 if a.code == E2M1 else 32)
    from mx_reference import scale_at
    at = scale_at(a.shape[0], n, a.K, a.code).cuda()
    return torch.equal(a.codes, b.codes) and torch.equal(a.scales[at], b.scales[at])


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("N", WIDTHS)
def test_norm(N, dtype):
    T = 5 if N < 20000 else 2
    x, r = rows(N, T, N, dtype), rows(N + 1, T, N, dtype, 0.3)
    w = (1.0 + 0.3 * torch.randn(N, generator=torch.Generator().manual_seed(N))).cuda().to(dtype)
    h = (x.float() + r.float()).to(dtype)
    for residual, total in ((None, x), (r, h)):
        y, s, q = bt.bt_rms_norm(x, w, 1e-6, residual=residual)
        assert q is None and (s is None if residual is None else torch.equal(s, h))
        check_rounding(y, exact(total, w, 1e-6))
        for code in (E4M3, E2M1):
            y2, s, q = bt.bt_rms_norm(x, w, 1e-6, residual=residual, code=code)
            assert torch.equal(y, y2) and same_operand(q, bt.bt_mx_quantize(y, code))
            none, s, q2 = bt.bt_rms_norm(x, w, 1e-6, residual=residual, code=code, want_out=False)
            assert none is None and same_operand(q, q2)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("T,N", [(1, 4096), (400, 4096), (700, 256), (330, 1001), (400, 12000), (1300, 4093), (1300, 2048), (2500, 128), (5000, 64),
                                 (30000, 96), (2600, 512), (2600, 1000), (2433, 1024), (2600, 90)])
def test_norm_many_rows_and_weights(T, N, dtype):
    x = rows(T, T, N, dtype)
    for w in (None, torch.rand(N).cuda() + 0.5, (torch.rand(N).cuda() - 0.5).to(dtype)):
        y, _, q = bt.bt_rms_norm(x, w, 1e-5, code=E2M1)
        check_rounding(y, exact(x, w, 1e-5))
        assert same_operand(q, bt.bt_mx_quantize(y, E2M1))


@pytest.mark.parametrize("N", [64, 100, 40000])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_norm_of_any_size_of_values(N, dtype):
    x = torch.randn(8, N)
    sizes = [1e30, 1e20, 1e-15, 1e-22, 1e-36, 1e18, 3e-39, 1.0]
    x = (x.double() * torch.tensor(sizes, dtype=torch.float64).view(-1, 1)).float().to(dtype).cuda()
    y, _, _ = bt.bt_rms_norm(x, None, 0.0)
    # values that are no normal fp32 numbers have fewer digits, not their norm
    check_rounding(y, exact(x, None, 0.0))
    y, _, _ = bt.bt_rms_norm(x, None, 1e-6)
    tiny = exact(x, None, 1e-6).abs() < 1e-30               # results next to fp32's end round in its steps
    y64 = exact(x, None, 1e-6)
    check_rounding(torch.where(tiny, torch.zeros_like(y), y), torch.where(tiny, torch.zeros_like(y64), y64))
    assert bool(((y.double() - y64).abs()[tiny] <= y64.abs()[tiny] * 2.0 ** -7 + 1e-40).all())


@pytest.mark.parametrize("N", [96, 101, 33000])
def test_norm_special_rows(N):
    x = torch.randn(5, N)
    x[0] = 0
    x[1, N // 2] = math.nan
    x[2, 3] = math.inf
    x[3, 4] = -math.inf
    x = x.to(BF16).cuda()
    y, _, q = bt.bt_rms_norm(x, None, 1e-6, code=E4M3)
    y = y.cpu()
    assert int(y[0].count_nonzero()) == 0 and bool(torch.isnan(y[1]).all())
    for i, c in ((2, 3), (3, 4)):
        assert bool(torch.isnan(y[i, c])) and int(torch.nan_to_num(y[i]).count_nonzero()) == 0 and int(torch.isnan(y[i]).sum()) == 1
    assert same_operand(q, bt.bt_mx_quantize(y.cuda(), E4M3))
    y, _, _ = bt.bt_rms_norm(x, None, 0.0)
    assert bool(torch.isnan(y[0]).all())                    # 0 / 0


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("N,ld,skip", [(256, 264, 0), (256, 257, 0), (100, 104, 8), (100, 100, 1), (4096, 4100, 3), (33000, 33003, 1)])
def test_norm_strides_and_in_place(N, ld, skip, dtype):
    T = 3

    def strided(t):
        buf = torch.full((T * ld + skip + 32,), 7.0, dtype=dtype, device="cuda")
        v = buf[skip:].as_strided((T, N), (ld, 1))
        if t is not None:
            v.copy_(t)
        return buf, v

    def untouched(buf):
        rest = torch.ones_like(buf, dtype=torch.bool)
        rest[skip:].as_strided((T, N), (ld, 1)).fill_(False)
        return bool((buf[rest] == 7.0).all())

    x, r = rows(1, T, N, dtype), rows(2, T, N, dtype)
    w = torch.rand(N).cuda().to(dtype)
    y, h, q = bt.bt_rms_norm(x, w, residual=r, code=E2M1)
    (bx, sx), (br, sr), (bs, ss), (bo, so) = strided(x), strided(r), strided(None), strided(None)
    a, b, c = bt.bt_rms_norm(sx, w, residual=sr, sum=ss, out=so, code=E2M1)
    assert a is so and b is ss and torch.equal(so, y) and torch.equal(ss, h) and same_operand(c, q)
    assert all(map(untouched, (bx, br, bs, bo)))
    # the sum over the residual, the result over x
    bt.bt_rms_norm(sx, w, residual=sr, sum=sr, out=sx)
    assert torch.equal(sr, h) and torch.equal(sx, y) and untouched(bx) and untouched(br)
    # the sum over x
    sx.copy_(x)
    sr.copy_(r)
    y3, _, _ = bt.bt_rms_norm(sx, w, residual=sr, sum=sx)
    assert torch.equal(sx, h) and torch.equal(y3, y)


# ---------------------------------------------------------------------------
def check_backward(T, N, dtype, residual=True, weight=True, seed=0, scale=1.0):
    h, g = (rows(seed + 1, T, N, F32) * scale).to(dtype), (rows(seed + 2, T, N, F32) * 0.01).to(dtype)
    gs = rows(seed + 3, T, N, dtype) if residual else None
    w = (1.0 + 0.3 * torch.randn(N, generator=torch.Generator().manual_seed(seed))).cuda().to(dtype) if weight else None
    eps = 1e-6
    gx, gw = bt.bt_rms_norm_backward(g, h, w, eps, grad_sum=gs)
    h64, g64, w64 = h.double(), g.double(), torch.ones(N, device="cuda").double() if w is None else w.double()
    inv = 1.0 / torch.sqrt(h64.square().mean(dim=1, keepdim=True) + eps)
    n = h64 * inv
    gwn = g64 * w64 * n
    want = inv * (g64 * w64 - n * gwn.mean(dim=1, keepdim=True))
    # a row's sums: a thread's part one after the other (at most 140 values), a tree above it; a few roundings a value
    c = 160 * 2.0 ** -24
    bound = c * inv * ((g64 * w64).abs() + n.abs() * gwn.abs().mean(dim=1, keepdim=True))
    if gs is not None:
        want = want + gs.double()
    bound = bound + want.abs() * (torch.finfo(dtype).eps / 2 + 2.0 ** -23) + torch.finfo(dtype).smallest_normal
    assert bool(((gx.double() - want).abs() <= bound).all())
    gw64 = (g64 * n).sum(dim=0)
    # rows one after the other, n itself to a few roundings and its row's sum
    assert bool(((gw.double() - gw64).abs() <= (T + 160) * 2.0 ** -24 * (g64 * n).abs().sum(dim=0) + 1e-37).all())
    return gx, gw, (h, g, gs, w)


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("N", WIDTHS)
def test_backward(N, dtype):
    check_backward(4 if N < 20000 else 2, N, dtype)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("T,N", [(1, 64), (3, 4096), (400, 512), (777, 1001), (1300, 96), (650, 4096), (40, 12000), (2500, 128), (2433, 8), (9000, 31),
                                 (2600, 512), (2600, 1000), (2433, 1024), (2600, 777), (700, 8192), (310, 16384), (310, 11005)])
def test_backward_many_rows(T, N, dtype):
    for residual, weight in ((True, True), (False, True), (False, False)):
        check_backward(T, N, dtype, residual, weight, seed=T)


@pytest.mark.parametrize("N", [128, 129])
@pytest.mark.parametrize("scale", [1e25, 1e-25])
def test_backward_of_any_size_of_values(N, scale):
    check_backward(6, N, F32, residual=False, scale=scale)


def test_backward_without_weight_gradient_and_in_place():
    for N in (256, 257):
        gx, gw, (h, g, gs, w) = check_backward(30, N, BF16)
        a, none = bt.bt_rms_norm_backward(g, h, w, grad_sum=gs, want_grad_weight=False)
        assert none is None and torch.equal(a, gx)
        for which in range(3):
            t = [g.clone(), h.clone(), gs.clone()]
            a, b = bt.bt_rms_norm_backward(t[0], t[1], w, grad_sum=t[2], grad_x=t[which])
            assert torch.equal(a, gx) and torch.equal(b, gw) and a is t[which]


@pytest.mark.parametrize("N,ld,skip", [(256, 264, 8), (256, 259, 1), (101, 107, 3)])
def test_backward_strides(N, ld, skip):
    T = 20
    gx, gw, (h, g, gs, w) = check_backward(T, N, BF16)

    def strided(t):
        buf = torch.full((T * ld + skip + 32,), 7.0, dtype=BF16, device="cuda")
        v = buf[skip:].as_strided((T, N), (ld, 1))
        if t is not None:
            v.copy_(t)
        return buf, v

    buf, out = strided(None)
    a, b = bt.bt_rms_norm_backward(strided(g)[1], strided(h)[1], w, grad_sum=strided(gs)[1], grad_x=out)
    # (aligned rows are summed in another order than others)
    assert bool(((a.double() - gx.double()).abs() <= gx.double().abs() * 2.0 ** -7 + 1e-6).all())
    assert bool(((b - gw).abs() <= 1e-4 * gw.abs().max()).all())
    rest = torch.ones_like(buf, dtype=torch.bool)
    rest[skip:].as_strided((T, N), (ld, 1)).fill_(False)
    assert bool((buf[rest] == 7.0).all())


def test_backward_is_the_gradient():
    # against central differences of the 64-bit norm: their error is of order step^2, their rounding 1e-16 / step
    gen = torch.Generator().manual_seed(9)
    T, N = 4, 48
    h, g, w, v = (torch.randn(*s, generator=gen, dtype=torch.float64) for s in ((T, N), (T, N), (N,), (T, N)))
    h, g, w = h.float().double(), g.float().double(), w.float().double()
    gx, gw = bt.bt_rms_norm_backward(g.float().cuda(), h.float().cuda(), w.float().cuda(), 1e-6)
    loss = lambda a, b: float((g * a / torch.sqrt(a.square().mean(dim=1, keepdim=True) + 1e-6) * b).sum())  # noqa: E731
    step = 1e-5
    diff = (loss(h + step * v, w) - loss(h - step * v, w)) / (2 * step)
    size = float(g.abs().sum())
    assert abs(float((gx.cpu().double() * v).sum()) - diff) <= 1e-6 * size
    u = torch.randn(N, generator=gen, dtype=torch.float64)
    diff = (loss(h, w + step * u) - loss(h, w - step * u)) / (2 * step)
    assert abs(float((gw.cpu().double() * u).sum()) - diff) <= 1e-6 * size


def test_rows_far_apart():
    # offsets beyond 32 bits, in every operand
    ld, T, N = (1 << 30) + 24, 3, 200
    def far(t):
        buf = torch.empty((T - 1) * ld + N, dtype=BF16, device="cuda")
        v = buf.as_strided((T, N), (ld, 1))
        v.copy_(t)
        return v
    x, r, g = rows(1, T, N, BF16), rows(2, T, N, BF16), rows(3, T, N, BF16)
    y, h, q = bt.bt_rms_norm(x, None, residual=r, code=E4M3)
    gx, gw = bt.bt_rms_norm_backward(g, h)
    fx, fr, fo = far(x), far(r), far(x)
    y2, h2, q2 = bt.bt_rms_norm(fx, None, residual=fr, sum=fr, out=fo, code=E4M3)
    assert torch.equal(y2, y) and torch.equal(h2, h) and same_operand(q, q2)
    assert same_operand(q, bt.bt_mx_quantize(fo, E4M3))
    bt.bt_mx_dequantize(q, out=fx)
    assert torch.equal(fx, bt.bt_mx_dequantize(q, BF16))
    fx.copy_(g)
    gx2, gw2 = bt.bt_rms_norm_backward(fx, fr, grad_x=fo)
    assert torch.equal(gx2, gx) and torch.equal(gw2, gw)


def test_empty_and_graph():
    y, s, q = bt.bt_rms_norm(torch.empty(0, 64, device="cuda"), None, residual=torch.empty(0, 64, device="cuda"), code=E2M1)
    assert y.shape == s.shape == q.shape == (0, 64)
    gw = torch.ones(64, device="cuda")
    bt.bt_rms_norm_backward(torch.empty(0, 64, device="cuda"), torch.empty(0, 64, device="cuda"), grad_weight=gw)
    assert int(gw.count_nonzero()) == 0
    x, g = rows(1, 40, 512, BF16), rows(2, 40, 512, BF16)
    want = bt.bt_rms_norm(x)[0], *bt.bt_rms_norm_backward(g, x)
    y, gx, gw = torch.zeros_like(x), torch.zeros_like(x), torch.zeros(512, device="cuda")
    ws = torch.empty(bt.bt_rms_norm_backward_workspace(40, 512), dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        bt.bt_rms_norm(x, out=y)
        bt.bt_rms_norm_backward(g, x, grad_x=gx, grad_weight=gw, workspace=ws)
    graph.replay()
    assert all(torch.equal(a, b) for a, b in zip((y, gx, gw), want))


# Several short rows to a warp: the last warp with some rows only, rows whose squares leave fp32 beside ordinary ones, rows of
# zeros without eps, and what lies behind the last row left as it was.
SHORT = [(2433, 128), (2435, 64), (2561, 120), (5003, 8), (2439, 72), (30001, 40)]


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("T,N", SHORT)
def test_norm_of_many_short_rows(T, N, dtype):
    x = rows(T, T, N, dtype)
    big, small = (0.0, 0.0) if dtype == F16 else (1e25, 1e-25)
    if big:
        x[5::7] = (x[5::7].float() / x[5::7].float().abs().amax(1, keepdim=True) * big).to(dtype)
        x[3::11] = (x[3::11].float() / x[3::11].float().abs().amax(1, keepdim=True) * small).to(dtype)
    w = (torch.rand(N, generator=torch.Generator().manual_seed(N)) + 0.5).cuda()
    for code in (E4M3, E2M1):
        buf = torch.full((T + 8, N), 7.0, dtype=dtype, device="cuda")
        _, _, q = bt.bt_rms_norm(x, w, 0.0, out=buf[:T], code=code)
        check_rounding(buf[:T], exact(x, w, 0.0))
        assert bool((buf[T:] == 7.0).all())
        assert same_operand(q, bt.bt_mx_quantize(buf[:T], code))
    x[T - 1] = 0                                # 0 / 0
    y, _, _ = bt.bt_rms_norm(x, w, 0.0)
    assert bool(torch.isnan(y[T - 1]).all()) and torch.equal(y[:T - 1], buf[:T - 1])


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("T,N", SHORT + [(2433, 127), (2434, 33)])
def test_backward_of_many_short_rows(T, N, dtype):
    gx, gw, (h, g, gs, w) = check_backward(T, N, dtype, seed=T)
    buf = torch.full((T + 8, N), 7.0, dtype=dtype, device="cuda")
    a, b = bt.bt_rms_norm_backward(g, h, w, grad_sum=gs, grad_x=buf[:T])
    assert torch.equal(a, gx) and torch.equal(b, gw) and bool((buf[T:] == 7.0).all())
    # without eps: rows behind the last add nothing, not 0 / 0
    a, b = bt.bt_rms_norm_backward(g, h, w, 0.0, grad_sum=gs)
    assert bool(torch.isfinite(a).all()) and bool(torch.isfinite(b).all())
