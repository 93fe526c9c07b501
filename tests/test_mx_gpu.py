"""Microscaled operands and the products on them against their definition in 64 bits (GPU)."""
import math

import pytest
import torch

import xnor_popcount_gemm_gb300 as bt
from mx_reference import quantized, unpacked

pytestmark = pytest.mark.gpu
E4M3, E2M1 = bt.BT_CODE_E4M3, bt.BT_CODE_E2M1
CODES = [E4M3, E2M1]
F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16


def activations(gen, R, K, dtype):
    x = torch.randn(R, K, generator=gen) * torch.exp(2 * torch.randn(R, 1, generator=gen))
    x *= torch.where(torch.rand(K, generator=gen) < 0.05, 30.0, 1.0)
    return x.to(dtype)


def check_operand(q, x):
    values, mag, scales = quantized(x, q.code)
    got_mag, got_sign, got_scales = unpacked(q)
    n = mag.shape[1]
    assert torch.equal(got_scales[:, :n // 32], scales.long())
    assert torch.equal(got_mag[:, :n], mag)
    assert int(got_mag[:, n:].sum()) == 0
    sign = torch.nn.functional.pad((x < 0).long(), (0, n - x.shape[1]))
    assert torch.equal(got_sign[:, :n][mag > 0], sign[mag > 0])
    return values


@pytest.mark.parametrize("code", CODES)
@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("R,K", [(1, 1), (1, 32), (3, 33), (7, 255), (130, 256), (129, 257), (64, 4100), (300, 1024), (5, 9000)])
def test_quantize_is_the_definition(code, dtype, R, K):
    x = activations(torch.Generator().manual_seed(R * 10007 + K), R, K, dtype)
    x[0, :1] = 0
    if R > 2:
        x[1] = 0
        x[2, ::2] = 0
    q = bt.bt_mx_quantize(x.cuda(), code)
    values = check_operand(q, x.float())
    # exact in fp32 and bf16
    for dt in (F32, BF16):
        assert torch.equal(bt.bt_mx_dequantize(q, dt).cpu().double(), values)
    assert torch.equal(bt.bt_mx_dequantize(q, F16).cpu(), values.float().to(F16))


@pytest.mark.parametrize("code", CODES)
def test_quantize_borders_and_range(code):
    # every midpoint and its neighbours, both signs, in blocks of every exponent that fp32 has
    from mx_reference import FORMAT, table
    t = table(code)
    mids = ((t[1:] + t[:-1]) / 2).float()
    vals = torch.cat([t.float(), mids, torch.nextafter(mids, torch.tensor(9e9)), torch.nextafter(mids, torch.tensor(0.0))])
    vals = torch.cat([vals, -vals])
    emax = FORMAT[code][2]
    rows = []
    for e in [-149, -140, -130, -127, -126, -125, -60, -3, 0, 1, 40, 100, 127 - emax]:
        block = torch.zeros(len(vals), 32)
        block[:, 0] = 2.0 ** emax                       # the block's largest magnitude
        block[:, 1] = vals.clamp(-2.0 ** emax * 1.99, 2.0 ** emax * 1.99)
        block[:, 5] = -block[:, 1]
        rows.append(torch.ldexp(block.double(), torch.tensor(e)).float())
    x = torch.cat(rows)
    q = bt.bt_mx_quantize(x.cuda(), code)
    values = check_operand(q, x)
    assert torch.equal(bt.bt_mx_dequantize(q, F32).cpu().double(), values.float().double())


@pytest.mark.parametrize("code", CODES)
@pytest.mark.parametrize("dtype", [F32, BF16, F16])
def test_quantize_nan_infinity_and_largest(code, dtype):
    x = torch.randn(6, 96).to(dtype)
    x[0, 3] = math.nan
    x[1, 40] = math.inf
    x[2, 70] = -math.inf
    x[3, :] = torch.finfo(dtype).max
    x[4, :] = torch.finfo(dtype).smallest_normal / 4
    x[5, 0] = torch.finfo(dtype).min
    q = bt.bt_mx_quantize(x.cuda(), code)
    check_operand(q, x.float())
    v = bt.bt_mx_dequantize(q, F32).cpu()
    want = quantized(x.float(), code)[0].float()
    assert torch.equal(torch.isnan(v), torch.isnan(want)) and int(torch.isnan(v).sum()) == 96
    assert torch.equal(torch.nan_to_num(v), torch.nan_to_num(want))


@pytest.mark.parametrize("code", CODES)
@pytest.mark.parametrize("K,ld,skip", [(100, 100, 1), (64, 67, 3), (96, 104, 8), (4100, 4100, 2)])
def test_quantize_strides_and_alignment(code, K, ld, skip):
    R = 9
    buf = torch.randn(R * ld + skip).to(BF16).cuda()
    x = buf[skip:].as_strided((R, K), (ld, 1))
    q = bt.bt_mx_quantize(x, code)
    check_operand(q, x.cpu().float())
    out = torch.full((R * ld + skip + 8,), 7.0, dtype=F32, device="cuda")
    o = out[skip:].as_strided((R, K), (ld, 1))
    bt.bt_mx_dequantize(q, out=o)
    assert torch.equal(o, bt.bt_mx_dequantize(q))
    rest = torch.ones_like(out, dtype=torch.bool)
    rest[skip:].as_strided((R, K), (ld, 1)).fill_(False)
    assert bool((out[rest] == 7.0).all())


@pytest.mark.parametrize("code", CODES)
@pytest.mark.parametrize("N,K", [(1, 1), (64, 64), (65, 130), (200, 300), (4093, 260)])
def test_transpose(code, N, K):
    w = (torch.randn(N, K, generator=torch.Generator().manual_seed(N + K)) * 0.02).to(BF16).cuda()
    q = bt.bt_mx_quantize(w, code)
    t = bt.bt_mx_transpose(q)
    ld = bt.bt_backward_weight_ld(N)
    assert t.shape == (K, ld)
    assert torch.equal(t[:, :N], bt.bt_mx_dequantize(q, BF16).t())
    assert int(t[:, N:].count_nonzero()) == 0
    t = bt.bt_mx_transpose(q, ld=(N + 7) // 8 * 8)
    assert torch.equal(t[:, :N], bt.bt_mx_dequantize(q, BF16).t())


def linear_bound(xv, wv, y, K, out_dtype):
    """fp32 sums that cut off: K / 32 steps (the shorter instruction's) and a few inside them, each at most 2^-23 of the
    magnitudes summed so far; then one rounding."""
    terms = xv.abs() @ wv.abs().t()
    return (K / 32 + 8) * 2.0 ** -23 * terms + y.abs() * torch.finfo(out_dtype).eps / 2 + torch.finfo(out_dtype).smallest_normal


def check_linear(M, N, K, code, dtype=BF16, out_dtype=BF16, packed=False, seed=0, out=None):
    gen = torch.Generator().manual_seed(seed + M * 7 + N * 13 + K)
    x = activations(gen, M, K, dtype).cuda()
    w = (torch.randn(N, K, generator=gen) * torch.exp(torch.randn(N, 1, generator=gen)) * 0.05).to(BF16).cuda()
    wq, xq = bt.bt_mx_quantize(w, code), bt.bt_mx_quantize(x, code)
    y = bt.bt_mx_linear(xq if packed else x, wq, out_dtype=out_dtype, out=out)
    xv, wv = bt.bt_mx_dequantize(xq).double(), bt.bt_mx_dequantize(wq).double()
    want = xv @ wv.t()
    off = (y.double() - want).abs()
    bound = linear_bound(xv, wv, want, K, out_dtype)
    assert bool((off <= bound).all()), (float((off - bound).max()), float((off / want.abs().mean()).max()))
    assert bt.bt_device_status() == 0
    return y


SHAPES = [(1, 1, 1), (1, 128, 32), (2, 300, 64), (5, 130, 100), (16, 256, 256), (17, 100, 4100), (33, 260, 512), (64, 512, 1000),
          (100, 129, 260), (128, 256, 2048), (129, 385, 640), (200, 1000, 300), (256, 512, 1024), (300, 517, 777),
          (777, 1093, 1100), (1030, 2050, 512)]


@pytest.mark.parametrize("code", CODES)
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_linear(code, M, N, K):
    check_linear(M, N, K, code)


@pytest.mark.parametrize("code", CODES)
@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("out_dtype", [F32, BF16, F16])
@pytest.mark.parametrize("M,N,K", [(3, 200, 300), (150, 264, 520), (300, 301, 300)])
def test_linear_types(code, dtype, out_dtype, M, N, K):
    check_linear(M, N, K, code, dtype, out_dtype)
    check_linear(M, N, K, code, dtype, out_dtype, packed=True)


@pytest.mark.parametrize("config", ["256,1", "128,1", "256,2", "128,2", "128,3", "pair,256,1", "pair,128,1", "pair,256,2", "pair,128,2",
                                    "pair,128,3", "256,1,4", "pair,256,1,4", "pair,128,2,4"])
@pytest.mark.parametrize("code", CODES)
def test_linear_every_shape_of_tiles(code, config, monkeypatch):
    monkeypatch.setenv("BT_MX_CONFIG", config)
    for M, N, K in [(1, 1, 1), (300, 517, 777), (515, 1290, 2300), (1500, 2600, 1300)]:
        check_linear(M, N, K, code, out_dtype=F32)
    check_linear(4000, 5000, 520, code)                     # several tiles a CTA


@pytest.mark.parametrize("split", [1, 2, 4, 8])
@pytest.mark.parametrize("code", CODES)
def test_linear_few_rows_every_split(code, split, monkeypatch):
    monkeypatch.setenv("BT_MX_CONFIG", f"small,{split}")
    for M, N, K in [(1, 1, 1), (1, 300, 2000), (7, 129, 1300), (16, 260, 4100), (17, 100, 3333), (32, 513, 2560), (31, 128, 9000)]:
        for packed in (False, True):
            check_linear(M, N, K, code, F32, F32, packed=packed)
            check_linear(M, N, K, code, F16, BF16, packed=packed)


@pytest.mark.parametrize("code", CODES)
def test_linear_few_rows_of_strided_x(code):
    for M, K, ld, skip in [(3, 1000, 1003, 1), (20, 257, 300, 4), (32, 512, 513, 0)]:
        for dtype in (F32, BF16, F16):
            buf = torch.randn(M * ld + skip).to(dtype).cuda()
            x = buf[skip:].as_strided((M, K), (ld, 1))
            wq = bt.bt_mx_quantize(torch.randn(200, K).cuda(), code)
            assert torch.equal(bt.bt_mx_linear(x, wq, out_dtype=F32), bt.bt_mx_linear(bt.bt_mx_quantize(x, code), wq, out_dtype=F32))


@pytest.mark.parametrize("code", CODES)
def test_linear_blocks_of_all_sizes(code):
    # blocks whose scales differ by up to 2^40 between neighbours, and rows of zeros
    gen = torch.Generator().manual_seed(5)
    M, N, K = 70, 140, 640
    x = torch.randn(M, K, generator=gen).view(M, -1, 32) * torch.exp2(torch.randint(-20, 20, (M, K // 32, 1), generator=gen).float())
    w = torch.randn(N, K, generator=gen).view(N, -1, 32) * torch.exp2(torch.randint(-20, 20, (N, K // 32, 1), generator=gen).float())
    x, w = x.view(M, K), w.view(N, K)
    x[3], w[5] = 0, 0
    xq, wq = bt.bt_mx_quantize(x.cuda(), code), bt.bt_mx_quantize(w.cuda(), code)
    xv, wv = bt.bt_mx_dequantize(xq).double(), bt.bt_mx_dequantize(wq).double()
    want = xv @ wv.t()
    y = bt.bt_mx_linear(xq, wq, out_dtype=F32)
    assert bool(((y.double() - want).abs() <= linear_bound(xv, wv, want, K, F32)).all())
    assert int(y[3].count_nonzero()) == 0 and int(y[:, 5].count_nonzero()) == 0


@pytest.mark.parametrize("code", CODES)
@pytest.mark.parametrize("M", [4, 200])
def test_linear_nan_stays_in_its_row(code, M):
    N, K = 150, 320
    x, w = torch.randn(M, K), torch.randn(N, K)
    x[1, 37] = math.nan
    x[2, 319] = math.inf
    w[149, 0] = math.nan
    y = bt.bt_mx_linear(x.cuda(), bt.bt_mx_quantize(w.cuda(), code), out_dtype=F32).cpu()
    want = torch.zeros(M, N, dtype=torch.bool)
    want[1:3], want[:, 149] = True, True
    assert torch.equal(torch.isnan(y), want)


@pytest.mark.parametrize("code", CODES)
@pytest.mark.parametrize("M,N,ld,skip", [(5, 100, 104, 0), (5, 100, 131, 3), (200, 333, 400, 1), (200, 256, 264, 8)])
def test_linear_strided_result(code, M, N, ld, skip):
    buf = torch.full((M * ld + skip + 64,), 7.0, dtype=BF16, device="cuda")
    out = buf[skip:].as_strided((M, N), (ld, 1))
    y = check_linear(M, N, 300, code, out=out)
    assert y is out
    rest = torch.ones_like(buf, dtype=torch.bool)
    rest[skip:].as_strided((M, N), (ld, 1)).fill_(False)
    assert bool((buf[rest] == 7.0).all())


@pytest.mark.parametrize("code", CODES)
@pytest.mark.parametrize("M,N,K", [(1, 8, 1), (3, 5, 7), (64, 128, 64), (100, 4093, 260), (300, 520, 1030)])
@pytest.mark.parametrize("out_dtype", [BF16, F32])
def test_linear_backward(code, M, N, K, out_dtype):
    gen = torch.Generator().manual_seed(M + N + K)
    g = (torch.randn(M, N, generator=gen) * 0.01).to(BF16).cuda()
    wq = bt.bt_mx_quantize((torch.randn(N, K, generator=gen) * 0.02).cuda(), code)
    wv = bt.bt_mx_dequantize(wq).double()
    gx = bt.bt_mx_linear_backward(g, bt.bt_mx_transpose(wq), out_dtype=out_dtype)
    want = g.double() @ wv
    # N / 16 instructions' sums, each off by at most 2^-23 of what was summed
    bound = (N / 16 + 8) * 2.0 ** -23 * (g.double().abs() @ wv.abs()) + want.abs() * torch.finfo(out_dtype).eps / 2 + 1e-30
    assert bool(((gx.double() - want).abs() <= bound).all())
    # strided, unaligned g
    buf = torch.randn(M * (N + 3) + 1).to(BF16).cuda()
    gs = buf[1:].as_strided((M, N), (N + 3, 1))
    gs.copy_(g)
    assert torch.equal(bt.bt_mx_linear_backward(gs, bt.bt_mx_transpose(wq), out_dtype=out_dtype), gx)


def test_linear_backward_is_the_gradient():
    # against differences of the 64-bit product of the dequantised values: linear, so a difference is exact
    g = torch.randn(9, 40, dtype=torch.float64)
    wq = bt.bt_mx_quantize(torch.randn(40, 70).cuda(), E4M3)
    wv = bt.bt_mx_dequantize(wq).double().cpu()
    gb = g.to(BF16)
    gx = bt.bt_mx_linear_backward(gb.cuda(), bt.bt_mx_transpose(wq), out_dtype=F32).double().cpu()
    x, v = torch.randn(9, 70, dtype=torch.float64), torch.randn(9, 70, dtype=torch.float64)
    loss = lambda t: float((gb.double() * (t @ wv.t())).sum())  # noqa: E731
    diff = (loss(x + v) - loss(x - v)) / 2
    # bound: the gradient's own, times |v|
    assert abs(float((gx * v).sum()) - diff) <= 12 * 2.0 ** -23 * float((gb.double().abs() @ wv.abs() * v.abs()).sum())


def test_empty():
    w = bt.bt_mx_quantize(torch.randn(8, 64).cuda(), E2M1)
    assert bt.bt_mx_linear(torch.empty(0, 64, device="cuda"), w).shape == (0, 8)
    none = bt.bt_mx_quantize(torch.empty(0, 64, device="cuda"), E2M1)
    assert bt.bt_mx_linear(torch.randn(3, 64).cuda(), none).shape == (3, 0)
    assert bt.bt_mx_dequantize(none).shape == (0, 64)
    assert bt.bt_mx_linear_backward(torch.empty(0, 8, dtype=BF16, device="cuda"), bt.bt_mx_transpose(w)).shape == (0, 64)
    assert int(bt.bt_mx_linear_backward(torch.empty(3, 0, dtype=BF16, device="cuda"), bt.bt_mx_transpose(w)).count_nonzero()) == 0


def test_streams_and_graphs():
    gen = torch.Generator().manual_seed(3)
    x1, x2 = (torch.randn(20, 512, generator=gen).to(BF16).cuda() for _ in range(2))
    w = bt.bt_mx_quantize(torch.randn(300, 512, generator=gen).cuda(), E2M1)
    want = [bt.bt_mx_linear(x, w) for x in (x1, x2)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = bt.bt_mx_linear(x1, w, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got, want[0])
    x = x1.clone()
    out = torch.empty(20, 300, dtype=BF16, device="cuda")
    ws = torch.empty(bt.bt_mx_linear_workspace(20, 300, 512, bt.BT_BF16, E2M1), dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        bt.bt_mx_linear(x, w, out=out, workspace=ws)
    for src, y in zip((x2, x1), reversed(want)):
        x.copy_(src)
        graph.replay()
        assert torch.equal(out, y)
