"""Clipping by the global norm against 64 bits (GPU)."""
import math

import pytest
import torch

import xnor_popcount_gemm_gb300 as bt

pytestmark = pytest.mark.gpu
F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16


def norm64(ts):
    return math.sqrt(sum(float(t.double().square().sum()) for t in ts))


def check(ts, max_norm, eps=1e-6):
    want, before = norm64(ts), [t.clone() for t in ts]
    norm = bt.bt_clip_grads(ts, max_norm, eps)
    # at most 64 fp32 additions of squares before the sums go on in 64 bits
    assert abs(float(norm) - want) <= want * 40 * 2.0 ** -24 + 1e-44
    f = min(1.0, max_norm / (want + eps)) if max_norm < math.inf else 1.0
    for t, b in zip(ts, before):
        y = b.double() * f
        # the factor's error and its rounding to fp32; one rounding of the product
        bound = y.abs() * (42 * 2.0 ** -24 + torch.finfo(t.dtype).eps / 2) + torch.finfo(t.dtype).tiny * torch.finfo(t.dtype).eps
        assert bool(((t.double() - y).abs() <= bound).all()) if f < 1.0 else torch.equal(t, b)
    return norm


def tensors(seed, sizes, dtype, std=1e-3):
    gen = torch.Generator().manual_seed(seed)
    return [(torch.randn(n, generator=gen) * std).to(dtype).cuda() for n in sizes]


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("sizes", [[1], [3, 0, 5], [4096], [8192, 8193, 1], [100000, 7, 65536], [17] * 70, [1000] * 300])
@pytest.mark.parametrize("clip", [True, False])
def test_clip(dtype, sizes, clip):
    ts = tensors(len(sizes), sizes, dtype)
    check(ts, 0.3 * norm64(ts) if clip else 2.0 * norm64(ts) + 1.0)


def test_mixed_types_shapes_and_offsets():
    flat = torch.randn(100000).cuda()
    half = torch.randn(50000).to(BF16).cuda()
    ts = [flat[1:8], flat[8:4105].view(17, 241), flat[5000:70001], half[1:4], half[5:20006], half[30000:30000],
          torch.randn(3, 5, 7).to(F16).cuda()]
    rest = torch.cat([flat[:1], flat[4105:5000], flat[70001:]]), torch.cat([half[:1], half[4:5], half[20006:]])
    kept = [t.clone() for t in rest]
    check(ts, 1.0)
    now = torch.cat([flat[:1], flat[4105:5000], flat[70001:]]), torch.cat([half[:1], half[4:5], half[20006:]])
    assert all(torch.equal(a, b) for a, b in zip(kept, now))


def test_more_tensors_than_a_launch_takes():
    flat = torch.randn(4000 * 33).cuda()
    check(list(flat.split(33)), 1.0)


@pytest.mark.parametrize("std", [1e-30, 1e-25, 1e-13, 1e15, 1e18])
def test_any_size_of_values(std):
    ts = [(torch.randn(5000, dtype=torch.float64) * std).float().cuda(), torch.zeros(3000, device="cuda")]
    check(ts, 0.5 * norm64(ts), eps=0.0)


def test_zeros_infinities_and_nan():
    z = [torch.zeros(1000, device="cuda"), torch.zeros(7, device="cuda")]
    assert float(bt.bt_clip_grads(z, 1.0)) == 0.0 and int(z[0].count_nonzero()) == 0
    t = [torch.ones(1000, device="cuda"), torch.ones(5, device="cuda").to(BF16)]
    t[0][3] = math.inf
    assert float(bt.bt_clip_grads(t, 1.0)) == math.inf
    assert bool(torch.isnan(t[0][3])) and int(torch.nan_to_num(t[0]).count_nonzero()) == 0 and int(t[1].count_nonzero()) == 0
    t = [torch.ones(1000, device="cuda"), torch.ones(5, device="cuda").to(BF16)]
    t[1][3] = math.nan
    assert math.isnan(float(bt.bt_clip_grads(t, 1.0))) and bool(torch.isnan(t[0]).all())


def test_the_norm_alone():
    t = tensors(1, [70000, 33], F32)
    t[0][5] = math.inf
    kept = t[0].clone()
    assert float(bt.bt_clip_grads(t, math.inf)) == math.inf and torch.equal(t[0], kept)
    t[0][5] = 0.0
    check(t, math.inf)
    assert float(check(t, 0.0)) > 0 and int(t[0].count_nonzero()) == 0


def test_equal_calls_give_equal_results_in_a_graph_too():
    sizes = [60000, 12345, 99]
    src = tensors(4, sizes, F32)
    ts, norm = [t.clone() for t in src], torch.zeros((), device="cuda")
    bt.bt_clip_grads(ts, 0.01, norm=norm)
    want, wanted = [t.clone() for t in ts], norm.clone()
    ws = torch.empty(bt.bt_clip_grads_workspace(3), dtype=torch.uint8, device="cuda")
    for t, s in zip(ts, src):
        t.copy_(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        bt.bt_clip_grads(ts, 0.01, norm=norm, workspace=ws)
    for _ in range(2):
        for t, s in zip(ts, src):
            t.copy_(s)
        graph.replay()
        assert torch.equal(norm, wanted) and all(torch.equal(a, b) for a, b in zip(ts, want))
