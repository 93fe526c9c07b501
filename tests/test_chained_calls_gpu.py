"""Calls that read what the call before them wrote, into the same buffers again and again with other values (GPU): a kernel may
start while the one before it still runs, and reads only what that one has finished."""
import pytest
import torch

import xnor_popcount_gemm_gb300 as bt

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


def _sources(T, N, n=4):
    gen = torch.Generator(device="cuda").manual_seed(T + N)
    return [(torch.randn(T, N, generator=gen, device="cuda") * 4.0 ** i).to(BF16) for i in range(n)]


# from one row to more than an SM holds at a time, aligned and not
@pytest.mark.parametrize("T,N", [(1, 256), (16, 4096), (40, 1001), (300, 768), (3000, 512), (2500, 128)])
@pytest.mark.parametrize("code", [bt.BT_CODE_E4M3, bt.BT_CODE_E2M1])
def test_norm_then_quantisation_then_back(T, N, code):
    xs = _sources(T, N)
    r = torch.ones(T, N, dtype=BF16, device="cuda")
    want = []
    for x in xs:
        y, h, _ = bt.bt_rms_norm(x, None, 1.0, residual=r)
        torch.cuda.synchronize()
        q = bt.bt_mx_quantize(h, code)
        torch.cuda.synchronize()
        v = bt.bt_mx_dequantize(q, BF16)
        torch.cuda.synchronize()
        want.append((y, h, v, bt.bt_rms_norm(v, None, 1.0)[0]))
        torch.cuda.synchronize()
    y, h, v, z = (torch.empty(T, N, dtype=BF16, device="cuda") for _ in range(4))
    q = bt.bt_mx_quantize(xs[0], code)
    kept = [tuple(torch.empty_like(y) for _ in range(4)) for _ in range(24)]
    torch.cuda.synchronize()
    for i, to in enumerate(kept):
        bt.bt_rms_norm(xs[i % 4], None, 1.0, residual=r, sum=h, out=y)
        bt.bt_mx_quantize(h, code, out=q)
        bt.bt_mx_dequantize(q, out=v)
        bt.bt_rms_norm(v, None, 1.0, out=z)
        for a, b in zip(to, (y, h, v, z)):
            a.copy_(b)
    for i, to in enumerate(kept):
        assert all(torch.equal(a, b) for a, b in zip(to, want[i % 4]))


# the rows' sums of wide rows and the parts of the weight's gradient go from kernel to kernel through the workspace
@pytest.mark.parametrize("T,N", [(1, 17000), (40, 20000), (300, 17001), (16, 4096), (2500, 128)])
def test_backward_through_one_workspace(T, N):
    hs = _sources(T, N)
    g = torch.ones(T, N, dtype=BF16, device="cuda")
    want = []
    for h in hs:
        want.append(bt.bt_rms_norm_backward(g, h))
        torch.cuda.synchronize()
    ws = torch.empty(bt.bt_rms_norm_backward_workspace(T, N), dtype=torch.uint8, device="cuda")
    got = [(torch.empty_like(g), torch.empty(N, device="cuda")) for _ in range(24)]
    torch.cuda.synchronize()
    for i, (gx, gw) in enumerate(got):
        bt.bt_rms_norm_backward(g, hs[i % 4], grad_x=gx, grad_weight=gw, workspace=ws)
    for i, (gx, gw) in enumerate(got):
        assert torch.equal(gx, want[i % 4][0]) and torch.equal(gw, want[i % 4][1])


# gradients that were just computed, clipped; few and many rows of a product whose operands were just written
@pytest.mark.parametrize("M", [1, 16, 24, 200])
def test_product_then_clipping(M):
    gen = torch.Generator(device="cuda").manual_seed(M)
    w = [bt.bt_mx_quantize(torch.randn(512, 768, generator=gen, device="cuda"), bt.BT_CODE_E2M1) for _ in range(2)]
    xs = _sources(M, 768)
    want = []
    for i in range(4):
        o = bt.bt_mx_linear(bt.bt_mx_quantize(xs[i], bt.BT_CODE_E2M1), w[i % 2], out_dtype=torch.float32)
        torch.cuda.synchronize()
        n = bt.bt_clip_grads([o], 1.0)
        torch.cuda.synchronize()
        want.append((o, n))
    q, o, n = bt.bt_mx_quantize(xs[0], bt.BT_CODE_E2M1), torch.empty(M, 512, device="cuda"), torch.empty((), device="cuda")
    got = [(torch.empty_like(o), torch.empty_like(n)) for _ in range(24)]
    torch.cuda.synchronize()
    for i, (a, b) in enumerate(got):
        bt.bt_mx_quantize(xs[i % 4], bt.BT_CODE_E2M1, out=q)
        bt.bt_mx_linear(q, w[i % 2], out=o, out_dtype=torch.float32)
        bt.bt_clip_grads([o], 1.0, norm=n)
        a.copy_(o)
        b.copy_(n)
    for i, (a, b) in enumerate(got):
        assert torch.equal(a, want[i % 4][0]) and torch.equal(b, want[i % 4][1])


# adapters beside a projection take what the norm has just written; the distillation's gradient takes its loss's statistics
@pytest.mark.parametrize("T", [1, 8, 100, 1500])
def test_norm_then_adapters(T):
    K, N, R, L = 512, 384, 16, 3
    gen = torch.Generator(device="cuda").manual_seed(T)
    a, b = (torch.randn(*s, generator=gen, device="cuda").to(BF16) for s in ((L, R, K), (L, N, R)))
    scale = torch.ones(L, device="cuda")
    plan = bt.bt_adapter_plan(torch.randint(-1, L, (T,), generator=torch.Generator().manual_seed(T)), L)
    xs = _sources(T, K)
    want = []
    for x in xs:
        y = bt.bt_rms_norm(x, None, 1.0)[0]
        torch.cuda.synchronize()
        u = torch.empty(T, R, device="cuda")
        o = bt.bt_adapter_linear(y, a, b, scale, plan, u=u)
        torch.cuda.synchronize()
        want.append((o, bt.bt_adapter_linear_backward(y, o, u, a, b, scale, plan)[0]))
        torch.cuda.synchronize()
    y, u, o, gx = torch.empty(T, K, dtype=BF16, device="cuda"), torch.empty(T, R, device="cuda"), torch.empty(T, N, dtype=BF16, device="cuda"), torch.empty(T, K, dtype=BF16, device="cuda")
    got = [(torch.empty_like(o), torch.empty_like(gx)) for _ in range(24)]
    torch.cuda.synchronize()
    for i, (p, q) in enumerate(got):
        bt.bt_rms_norm(xs[i % 4], None, 1.0, out=y)
        bt.bt_adapter_linear(y, a, b, scale, plan, out=o, u=u)
        bt.bt_adapter_linear_backward(y, o, u, a, b, scale, plan, grad_x=gx)
        p.copy_(o)
        q.copy_(gx)
    for i, (p, q) in enumerate(got):
        assert torch.equal(p, want[i % 4][0]) and torch.equal(q, want[i % 4][1])


@pytest.mark.parametrize("T,V", [(1, 5000), (16, 32000), (700, 2000)])
def test_distillation_and_its_gradient(T, V):
    S = 8
    zs = _sources(T, V)
    ids = torch.arange(S, device="cuda").repeat(T, 1)
    top, gl = torch.randn(T, S, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda"), torch.ones(T, device="cuda")
    want = []
    for z in zs:
        _, stats = bt.bt_distill_topk(z, ids, top)
        torch.cuda.synchronize()
        want.append(bt.bt_distill_topk_backward(gl, z, ids, top, stats))
        torch.cuda.synchronize()
    stats, loss, got = torch.empty(T, 2, device="cuda"), torch.empty(T, device="cuda"), [torch.empty_like(zs[0]) for _ in range(24)]
    torch.cuda.synchronize()
    for i, g in enumerate(got):
        bt.bt_distill_topk(zs[i % 4], ids, top, loss=loss, stats=stats)
        bt.bt_distill_topk_backward(gl, zs[i % 4], ids, top, stats, grad=g)
    assert all(torch.equal(g, want[i % 4]) for i, g in enumerate(got))
