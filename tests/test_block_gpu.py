"""Norm, microscaled projection, adapters, distillation and clipping run together, as a training step and as decoding (GPU)."""
import pytest
import torch

import xnor_popcount_gemm_gb300 as bt

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


def _model(gen, K, N, R, L, code):
    w = torch.randn(N, K, generator=gen) * K ** -0.5
    return dict(norm=(1.0 + 0.2 * torch.randn(K, generator=gen)).to(BF16).cuda(), w=bt.bt_mx_quantize(w.cuda(), code),
                a=(torch.randn(L, R, K, generator=gen) * K ** -0.5).to(BF16).cuda(), b=(torch.randn(L, N, R, generator=gen) * 0.3).to(BF16).cuda(),
                scale=(torch.rand(L, generator=gen) + 0.5).cuda())


def _forward(m, x, r, plan, code, u=None):
    y, h, q = bt.bt_rms_norm(x, m["norm"], 1e-6, residual=r, code=code)
    base = bt.bt_mx_linear(q, m["w"])
    return y, h, q, bt.bt_adapter_linear(y, m["a"], m["b"], m["scale"], plan, base=base, u=u)


@pytest.mark.parametrize("code", [bt.BT_CODE_E4M3, bt.BT_CODE_E2M1])
@pytest.mark.parametrize("T,K,N", [(96, 512, 640), (50, 260, 1001)])
def test_a_training_step(T, K, N, code):
    gen = torch.Generator().manual_seed(T)
    R, L, S, tau = 8, 2, 16, 2.0
    m = _model(gen, K, N, R, L, code)
    x, r = (torch.randn(T, K, generator=gen).to(BF16).cuda() for _ in range(2))
    ids = torch.randint(0, L, (T,), generator=gen)
    plan = bt.bt_adapter_plan(ids, L)
    top, top_ids = (torch.randn(T, N, generator=gen) * 2).cuda().topk(S, dim=1)
    u = torch.empty(T, R, device="cuda")
    y, h, q, logits = _forward(m, x, r, plan, code, u)
    loss, g = bt.bt_distill_topk_step(torch.full((T,), 1.0 / T, device="cuda"), logits, top_ids.int(), top, temperature=tau)
    gy = bt.bt_mx_linear_backward(g, bt.bt_mx_transpose(m["w"]))
    gx, ga, gb = bt.bt_adapter_linear_backward(y, g, u, m["a"], m["b"], m["scale"], plan, grad_base=gy)
    gsum = (torch.randn(T, K, generator=gen) * 1e-3).to(BF16).cuda()
    gh, gw = bt.bt_rms_norm_backward(gx, h, m["norm"], 1e-6, grad_sum=gsum)
    grads = [ga, gb, gw]
    before = [t.clone() for t in grads]
    norm = bt.bt_clip_grads(grads, 1e-3)
    assert bt.bt_device_status() == 0

    # the same in 64 bits, each step from the values that the step before left, rounded where they are rounded
    half = torch.finfo(BF16).eps / 2
    h64 = (x.double() + r.double()).to(BF16).double()
    y64 = h64 / torch.sqrt(h64.square().mean(dim=1, keepdim=True) + 1e-6) * m["norm"].double()
    assert torch.equal(h.double(), h64) and bool(((y.double() - y64).abs() <= y64.abs() * half * 1.001 + 1e-30).all())
    wv, qv, s = bt.bt_mx_dequantize(m["w"]).double(), bt.bt_mx_dequantize(q).double(), m["scale"].double()[ids.cuda()].unsqueeze(1)
    assert torch.equal(bt.bt_mx_dequantize(q), bt.bt_mx_dequantize(bt.bt_mx_quantize(y, code)))
    A, B = m["a"].double()[ids.cuda()], m["b"].double()[ids.cuda()]
    base64 = qv @ wv.t()
    low = s * torch.einsum("tnr,tr->tn", B, torch.einsum("trk,tk->tr", A, y.double()))
    want = base64 + low
    # base and the result are rounded to bf16; fp32 sums beside that
    sums = 2.0 ** -17 * (qv.abs() @ wv.abs().t() + s * torch.einsum("tnr,tr->tn", B.abs(), torch.einsum("trk,tk->tr", A.abs(), y.double().abs())))
    assert bool(((logits.double() - want).abs() <= (base64.abs() + want.abs() * 1.01) * half + sums).all())
    g64 = g.double()
    gx64 = g64 @ wv + torch.einsum("trk,tr->tk", A, s * torch.einsum("tnr,tn->tr", B, g64))
    sums = 2.0 ** -17 * (g64.abs() @ wv.abs() + torch.einsum("trk,tr->tk", A.abs(), s * torch.einsum("tnr,tn->tr", B.abs(), g64.abs())))
    assert bool(((gx.double() - gx64).abs() <= ((g64 @ wv).abs() + gx64.abs() * 1.01) * half + sums).all())
    inv = 1.0 / torch.sqrt(h64.square().mean(dim=1, keepdim=True) + 1e-6)
    n, gn = h64 * inv, gx.double() * m["norm"].double()
    gh64 = inv * (gn - n * (gn * n).mean(dim=1, keepdim=True)) + gsum.double()
    assert bool(((gh.double() - gh64).abs() <= gh64.abs() * half * 1.01 + 2.0 ** -17 * inv * (gn.abs() + n.abs() * (gn * n).abs().mean(dim=1, keepdim=True))).all())
    norm64 = torch.sqrt(sum(t.double().square().sum() for t in before))
    assert abs(float(norm - norm64)) <= 1e-5 * float(norm64) and float(norm64) > 1e-3
    for t, b in zip(grads, before):
        f = 1e-3 / (float(norm64) + 1e-6)
        assert bool(((t.double() - b.double() * f).abs() <= b.double().abs() * f * 1e-5 + 1e-37).all())
    assert bool(torch.isfinite(loss).all())


@pytest.mark.parametrize("code", [bt.BT_CODE_E4M3, bt.BT_CODE_E2M1])
def test_a_token_alone_is_as_in_its_prompt(code):
    gen = torch.Generator().manual_seed(1)
    T, K, N, R, L = 200, 768, 520, 8, 3
    m = _model(gen, K, N, R, L, code)
    x, r = (torch.randn(T, K, generator=gen).to(BF16).cuda() for _ in range(2))
    ids = torch.randint(-1, L, (T,), generator=gen)
    y, h, q, out = _forward(m, x, r, bt.bt_adapter_plan(ids, L), code)
    for t in (0, 77, 199):
        y1, h1, q1, out1 = _forward(m, x[t:t + 1], r[t:t + 1], bt.bt_adapter_plan(ids[t:t + 1], L), code)
        assert torch.equal(h1, h[t:t + 1]) and torch.equal(y1, y[t:t + 1]) and torch.equal(q1.codes, q.codes[t:t + 1])
        # sums in another order, each result rounded twice (base, then the sum)
        assert bool(((out1.double() - out[t:t + 1].double()).abs() <= 4 * 2.0 ** -8 * out[t:t + 1].double().abs() + 0.01).all())


def test_two_streams_at_once():
    gen = torch.Generator().manual_seed(2)
    code = bt.BT_CODE_E2M1
    w = bt.bt_mx_quantize(torch.randn(1024, 2048, generator=gen).cuda(), code)
    xs = [torch.randn(M, 2048, generator=gen).to(BF16).cuda() for M in (8, 700)]
    gs = [torch.randn(200000, generator=gen).cuda() for _ in range(2)]

    def run(i, n):
        for _ in range(n):
            y, _, _ = bt.bt_rms_norm(xs[i], None)
            o = bt.bt_mx_linear(y, w)
            gx, gw = bt.bt_rms_norm_backward(y, xs[i])
            c = gs[i].clone()
            norm = bt.bt_clip_grads([c], 1.0)
        return o, gx, gw, c, norm

    want = [run(i, 1) for i in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = []
    for i, s in enumerate(streams):
        with torch.cuda.stream(s):
            got.append(run(i, 20))
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        assert all(torch.equal(p, q) for p, q in zip(a, b))
    assert bt.bt_device_status() == 0


@pytest.mark.parametrize("config", ["small,1", "small,4", "256,1", "128,2", "pair,256,1", "pair,128,2"])
def test_a_wait_that_runs_out_is_reported(config, monkeypatch):
    """With a limit of 1 ns the first wait for a copy or a product in flight gives up: TIMEOUT, once; what is in flight still
    ends, and the next call is right."""
    monkeypatch.setenv("BT_MX_CONFIG", config)
    M, N, K = (20 if config.startswith("small") else 700), 600, 4096
    gen = torch.Generator().manual_seed(4)
    x, w = bt.bt_mx_quantize(torch.randn(M, K, generator=gen).cuda(), bt.BT_CODE_E2M1), bt.bt_mx_quantize(torch.randn(N, K, generator=gen).cuda(), bt.BT_CODE_E2M1)
    want = bt.bt_mx_linear(x, w)
    assert bt.bt_device_status() == 0
    bt.bt_set_wait_timeout(1)
    try:
        bt.bt_mx_linear(x, w)
        status = bt.bt_device_status()
    finally:
        bt.bt_set_wait_timeout(0)
    assert status == bt.BT_ERR_TIMEOUT and bt.bt_device_status() == 0
    assert torch.equal(bt.bt_mx_linear(x, w), want) and bt.bt_device_status() == 0
