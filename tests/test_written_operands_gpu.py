"""Results that a call writes into a caller's tensors count as in-place changes for autograd (GPU): a graph that holds such a
tensor for its backward says so instead of computing from the new values."""
import math

import pytest
import torch

import xnor_popcount_gemm_gb300 as bt

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


def _rows(*shape, dtype=BF16):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(sum(shape))).to(dtype).cuda()


def _moved(call, written, kept=()):
    before = [t._version for t in (*written, *kept)]
    call()
    now = [t._version for t in (*written, *kept)]
    n = len(written)
    assert all(a > b for a, b in zip(now[:n], before[:n])), (before, now)
    assert now[n:] == before[n:]


def test_norm():
    x, r, s, o, w = _rows(4, 64), _rows(4, 64), _rows(4, 64), _rows(4, 64), _rows(64)
    _moved(lambda: bt.bt_rms_norm(x, w, residual=r, sum=s, out=o), (s, o), (x, r, w))
    _moved(lambda: bt.bt_rms_norm(x, w, residual=r, sum=r, out=x), (x, r), (w,))
    g, gx, gw = _rows(4, 64), _rows(4, 64), torch.empty(64, device="cuda")
    _moved(lambda: bt.bt_rms_norm_backward(g, x, w, grad_x=gx, grad_weight=gw), (gx, gw), (g, x, w))
    _moved(lambda: bt.bt_rms_norm_backward(g, x, w, grad_sum=r, grad_x=r), (r,), (g, x, w))


def test_clipping():
    ts, norm = [_rows(100), _rows(5, 7, dtype=torch.float32)], torch.empty((), device="cuda")
    _moved(lambda: bt.bt_clip_grads(ts, 0.5, norm=norm), (*ts, norm))
    _moved(lambda: bt.bt_clip_grads(iter(ts), 0.5), ts)
    # the norm alone writes no gradient
    _moved(lambda: bt.bt_clip_grads(ts, math.inf, norm=norm), (norm,), ts)


def test_microscaled():
    x, w = _rows(40, 64), bt.bt_mx_quantize(_rows(24, 64), bt.BT_CODE_E2M1)
    out, g, gx, values = _rows(40, 24), _rows(40, 24), _rows(40, 64), _rows(24, 64)
    _moved(lambda: bt.bt_mx_linear(x, w, out=out), (out,), (x,))
    _moved(lambda: bt.bt_mx_linear(x[:3], w, out=out[:3]), (out,), (x,))       # (views share the count)
    wt = bt.bt_mx_transpose(w)
    _moved(lambda: bt.bt_mx_transpose(w, out=wt), (wt,))
    _moved(lambda: bt.bt_mx_linear_backward(g, wt, grad_x=gx), (gx,), (g, wt))
    _moved(lambda: bt.bt_mx_dequantize(w, out=values), (values,))


def test_results_over_the_operands_of_adapters_and_distillation():
    T, K, N, R, L = 6, 64, 32, 8, 2
    x, a, b, base, scale = _rows(T, K), _rows(L, R, K), _rows(L, N, R), _rows(T, N), torch.ones(L, device="cuda")
    u = torch.empty(T, R, device="cuda")
    plan = bt.bt_adapter_plan(torch.randint(-1, L, (T,), generator=torch.Generator().manual_seed(0)), L)
    _moved(lambda: bt.bt_adapter_linear(x, a, b, scale, plan, base=base, out=base, u=u), (base, u), (x, a, b))
    g, gb, ga, gbb = _rows(T, N), _rows(T, K), torch.empty(L, R, K, device="cuda"), torch.empty(L, N, R, device="cuda")
    _moved(lambda: bt.bt_adapter_linear_backward(x, g, u, a, b, scale, plan, grad_base=gb, grad_x=gb, grad_a=ga, grad_b=gbb),
           (gb, ga, gbb), (x, g, u, a, b))
    V, S = 50, 4
    logits, gl = _rows(T, V), torch.ones(T, device="cuda")
    ids, top = torch.arange(S).repeat(T, 1).cuda(), _rows(T, S, dtype=torch.float32)
    loss, stats = bt.bt_distill_topk(logits, ids, top)
    _moved(lambda: bt.bt_distill_topk(logits, ids, top, loss=loss, stats=stats), (loss, stats), (logits, top))
    _moved(lambda: bt.bt_distill_topk_backward(gl, logits, ids, top, stats, grad=logits), (logits,), (stats, top))
    logits = _rows(T, V)
    _moved(lambda: bt.bt_distill_topk_step(gl, logits, ids, top, grad=logits), (logits,), (top,))


def test_a_graph_that_holds_a_gradient_refuses():
    p = torch.ones(8, device="cuda", requires_grad=True)
    held = torch.full((8,), 3.0, device="cuda")
    loss = (p * held).sum()
    bt.bt_clip_grads([held], 0.1)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()
