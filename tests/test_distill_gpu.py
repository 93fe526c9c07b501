"""GPU parity of the distillation from a teacher's top logits (bt_distill_topk,
bt_distill_topk_backward, bt_distill_topk_step) against the definition in 64
bits on the CPU.

Tolerances, u = 2^-24. The loss is a sum of terms q_k D_k, D_k = log q_k - log
p_k built from a handful of fp32 quantities (t / tau, the teacher's log sum,
(z - m) / tau, log sum), each within 8 u of its magnitude, the sums s within
32 u (at most 2^10 terms one after another, whose errors have either sign), and
q_k from an exponent with the same error: 2^-19 times the sum of q_k (1 + |D_k|)
(1 + the quantities' magnitudes); the rest's term likewise, q_r being within
2^-19 of 1 - sum q. stats: 2^-19 (1 + |value|). A gradient w / tau (p - q) has
p and q within 2^-18 (1 + magnitude of their exponent) of themselves, and one
rounding to its type: half a step, 2^-9, 2^-12 (2^-25 where subnormal) or
2^-24 of it, doubled for a rounding that falls the other way.
"""
import ctypes
import math

import pytest
import torch

import xnor_popcount_gemm_gb300 as bt

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
HALF = {torch.float32: (2.0 ** -23, 0.0), torch.bfloat16: (2.0 ** -8, 0.0), torch.float16: (2.0 ** -11, 2.0 ** -24)}


@pytest.fixture(autouse=True)
def _device_clean():
    yield
    assert bt.bt_device_status() == 0


def _reference(z, ids, top, tlse, tau, w=None):
    """(loss, stats, grad, loss bound, grad bound) in 64 bits, row by row."""
    z, top = z.double(), top.double()
    T, V = z.shape
    loss, stats = torch.zeros(T).double(), torch.zeros(T, 2).double()
    lb, gb = torch.zeros(T).double(), torch.zeros(T, V).double()
    grad = torch.zeros(T, V).double()
    for t in range(T):
        ok = (ids[t] >= 0) & (ids[t] < V) & (top[t] > -math.inf)
        if not ok.any():
            continue
        k = ids[t][ok].long()
        a, x = z[t] / tau, top[t][ok] / tau
        tl = torch.logsumexp(x, 0) if tlse is None else tlse[t].double()
        lq = x - tl
        q = lq.exp()
        inside = torch.zeros(V, dtype=torch.bool)
        inside[k] = True
        fill = z[t] <= -1.7e38                       # a mask's fill value: nothing left where there is no other
        lse = torch.logsumexp(a, 0) if not fill.all() else torch.tensor(-math.inf).double()
        r = torch.logsumexp(a.masked_fill(inside, -math.inf), 0) if not (fill | inside).all() else \
            torch.tensor(-math.inf).double()
        stats[t] = torch.stack([lse, r])
        if lse == -math.inf:
            continue
        lp = a - lse
        terms = torch.where(q > 0, q * (lq - lp[k]), 0.0)
        loss[t] = terms.sum()
        size = 1 + x.abs() + tl.abs() + torch.where(a[k] > -math.inf, (a[k] - a.max()).abs(), 0.0) + math.log(V + 1)
        lb[t] = 2.0 ** -19 * (q * (1 + torch.where(a[k] > -math.inf, (lq - lp[k]).abs(), 0.0)) * size).sum()
        g = lp.exp()
        e = g * (1 + torch.where(g > 0, lp.abs() + lse.abs() + (a.abs() if w is not None else 0), 0.0))
        if tlse is not None:
            qr = (1 - q.sum()).clamp(min=0)
            if qr > 0 and r > -math.inf:
                loss[t] += qr * (qr.log() - (r - lse))
                lb[t] += 2.0 ** -19 * (1 + (qr.log() - (r - lse)).abs()) * size.max()
            rel = (a - r).exp() if r > -math.inf else torch.zeros_like(a)
            g = torch.where(inside, g, ((r - lse).exp() - qr) * rel)
            e = torch.where(inside, e, ((r - lse).exp() + 1) * rel * (1 + lse.abs() + size.max() +
                                                                    torch.where(rel > 0, a.abs(), 0.0)))
        g[k] -= q
        e[k] += q * size
        if w is not None:
            grad[t] = w[t].double() / tau * g
            gb[t] = w[t].double().abs() / tau * 2.0 ** -18 * e
    return loss, stats, grad, lb, gb


def _inputs(T, V, S, dtype, seed=0, std=2.0):
    gen = torch.Generator().manual_seed(seed)
    z = (torch.randn(T, V, generator=gen) * std).to(dtype)
    t = z.float() + torch.randn(T, V, generator=gen)
    top, ids = t.topk(S, dim=1)
    w = torch.randn(T, generator=gen)
    return z, ids, top, t, w


def _near(got, want, bound, what):
    got, want = got.cpu().double(), want.double()
    same = (got == want) | (got.isnan() & want.isnan())
    bad = ~(same | ((got - want).abs() <= bound))
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} off, first {bad.nonzero()[0].tolist()}: " \
        f"{got[tuple(bad.nonzero()[0])]} for {want[tuple(bad.nonzero()[0])]}, bound {bound[tuple(bad.nonzero()[0])]}"


def _check(z, ids, top, tlse, tau, w, *, zd=None, grad_out=None):
    """All three calls on one input."""
    loss, stats, grad, lb, gb = _reference(z, ids, top, tlse, tau, w)
    rel, sub = HALF[z.dtype]
    gb = gb + rel * grad.abs() + sub
    zd = z.to(DEV) if zd is None else zd
    d = [ids.to(DEV), top.to(DEV)]
    tl = None if tlse is None else tlse.to(DEV)
    wd = w.to(DEV)
    l1, s1 = bt.bt_distill_topk(zd, *d, tl, tau)
    _near(l1, loss, lb, "loss")
    _near(s1, stats, 2.0 ** -19 * (1 + torch.where(stats.abs() < math.inf, stats.abs(), 0.0)), "stats")
    g1 = bt.bt_distill_topk_backward(wd, zd, *d, s1, tl, tau)
    assert g1.dtype == z.dtype
    _near(g1, grad, gb, "backward")
    s2 = torch.full_like(s1, 7.0)
    l2, g2 = bt.bt_distill_topk_step(wd, zd, *d, tl, tau, stats=s2, grad=grad_out)
    _near(g2, grad, gb, "step")
    assert torch.equal(l1, l2) and torch.equal(s1, s2)            # the same sums
    return l1, g1


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("T,V,S", [
    (1, 1, 1), (3, 2, 1), (2, 7, 7), (4, 8, 3), (5, 9, 9), (2, 33, 8), (7, 250, 5), (3, 1000, 33), (2, 4099, 64),
    (40, 2049, 16), (3, 32000, 32), (2, 50001, 100), (200, 515, 7),
])
@pytest.mark.parametrize("rest", [False, True])
def test_sizes(T, V, S, dtype, rest):
    z, ids, top, t, w = _inputs(T, V, S, dtype, seed=T + V)
    tau = 2.0 if rest else 1.0
    _check(z, ids, top, torch.logsumexp(t / tau, 1) if rest else None, tau, w)


@pytest.mark.parametrize("T,V,S,dtype", [(2, 131072, 64, torch.float32), (170, 70001, 3, torch.bfloat16),
                                         (1, 393216, 10, torch.float32), (1, 786432, 10, torch.float16),
                                         (2, 3000, 1024, torch.bfloat16)])
def test_large_rows(T, V, S, dtype):
    z, ids, top, t, w = _inputs(T, V, S, dtype, seed=3)
    _check(z, ids, top, torch.logsumexp(t / 1.5, 1), 1.5, w)


@pytest.mark.parametrize("tau", [0.25, 1.0, 7.0])
def test_temperatures_and_types_of_the_teacher(tau):
    z, ids, top, t, w = _inputs(6, 777, 20, torch.bfloat16, seed=5)
    lse = torch.logsumexp(t / tau, 1)
    for ids_t in (torch.int32, torch.int64):
        for top_t in (torch.float32, torch.bfloat16, torch.float16):
            _check(z, ids.to(ids_t), top.to(top_t), lse, tau, w)
            _check(z, ids.to(ids_t), top.to(top_t), None, tau, w)


@pytest.mark.parametrize("rest", [False, True])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_empty_slots_masked_logits_and_rows_that_keep_nothing(rest, dtype):
    T, V, S = 9, 1003, 12
    z, ids, top, t, w = _inputs(T, V, S, dtype, seed=6)
    tlse = torch.logsumexp(t, 1) if rest else None
    ids[0, 3:] = -1                                  # some slots empty
    ids[1] = -1                                      # a padding token
    ids[2, 5] = V                                    # outside the vocabulary: empty
    top[3, 4] = -math.inf                            # a teacher's masked entry: empty
    z[4, 500:] = -math.inf                           # masked part of the vocabulary, slots among it or not
    z[5] = -math.inf                                 # nothing left
    z[6] = torch.finfo(dtype).min                    # all at the type's lowest value: a uniform row
    z[7] = torch.finfo(dtype).min
    z[7, ids[7, 0]] = 1.0                            # one logit against masked ones
    z[8, :] = 3.0
    z[1, 0] = math.nan                               # a padding token's logits are not used
    loss, grad = _check(z, ids, top, tlse, 1.0, w)
    assert loss[1] == 0 and not grad[1].any() and loss[5] == 0 and not grad[5].any()


def test_a_student_without_mass_on_the_teachers_choice():
    z, ids, top, t, w = _inputs(2, 64, 4, torch.float32, seed=7)
    z[0, ids[0, 1]] = -math.inf
    loss, stats = bt.bt_distill_topk(z.to(DEV), ids.to(DEV), top.to(DEV))
    assert loss[0] == math.inf and math.isfinite(loss[1].item())
    _check(z, ids, top, None, 1.0, w)


def test_all_slots_leaves_no_rest():
    z, ids, top, t, w = _inputs(3, 16, 16, torch.float32, seed=8)
    _check(z, ids, top, torch.logsumexp(t, 1), 1.0, w)


def test_nan_and_infinity_stay_in_their_rows():
    z, ids, top, t, w = _inputs(4, 3000, 8, torch.bfloat16, seed=9)
    clean = bt.bt_distill_topk_step(w.to(DEV), z.to(DEV), ids.to(DEV), top.to(DEV))
    z[1, 2000] = math.nan
    z[2, 17] = math.inf
    loss, grad = bt.bt_distill_topk_step(w.to(DEV), z.to(DEV), ids.to(DEV), top.to(DEV))
    assert loss[1].isnan() and loss[2].isnan() and grad[1].isnan().any() and grad[2].isnan().any()
    for r in (0, 3):
        assert loss[r] == clean[0][r] and torch.equal(grad[r], clean[1][r])


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("skew", [1, 3])
def test_strided_rows_odd_starts_and_in_place(dtype, skew):
    T, V, S = 5, 1001, 9
    z, ids, top, t, w = _inputs(T, V, S, dtype, seed=10)
    big = torch.full((T, V + 13), 99.0, dtype=dtype, device=DEV)
    view = big[:, skew:skew + V]
    view.copy_(z.to(DEV))
    out = torch.full((T, V + 6), 55.0, dtype=dtype, device=DEV)
    tl = torch.logsumexp(t / 2.0, 1)
    _check(z, ids, top, tl, 2.0, w, zd=view, grad_out=out[:, 2:2 + V])
    assert (out[:, :2] == 55).all() and (out[:, 2 + V:] == 55).all()
    want = out[:, 2:2 + V].clone()
    # in place, on a copy for either call
    args = (ids.to(DEV), top.to(DEV))
    stats = bt.bt_distill_topk(view, *args, tl.to(DEV), 2.0)[1]
    again = big.clone()
    bt.bt_distill_topk_step(w.to(DEV), view, *args, tl.to(DEV), 2.0, grad=view)
    assert torch.equal(view, want)
    v2 = again[:, skew:skew + V]
    apart = bt.bt_distill_topk_backward(w.to(DEV), v2, *args, stats, tl.to(DEV), 2.0)
    bt.bt_distill_topk_backward(w.to(DEV), v2, *args, stats, tl.to(DEV), 2.0, grad=v2)
    assert torch.equal(apart, v2)
    for b in (big, again):
        assert (b[:, :skew] == 99).all() and (b[:, skew + V:] == 99).all()


@pytest.mark.parametrize("rest", [False, True])
def test_gradient_against_differences(rest):
    """Central differences of the fp32 loss: h^2 / 6 times the third derivative (at most 1 for tau = 1) and the
    loss's own bound over h."""
    V, S, h = 40, 6, 2.0 ** -5
    z, ids, top, t, w = _inputs(1, V, S, torch.float32, seed=11, std=1.0)
    tl = torch.logsumexp(t, 1).to(DEV) if rest else None
    args = (ids.expand(V, S).contiguous().to(DEV), top.expand(V, S).contiguous().to(DEV), tl.expand(V).contiguous() if rest else None)
    plus = bt.bt_distill_topk((z + h * torch.eye(V)).to(DEV), *args)[0]
    minus = bt.bt_distill_topk((z - h * torch.eye(V)).to(DEV), *args)[0]
    num = ((plus.double() - minus.double()) / (2 * h)).cpu()
    one = torch.ones(1, device=DEV)
    got = bt.bt_distill_topk_step(one, z.to(DEV), ids.to(DEV), top.to(DEV), tl)[1][0].cpu().double()
    lb = _reference(z, ids, top, None if tl is None else tl.cpu(), 1.0)[3]
    assert ((got - num).abs() <= h * h / 6 + lb.max() / h).all()


def test_equal_calls_are_equal_and_streams():
    z, ids, top, t, w = _inputs(64, 9001, 16, torch.bfloat16, seed=12)
    a = (w.to(DEV), z.to(DEV), ids.to(DEV), top.to(DEV))
    l1, g1 = bt.bt_distill_topk_step(*a)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for _ in range(3):
        l2, g2 = bt.bt_distill_topk_step(*a, stream=s)
        s.synchronize()
        assert torch.equal(l1, l2) and torch.equal(g1, g2)


def test_in_a_graph():
    z, ids, top, t, w = _inputs(8, 5000, 16, torch.bfloat16, seed=13)
    wd, zd, idd, td = w.to(DEV), z.to(DEV), ids.to(DEV), top.to(DEV)
    want = bt.bt_distill_topk_step(wd, zd, idd, td)
    loss, grad = torch.zeros_like(want[0]), torch.zeros_like(want[1])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        bt.bt_distill_topk_step(wd, zd, idd, td, loss=loss, grad=grad)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(loss, want[0]) and torch.equal(grad, want[1])


def test_offsets_beyond_32_bits():
    T, V, S = 66000, 32800, 4                        # 2.16e9 logits
    z = torch.zeros(T, V, dtype=torch.bfloat16, device=DEV)
    ids = torch.full((T, S), -1, dtype=torch.int32, device=DEV)
    top = torch.zeros(T, S, device=DEV)
    zs, i2, t2, t, w2 = _inputs(2, V, S, torch.bfloat16, seed=14)
    w = torch.ones(T, device=DEV)
    z[-2:], ids[-2:], top[-2:], w[-2:] = zs.to(DEV), i2.int().to(DEV), t2.to(DEV), w2.to(DEV)
    loss, stats, grad, lb, gb = _reference(zs, i2, t2, None, 1.0, w2)
    rel, sub = HALF[torch.bfloat16]
    l1, s1 = bt.bt_distill_topk(z, ids, top)
    _near(l1[-2:], loss, lb, "loss")
    assert not l1[:-2].any()
    g = bt.bt_distill_topk_backward(w, z, ids, top, s1)
    _near(g[-2:], grad, gb + rel * grad.abs() + sub, "backward")
    assert not g[-3].any()
    l2, g2 = bt.bt_distill_topk_step(w, z, ids, top, grad=z)
    assert torch.equal(l1, l2)
    _near(z[-2:], grad, gb + rel * grad.abs() + sub, "step")


def test_wait_limit_is_reported():
    """A wait that runs out is recorded and the call returns (the copies land within the drain)."""
    z, ids, top, t, w = _inputs(4, 32000, 8, torch.bfloat16, seed=15)
    bt.bt_set_wait_timeout(1)
    try:
        bt.bt_distill_topk(z.to(DEV), ids.to(DEV), top.to(DEV))
        assert bt.bt_device_status() in (0, bt.BT_ERR_TIMEOUT)
    finally:
        bt.bt_set_wait_timeout(0)
    _check(z, ids, top, None, 1.0, w)
