"""GPU: numbers of the distillation (bt_distill_topk, _backward, _step) where they can go wrong: temperatures whose
log2(e) / temperature rounds either way, masked parts of a row of any size, rows filled with finite values, teachers
and students with nothing left.

The definition in 64 bits takes every logit relative to its row's largest, which is exact. Tolerances, u = 2^-24. A
probability or a sum of them is built from exponents (z - m) / temperature, each within 4 u of its magnitude, by exp2
within 4 u and by sums within 32 u: 2^-18 (1 + |log p|) of itself. A term q (log q - log p) has q and both logarithms
within 2^-19 times the magnitudes that they are differences of. What is given or kept as one fp32 number, the teacher's
log sum and the statistics that the backward reads, adds u of its own magnitude to an exponent. Results in 16 bits are
rounded once, by half a step, doubled for a rounding that falls the other way.
"""
import math

import pytest
import torch

import xnor_popcount_gemm_gb300 as bt

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
HALF = {torch.float32: (2.0 ** -23, 0.0), torch.bfloat16: (2.0 ** -8, 0.0), torch.float16: (2.0 ** -11, 2.0 ** -24)}
MASKED = -1.0e30                                     # logits below count as masked
INF = math.inf


@pytest.fixture(autouse=True)
def _device_clean():
    yield
    assert bt.bt_device_status() == 0


def _log_sum(a, keep):
    """(largest of the kept, log of the sum of exp(a - largest) over them); -inf for none."""
    a = torch.where(keep, a, -INF)
    m = a.amax(dim=1)
    m0 = torch.where(m > -INF, m, 0.0)
    return m, (a - m0[:, None]).exp().sum(dim=1).log()


def definition(z, ids, top, tlse, tau, w):
    """loss, stats, grad and the bounds (loss, step's gradient, backward's gradient) in 64 bits, all rows at once."""
    z, top = z.double(), top.double()
    T, V = z.shape
    live = (ids >= 0) & (ids < V) & (top > -INF)
    at = torch.where(live, ids.long(), V)
    inside = torch.zeros(T, V + 1, dtype=torch.bool).scatter_(1, at, True)[:, :V]
    some = live.any(dim=1)
    keep = z >= MASKED
    m, s = _log_sum(z / tau, keep)
    mr, sr = _log_sum(z / tau, keep & ~inside)
    left, rest = some & (m > -INF), some & (mr > -INF)
    m0, mr0 = torch.where(left, m, 0.0), torch.where(rest, mr, 0.0)
    s0, sr0 = torch.where(left, s, 0.0), torch.where(rest, sr, 0.0)
    stats = torch.stack([torch.where(left, m0 + s0, -INF), torch.where(rest, mr0 + sr0, -INF)], 1)
    stats = torch.where(some[:, None], stats, 0.0)
    gather = torch.cat([z, torch.zeros(T, 1).double()], 1).gather(1, at)

    # the teacher
    t = torch.where(live, top / tau, -INF)
    mt = t.amax(dim=1)
    mt0 = torch.where(mt > -INF, mt, 0.0)
    if tlse is None:
        lt = (t - mt0[:, None]).exp().sum(dim=1).clamp(min=1e-300).log()
        lq, size_t = t - mt0[:, None] - lt[:, None], 1 + (t - mt0[:, None]).abs() + lt.abs()[:, None]
    else:
        lq, size_t = t - tlse.double()[:, None], 1 + t.abs() + tlse.double().abs()[:, None]
    q = torch.where(live, lq.exp(), 0.0)
    size_t = torch.where(live, size_t, 0.0)
    qr = (1 - q.sum(dim=1)).clamp(min=0) if tlse is not None else torch.zeros(T).double()

    # the student at the slots
    lp = torch.where(live & (gather > -INF), gather / tau - m0[:, None] - s0[:, None], -INF)
    term = torch.where(q > 0, q * (lq - lp), 0.0)
    mag = torch.where(lp > -INF, lp.abs() + s0.abs()[:, None], 0.0) + 1
    loss = term.sum(dim=1)
    far = torch.where(q > 0, lq - lp, 0.0).abs().nan_to_num(0.0, 0.0)
    lb = 2.0 ** -19 * (q * ((1 + far) * size_t + mag)).nan_to_num(0.0).sum(dim=1)
    lpr = (mr0 - m0) + (sr0 - s0)                    # log of what the student leaves
    if tlse is not None:
        take = rest & (qr > 0)
        d = torch.where(take, qr.clamp(min=1e-300).log() - lpr, 0.0)
        loss = loss + torch.where(take, qr * d, 0.0)
        lb = lb + torch.where(take, 2.0 ** -19 * ((1 + d.abs()) * (q * size_t).nan_to_num(0.0).sum(dim=1) +
                                                  qr * (1 + lpr.abs() + s0.abs())), 0.0)
    loss = torch.where(left, loss, 0.0)

    # the gradient
    a = z / tau
    lpv = torch.where(keep, a - m0[:, None] - s0[:, None], -INF)
    p = lpv.exp()
    own = 1 + torch.where(p > 0, lpv.abs(), 0.0) + s0.abs()[:, None]
    kept = own + torch.where(p > 0, a.abs(), 0.0) + (m0 + s0).abs()[:, None]
    g, es, eb = p.clone(), p * own, p * kept
    if tlse is not None:
        pr = lpr.exp() * rest
        rel = torch.where(keep & rest[:, None], a - mr0[:, None] - sr0[:, None], -INF)
        own = 1 + torch.where(rel > -INF, rel.abs(), 0.0) + lpr.abs()[:, None] + s0.abs()[:, None]
        kept = own + torch.where(rel > -INF, a.abs(), 0.0) + (m0 + s0).abs()[:, None]
        slots = (q * size_t).nan_to_num(0.0).sum(dim=1)
        g = torch.where(inside, g, (pr - qr)[:, None] * rel.exp())
        weigh = ((pr + qr)[:, None] + slots[:, None]) * rel.exp()
        es, eb = torch.where(inside, es, weigh * own), torch.where(inside, eb, weigh * kept)
    pad = torch.zeros(T, 1).double()
    take = lambda v, x: torch.cat([v, pad], 1).scatter_add(1, at, torch.where(live, x, 0.0))[:, :V]  # noqa: E731
    g, es, eb = take(g, -q), take(es, q * size_t), take(eb, q * size_t)
    c = torch.where(left, w.double() / tau, 0.0)[:, None]
    return loss, stats, (c * g).nan_to_num(0.0), lb, c.abs() * 2.0 ** -18 * es, c.abs() * 2.0 ** -18 * eb


def near(got, want, bound, what):
    got, want = got.cpu().double(), want.double()
    bad = ~((got == want) | ((got - want).abs() <= bound))
    if bad.any():
        i = tuple(bad.nonzero()[0].tolist())
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} off, first {i}: {got[i]} for {want[i]}, bound {bound[i]}")


def check(z, ids, top, tlse, tau, w, grad_out=None):
    """All three calls on one input."""
    loss, stats, grad, lb, es, eb = definition(z, ids, top, tlse, tau, w)
    rel, sub = HALF[z.dtype]
    zd, idd, td, wd = (v.to(DEV) for v in (z, ids, top, w))
    tl = None if tlse is None else tlse.to(DEV)
    l1, s1 = bt.bt_distill_topk(zd, idd, td, tl, tau)
    near(l1, loss, lb, "loss")
    near(s1, stats, 2.0 ** -19 * (1 + torch.where(stats.abs() < INF, stats.abs(), 0.0)), "stats")
    nan = torch.full_like(zd, math.nan)
    g1 = bt.bt_distill_topk_backward(wd, zd, idd, td, s1, tl, tau, grad=nan)
    near(g1, grad, eb + rel * grad.abs() + sub, "backward")
    nan = torch.full_like(zd, math.nan) if grad_out is None else grad_out
    l2, g2 = bt.bt_distill_topk_step(wd, zd, idd, td, tl, tau, grad=nan, stats=(s2 := torch.full_like(s1, 7.0)))
    near(g2, grad, es + rel * grad.abs() + sub, "step")
    assert torch.equal(l1, l2) and torch.equal(s1, s2)
    return l1, g2


def inputs(T, V, S, dtype, seed, std=2.0):
    gen = torch.Generator().manual_seed(seed)
    z = (torch.randn(T, V, generator=gen) * std).to(dtype)
    t = z.float() + torch.randn(T, V, generator=gen)
    top, ids = t.topk(S, dim=1)
    return z, ids, top, t, torch.randn(T, generator=gen)


# log2(e) / tau is rounded up for some of these and down for others
TAUS = [0.6, 0.9, 1.1, 1.2, 1.7, 2.5, 5.0, 10.0, 20.0, 1.0, 4.0]


@pytest.mark.parametrize("tau", TAUS)
@pytest.mark.parametrize("rest", [False, True])
@pytest.mark.parametrize("T,V,S,dtype", [
    (5, 9, 4, torch.float32), (7, 250, 5, torch.bfloat16), (3, 1000, 33, torch.float16), (40, 2049, 16, torch.bfloat16),
    (2, 32000, 32, torch.float32),                   # up to half a machine of rows: a cluster each
    (200, 515, 7, torch.float16), (180, 4096, 16, torch.bfloat16), (160, 5003, 20, torch.float32),
])
def test_temperatures(T, V, S, dtype, rest, tau):
    z, ids, top, t, w = inputs(T, V, S, dtype, seed=V)
    check(z, ids, top, torch.logsumexp(t / tau, 1) if rest else None, tau, w)


@pytest.mark.parametrize("tau", [1.0, 1.2, 2.5])
@pytest.mark.parametrize("rest", [False, True])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,V", [(3, 32000), (170, 9001)])
def test_masked_parts(T, V, dtype, rest, tau):
    """Masked columns from a fortieth of the row to all but a few of it, by -inf and by finite values."""
    S = 12
    z, ids, top, t, w = inputs(T, V, S, dtype, seed=2)
    fills = [-INF, -1e10, -1e15, -1e20, torch.finfo(dtype).min]
    keeps = [V - V // 40, V // 3, 40]
    for r in range(T):
        z[r, keeps[r % 3]:] = fills[(r // 3) % 5]
        # the teacher's choice lies in what is kept
        ids[r] = torch.arange(S) * 3 + r % 2
    check(z, ids, top, torch.logsumexp(t / tau, 1) if rest else None, tau, w)


@pytest.mark.parametrize("tau", [1.0, 1.2, 2.5])
@pytest.mark.parametrize("rest", [False, True])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,V", [(25, 3001), (175, 3001), (175, 61)])
def test_rows_of_one_value(T, V, dtype, rest, tau):
    """Rows whose logits all have one value: nothing left where it is masked, all alike where it is not."""
    z, ids, top, t, w = inputs(T, V, 9, dtype, seed=3)
    for r, v in enumerate([-INF, torch.finfo(dtype).min, 3.0, 0.0] * 3):
        z[r] = v
    check(z, ids, top, torch.logsumexp(t / tau, 1) if rest else None, tau, w)


@pytest.mark.parametrize("tau", [0.6, 1.0, 1.2, 2.5])
@pytest.mark.parametrize("T,V", [(6, 3001), (170, 3001)])
def test_nothing_outside_the_slots(T, V, tau):
    """The student has logits in the slots alone: the rest's term is left out, what lies outside gets no gradient."""
    for dtype, fill in ((torch.float32, -INF), (torch.bfloat16, torch.finfo(torch.bfloat16).min), (torch.float16, -INF)):
        z, ids, top, t, w = inputs(T, V, 8, dtype, seed=4)
        only = torch.full_like(z, fill).scatter_(1, ids, z.gather(1, ids))
        only[0] = z[0]
        for tlse in (None, torch.logsumexp(t / tau, 1)):
            grad = check(only, ids, top, tlse, tau, w)[1]
            outside = torch.ones(T, V, dtype=torch.bool).scatter_(1, ids, False)
            assert not grad.cpu()[1:][outside[1:]].any()


@pytest.mark.parametrize("tau", [1.0, 1.2, 2.5])
@pytest.mark.parametrize("rest", [False, True])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,V", [(25, 3001), (175, 3001), (175, 61)])
def test_gradients_of_rows_of_one_huge_value(T, V, dtype, rest, tau):
    """The same of values whose log sum fp32 cannot tell from their largest: the step's gradient, which comes from the
    sums, is the definition's, the backward's, from the statistics, is that of probabilities of at most one."""
    z, ids, top, t, w = inputs(T, V, 9, dtype, seed=3)
    for r, v in enumerate([-1e10, -1e15, -1e20, 1e10] * 3):
        z[r] = v
    z[3, 5] = -1e15                                  # and of one value beside another
    z[9, : V // 2] = -3e15
    z[11, V // 2:] = 2e10
    tlse = torch.logsumexp(t / tau, 1) if rest else None
    grad, es = (definition(z, ids, top, tlse, tau, w)[i] for i in (2, 4))
    rel, sub = HALF[dtype]
    args = [w.to(DEV), z.to(DEV), ids.to(DEV), top.to(DEV)]
    tl = None if tlse is None else tlse.to(DEV)
    stats = torch.empty(T, 2, device=DEV)
    near(bt.bt_distill_topk_step(*args, tl, tau, stats=stats)[1], grad, es + rel * grad.abs() + sub, "step")
    got = bt.bt_distill_topk_backward(*args, stats, tl, tau).cpu().double()
    assert (got[:12].abs() <= (1 + rel) * w[:12, None].double().abs() / tau).all()


@pytest.mark.parametrize("tau", [1.0, 1.2, 2.5])
@pytest.mark.parametrize("rest", [False, True])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,V", [(25, 3001), (175, 3001), (175, 61)])
def test_rows_of_one_huge_value(T, V, dtype, rest, tau):
    """The same of values whose logarithms do not show next to them: the loss comes from the sums."""
    z, ids, top, t, w = inputs(T, V, 9, dtype, seed=3)
    for r, v in enumerate([-1e10, -1e15, -1e20, 1e10] * 3):
        z[r] = v
    # and those with one value beside another
    z[3, 5] = -1e15
    z[9, : V // 2] = -3e15
    z[11, V // 2:] = 2e10
    check(z, ids, top, torch.logsumexp(t / tau, 1) if rest else None, tau, w)


@pytest.mark.parametrize("rest", [False, True])
@pytest.mark.parametrize("T,tau", [(20, 1.0), (20, 4.0), (180, 2.5)])
def test_a_common_offset_does_not_show(T, tau, rest):
    """What all logits of a row share changes its statistics, and its loss no more than by a rounding."""
    z, ids, top, t, w = inputs(T, 4000, 24, torch.float32, seed=6)
    z = (z * 1024).round() / 1024                    # the offsets below are exact
    tlse = torch.logsumexp(t / tau, 1) if rest else None
    for offset in (0.0, 24.0, 4096.0, -8192.0):
        check(z + offset, ids, top, tlse, tau, w)


@pytest.mark.parametrize("rest", [False, True])
@pytest.mark.parametrize("top_dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("T", [12, 180])
def test_teachers_at_their_types_lowest_value(T, top_dtype, rest):
    """A slot is empty where its logit is -inf alone: lowest values among others have a probability of 0, lowest values
    alone are all alike."""
    V, S, tau = 2500, 40, 1.2
    z, ids, top, t, w = inputs(T, V, S, torch.bfloat16, seed=7)
    low = torch.finfo(top_dtype).min
    tlse = torch.logsumexp(t / tau, 1) if rest else None
    top = top.to(top_dtype)
    top[0, 5:] = low
    top[1, :-1] = low
    top[2, ::2], top[2, 1::2] = -INF, low
    if not rest:                                     # (a log sum of such a row is not an fp32 number)
        top[3], top[T - 1] = low, low
        top[4], ids[4, 7:] = low, -1
        top[5, :3], top[5, 3:] = low, -INF
    loss, grad = check(z, ids, top, tlse, tau, w)
    assert loss.isfinite().all() and grad.isfinite().all()


def _derivative(z, ids, top, tlse, tau, w):
    """The loss's derivative by autograd, in 64 bits."""
    z = z.double().requires_grad_()
    lp = torch.log_softmax(z / tau, 1)
    q = (top.double() / tau - tlse.double()[:, None]).exp()
    qr = (1 - q.sum(1)).clamp(min=0)
    inside = torch.zeros(z.shape, dtype=torch.bool).scatter_(1, ids, True)
    lpr = torch.logsumexp(lp.masked_fill(inside, -INF), 1)
    loss = (q * (q.log() - lp.gather(1, ids))).sum(1) + torch.where(qr > 0, qr * (qr.clamp(min=1e-300).log() - lpr), 0.0)
    (loss * w.double()).sum().backward()
    return z.grad, q.sum(1)


@pytest.mark.parametrize("top_dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("T", [30, 170])
def test_a_teacher_in_few_bits(T, top_dtype):
    """16-bit logits under a log sum of all of their bits: the gradient is p - q whatever the q sum to, as stated, and the
    loss's derivative where they sum to one or less, which a raised log sum sees to."""
    tau = 0.25
    z, ids, top, t, w = inputs(T, 777, 20, torch.float32, seed=9)
    top, tlse = top.to(top_dtype), torch.logsumexp(t / tau, 1)
    check(z, ids, top, tlse, tau, w)
    want, total = _derivative(z, ids, top, tlse, tau, w)
    assert (total > 1.003).any() == (top_dtype != torch.float32)
    es = definition(z, ids, top, tlse, tau, w)[4]
    args = [v.to(DEV) for v in (w, z, ids, top)]
    got = bt.bt_distill_topk_step(*args, tlse.to(DEV), tau)[1].cpu()
    below = total <= 1
    near(got[below], want[below], es[below] + 2.0 ** -23 * want[below].abs(), "gradient")
    raised = torch.maximum(tlse, torch.logsumexp(top.float() / tau, 1))
    want, total = _derivative(z, ids, top, raised, tau, w)
    es = definition(z, ids, top, raised, tau, w)[4]
    got = bt.bt_distill_topk_step(*args, raised.to(DEV), tau)[1].cpu()
    near(got, want, es + 2.0 ** -22 * want.abs(), "gradient under a raised log sum")
