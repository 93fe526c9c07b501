"""GPU: the distillation's kernel for many rows with several rows to a CTA, and its waits."""
import math

import pytest
import torch

import xnor_popcount_gemm_gb300 as bt
from test_distill_numerics_gpu import DEV, HALF, INF, definition, inputs, near

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _device_clean():
    yield
    assert bt.bt_device_status() == 0


def _mixed(T, V, S, dtype, seed, dead=0.3):
    """Rows of every kind at random: padding (no slot, over NaN), masked parts, a NaN, nothing left, empty slots."""
    gen = torch.Generator().manual_seed(seed)
    z, ids, top, t, w = inputs(T, V, S, dtype, seed)
    kind = torch.randint(0, 8, (T,), generator=gen)
    cut = torch.randint(1, V + 1, (T,), generator=gen)
    for r in range(T):
        if kind[r] == 0:
            z[r, cut[r]:] = -INF
        elif kind[r] == 1:
            z[r, : cut[r] - 1] = -1e34 if dtype != torch.float16 else -INF
        elif kind[r] == 2:
            z[r] = -INF
        elif kind[r] == 3:
            ids[r, cut[r] % S:] = -1
        elif kind[r] == 4:
            top[r, : cut[r] % S] = -INF
    pad = torch.rand(T, generator=gen) < dead
    ids[pad] = -1
    z[pad, 0] = math.nan
    bad = (kind == 5) & ~pad & (torch.rand(T, generator=gen) < 0.2)
    bad[0] = bad[-1] = False
    return z, ids, top, t, w, bad, cut % V


@pytest.mark.parametrize("rest", [False, True])
@pytest.mark.parametrize("T,V,S,dtype,tau", [
    (1521, 3, 2, torch.float32, 1.0),                # no vectors or hardly any
    (1217, 29, 9, torch.bfloat16, 1.2),
    (913, 1003, 16, torch.float16, 2.5),             # fewer chunks than warps
    (1000, 2048, 5, torch.float32, 1.1),
    (925, 12289, 33, torch.bfloat16, 2.0),           # one chunk a warp and two
    (620, 30011, 40, torch.float16, 1.7),            # several
    (700, 4099, 1024, torch.bfloat16, 1.0),          # as many slots as there may be
    (5000, 515, 7, torch.bfloat16, 5.0),             # sixteen rows a CTA
])
def test_many_rows_of_every_kind_one_after_another(T, V, S, dtype, tau, rest):
    """Several rows to every CTA of the kernel for many rows, live and padding ones in any order: the copies run on into
    the next row, its slots and the one after's are fetched meanwhile. Rows pitched apart, the gradient in place and
    apart, over NaN: every row has to be written."""
    z, ids, top, t, w, bad, at = _mixed(T, V, S, dtype, seed=T)
    tlse = torch.logsumexp(t / tau, 1) if rest else None
    z[torch.arange(T)[bad], at[bad]] = math.nan
    sound = ~bad
    clean = z.clone()
    clean[bad] = 0.0
    loss, stats, grad, lb, es, eb = definition(torch.where(clean.isnan(), 0.0, clean), ids, top, tlse, tau, w)
    rel, sub = HALF[dtype]
    wd, idd, td = w.to(DEV), ids.int().to(DEV), top.to(DEV)
    tl = None if tlse is None else tlse.to(DEV)
    pitch = V + (5 if V % 2 else 8)
    room = torch.full((T, pitch), math.nan, dtype=dtype, device=DEV)
    zd = room[:, 1:1 + V] if V % 2 else room[:, :V]
    zd.copy_(z.to(DEV))
    l1, s1 = bt.bt_distill_topk(zd, idd, td, tl, tau)
    near(l1[sound.to(DEV)], loss[sound], lb[sound], "loss")
    fine = torch.where(stats.abs() < INF, stats.abs(), 0.0)
    near(s1[sound.to(DEV)], stats[sound], 2.0 ** -19 * (1 + fine)[sound], "stats")
    assert l1[bad.to(DEV)].isnan().all()
    out = torch.full((T, V), math.nan, dtype=dtype, device=DEV)
    l2, g2 = bt.bt_distill_topk_step(wd, zd, idd, td, tl, tau, grad=out, stats=(s2 := torch.full_like(s1, 7.0)))
    near(g2[sound.to(DEV)], grad[sound], (es + rel * grad.abs() + sub)[sound], "step")
    same = torch.equal(l1.nan_to_num(1.5), l2.nan_to_num(1.5)) and torch.equal(s1.nan_to_num(1.5), s2.nan_to_num(1.5))
    assert same and g2[bad.to(DEV)].isnan().any(dim=1).all()
    g1 = bt.bt_distill_topk_backward(wd, zd, idd, td, s1, tl, tau, grad=torch.full_like(out, math.nan))
    near(g1[sound.to(DEV)], grad[sound], (eb + rel * grad.abs() + sub)[sound], "backward")
    for _ in range(2):                               # the same again
        l3, g3 = bt.bt_distill_topk_step(wd, zd, idd, td, tl, tau, grad=torch.full_like(out, math.nan))
        assert torch.equal(l3.nan_to_num(1.5), l1.nan_to_num(1.5)) and torch.equal(g3.nan_to_num(1.5), g2.nan_to_num(1.5))
    bt.bt_distill_topk_step(wd, zd, idd, td, tl, tau, grad=zd)
    assert torch.equal(zd.nan_to_num(1.5), g2.nan_to_num(1.5))
    assert room[:, V + 1 if V % 2 else V:].isnan().all() and (V % 2 == 0 or room[:, 0].isnan().all())


def test_a_wait_that_runs_out_is_reported():
    """With a limit of 1 ns the first wait for a copy in flight gives up: TIMEOUT, once; the copies still land, and the
    next call is as always. (A copy may have landed by the first look: out of memory, not out of L2, and several calls.)"""
    flush = torch.empty(1 << 28, dtype=torch.uint8, device=DEV)
    z, ids, top, t, w = inputs(400, 32000, 8, torch.bfloat16, seed=8)
    args = (z.to(DEV), ids.to(DEV), top.to(DEV))
    want = bt.bt_distill_topk(*args)[0]
    assert bt.bt_device_status() == 0
    seen = []
    bt.bt_set_wait_timeout(1)
    try:
        while bt.BT_ERR_TIMEOUT not in seen and len(seen) < 200:
            flush.zero_()
            bt.bt_distill_topk(*args)
            seen.append(bt.bt_device_status())
    finally:
        bt.bt_set_wait_timeout(0)
    assert set(seen) <= {0, bt.BT_ERR_TIMEOUT} and seen[-1] == bt.BT_ERR_TIMEOUT
    assert bt.bt_device_status() == 0
    assert torch.equal(bt.bt_distill_topk(*args)[0], want)
