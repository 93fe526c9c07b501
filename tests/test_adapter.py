"""CPU checks of the adapters' entry points: the plan (host code) and the
refusals before anything is launched (no pointer below is dereferenced on a
device)."""
import ctypes
import random

import pytest
import torch

import xnor_popcount_gemm_gb300 as bt

TILE, SMALL, PARTS = 128, 16, 8


def _plan(ids, L):
    p = bt.bt_adapter_plan(ids, L, device="cpu")
    T, w = len(ids), p.buffer.tolist()
    tiles0 = (T + 3) // 4 * 4
    small0 = tiles0 + 4 * min(T, T // TILE + L + 1)
    parts0 = small0 + 4 * min(T, T // SMALL + L + 1)

    def table(at, n):
        return [tuple(w[at + 4 * i:at + 4 * i + 4]) for i in range(n)]

    return p.info, w[:T], table(tiles0, p.info.tiles), table(small0, p.info.small_tiles), table(parts0, p.info.parts)


def _ids(T, L, seed, none=0.2, skew=1.0):
    r = random.Random(seed)
    return [-1 if r.random() < none else int(L * r.random() ** skew) for _ in range(T)]


@pytest.mark.parametrize("T,L,none,skew", [(0, 1, 0, 1), (1, 1, 0, 1), (1, 3, 1, 1), (5, 2, 0.5, 1), (33, 1, 0, 1),
                                           (64, 48, 0.1, 1), (129, 2, 0, 1), (1000, 7, 0.3, 2), (3000, 100, 0.1, 4),
                                           (5000, 1, 0, 1), (4096, 3, 0, 3)])
def test_plan_covers_every_token_once(T, L, none, skew):
    ids = _ids(T, L, T + L, none, skew)
    info, rows, tiles, small, parts = _plan(ids, L)
    count = [ids.count(a) for a in range(L)]
    assert sorted(rows) == list(range(T))
    assert info.tokens == T and info.adapters == L and info.without == ids.count(-1)
    assert info.used == sum(n > 0 for n in count) and info.most_tokens == max(count)
    assert all(ids[t] == -1 for t in rows[T - info.without:])

    def covered(table, most, adapters):
        seen = []
        for a, first, n, _ in table:
            assert 1 <= n <= most and all(ids[t] == a for t in rows[first:first + n])
            seen += rows[first:first + n]
        assert sorted(seen) == [t for t in range(T) if ids[t] in adapters]

    covered(tiles, TILE, [a for a in range(L) if count[a]])
    covered(small, SMALL, [a for a in range(L) if count[a]])
    assert info.small_most == max([n for _, _, n, _ in small], default=0)
    # every adapter has its parts, one after the other; those of split ones come first and have the slots in order
    length = max(256, (-(-T // (PARTS if info.used <= 2 else PARTS // 2)) + 63) // 64 * 64)
    assert sorted({a for a, *_ in parts}) == list(range(L))
    slots = [p[3] for p in parts]
    assert slots == list(range(info.slots)) + [-1] * (len(parts) - info.slots) and info.slots <= 2 * PARTS
    for a in range(L):
        mine = [p for p in parts if p[0] == a]
        at = parts.index(mine[0])
        assert parts[at:at + len(mine)] == mine
        assert len(mine) == max(1, -(-count[a] // length)) and all(p[2] <= length for p in mine)
        assert (mine[0][3] >= 0) == (len(mine) > 1)
        got = [t for _, first, n, _ in mine for t in rows[first:first + n]]
        assert got == [t for t in range(T) if ids[t] == a]


def test_plan_takes_tensors_and_refuses():
    want = bt.bt_adapter_plan([1, -1, 0], 2, device="cpu").buffer
    for dt in (torch.int32, torch.int64, torch.int16):
        assert torch.equal(bt.bt_adapter_plan(torch.tensor([1, -1, 0], dtype=dt), 2, device="cpu").buffer, want)
    for ids in ([2], [-2], [0, 1, 5]):
        with pytest.raises(bt.BtError):
            bt.bt_adapter_plan(ids, 2, device="cpu")
    with pytest.raises(bt.BtError):
        bt.bt_adapter_plan(torch.tensor([1 << 32]), 2, device="cpu")       # not cut to 32 bits
    with pytest.raises(ValueError):
        bt.bt_adapter_plan(torch.zeros(2), 2, device="cpu")
    with pytest.raises(ValueError):
        bt.bt_adapter_plan(torch.zeros(2, 2, dtype=torch.int32), 2, device="cpu")


def test_plan_refusals():
    ids = (ctypes.c_int32 * 4)(0, 1, -1, 0)
    need = bt.bt_adapter_plan_bytes(4, 2)
    buf = (ctypes.c_int32 * (need // 4))()
    info = bt.AdapterPlanInfo()

    def call(a=ids, T=4, L=2, p=buf, n=need, i=info):
        return bt._c_aplan(a, T, L, p, n, None if i is None else ctypes.byref(i))

    assert call() == bt.BT_OK
    assert call(a=None) == call(p=None) == call(i=None) == call(T=-1) == call(L=0) == call(L=1) == bt.BT_ERR_INVALID_ARG
    assert call(n=need - 4) == bt.BT_ERR_WORKSPACE
    assert call(T=(1 << 24) + 1) == call(L=65537) == bt.BT_ERR_UNSUPPORTED
    assert call(p=ctypes.cast(ctypes.addressof(buf) + 2, ctypes.c_void_p)) == bt.BT_ERR_ALIGNMENT
    assert call(a=None, T=0) == bt.BT_OK
    assert bt.bt_adapter_plan_bytes(-1, 1) == bt.bt_adapter_plan_bytes(1, 0) == bt.bt_adapter_plan_bytes(1, 65537) == 0


def _info(T=4, L=2, **kw):
    i = bt.bt_adapter_plan([0] * T, L, device="cpu").info
    for k, v in kw.items():
        setattr(i, k, v)
    return ctypes.byref(i)


def _fwd(**kw):
    a = dict(x=256, xt=bt.BT_BF16, ldx=64, A=512, B=1024, s=2048, plan=4096, info=_info(), T=4, K=64, N=32, R=8,
             base=None, bt_=bt.BT_F32, ldb=0, out=8192, ot=bt.BT_BF16, ldo=32, u=None, ws=16384, wsb=1 << 20, st=None)
    a.update(kw)
    return bt._c_alin(*a.values())


def _bwd(**kw):
    a = dict(x=256, ldx=64, g=512, ldg=32, u=768, A=1024, B=2048, s=4096, plan=8192, info=_info(), T=4, K=64, N=32, R=8,
             gb=None, ldgb=0, gx=16384, ldgx=64, ga=32768, gbo=65536, ws=131072, wsb=1 << 20, st=None)
    a.update(kw)
    return bt._c_abwd(*a.values())


def test_forward_refusals(monkeypatch):
    for bad in (dict(xt=bt.BT_F32), dict(xt=bt.BT_I32), dict(ot=bt.BT_F16), dict(ot=bt.BT_I32), dict(K=0, ldx=64),
                dict(T=-1), dict(N=-1), dict(R=0), dict(ldx=63), dict(ldo=31), dict(base=256, ldb=31),
                dict(base=256, ldb=32, bt_=bt.BT_F16), dict(info=None), dict(T=5), dict(info=_info(T=3)), dict(x=None),
                dict(A=None), dict(B=None), dict(s=None), dict(plan=None), dict(out=None),
                dict(base=8192, ldb=32, bt_=bt.BT_F32), dict(base=8192, ldb=40, bt_=bt.BT_BF16, ldo=32),
                dict(info=_info(tiles=5)), dict(info=_info(tiles=-1)), dict(info=_info(without=5)),
                dict(info=_info(slots=17)), dict(info=_info(parts=0))):
        assert _fwd(**bad) == bt.BT_ERR_INVALID_ARG, bad
    for bad in (dict(R=129), dict(K=1 << 24, ldx=1 << 24), dict(N=1 << 24, ldo=1 << 24), dict(ldx=1 << 37)):
        assert _fwd(**bad) == bt.BT_ERR_UNSUPPORTED, bad
    for bad in (dict(x=257), dict(A=513), dict(B=1025), dict(s=2050), dict(plan=4100), dict(out=8193), dict(u=2),
                dict(ot=bt.BT_F32, out=8194), dict(base=258, ldb=32, bt_=bt.BT_F32)):
        assert _fwd(**bad) == bt.BT_ERR_ALIGNMENT, bad
    monkeypatch.setenv("BT_ADAPTER_PATH", "large")
    large = dict(T=40, info=_info(T=40))
    assert _fwd(**large, ws=None) == _fwd(**large, wsb=3 * 1280 - 1) == bt.BT_ERR_WORKSPACE
    assert _fwd(**large, ws=16384 + 16) == bt.BT_ERR_ALIGNMENT
    monkeypatch.delenv("BT_ADAPTER_PATH")
    assert _fwd(T=0, info=_info(T=0), x=None) == _fwd(N=0, out=None) == bt.BT_OK


def test_workspace_queries(monkeypatch):
    ws = bt.bt_adapter_linear_workspace
    one, many, most = (bt.bt_adapter_plan([0] * n, 2, device="cpu") for n in (1, 40, 8192))
    assert ws(1, 4096, 4096, 16, one) == 0                       # one kernel
    assert ws(8192, 4096, 4096, 64, most) == 3 * 8192 * 128
    monkeypatch.setenv("BT_ADAPTER_PATH", "large")
    assert ws(40, 64, 32, 8, many) == 3 * 1280                   # two 16-bit values of 16 ranks, and a third or a power
    # a width that is no multiple of 4: room for the rows of x and A at 16-byte multiples
    assert ws(40, 66, 32, 8, many) == 3 * 1280 + 5888 + 2304
    assert ws(40, 64, 32, 129, many) == ws(41, 64, 32, 8, many) == 0
    monkeypatch.setenv("BT_ADAPTER_PATH", "small")
    assert ws(8192, 4096, 4096, 64, most) == 0


def test_backward_refusals():
    for bad in (dict(K=0), dict(N=0), dict(T=-1), dict(R=0), dict(ldx=63), dict(ldg=31), dict(ldgx=63),
                dict(gb=256, ldgb=63), dict(info=None), dict(T=5), dict(x=None), dict(g=None), dict(u=None), dict(A=None),
                dict(B=None), dict(s=None), dict(plan=None), dict(gx=None), dict(ga=None), dict(gbo=None),
                dict(gb=16384, ldgb=72)):
        assert _bwd(**bad) == bt.BT_ERR_INVALID_ARG, bad
    for bad in (dict(R=129), dict(K=1 << 24, ldx=1 << 24, ldgx=1 << 24), dict(ldg=1 << 37)):
        assert _bwd(**bad) == bt.BT_ERR_UNSUPPORTED, bad
    for bad in (dict(x=257), dict(g=513), dict(u=770), dict(A=1025), dict(B=2049), dict(s=4098), dict(plan=8200),
                dict(gx=16385), dict(ga=32770), dict(gbo=65538), dict(ws=131088)):
        assert _bwd(**bad) == bt.BT_ERR_ALIGNMENT, bad
    assert _bwd(ws=None) == _bwd(wsb=127) == bt.BT_ERR_WORKSPACE
    many = bt.bt_adapter_plan([0] * 4, 65536, device="cpu").info
    assert _bwd(info=ctypes.byref(many), K=1 << 23, ldx=1 << 23, ldgx=1 << 23) == bt.BT_ERR_UNSUPPORTED


def test_binding_refuses_what_it_cannot_pass_on():
    p = bt.bt_adapter_plan([0, 1], 2, device="cpu")
    x, a, b, s = torch.zeros(2, 8).bfloat16(), torch.zeros(2, 4, 8).bfloat16(), torch.zeros(2, 6, 4).bfloat16(), torch.ones(2)
    with pytest.raises(ValueError, match="CUDA"):
        bt.bt_adapter_linear(x, a, b, s, p)
