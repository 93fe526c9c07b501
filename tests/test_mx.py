"""CPU checks of the microscaled operands', the norm's and the clipping's entry points: sizes, and refusals before anything
is launched (no pointer below is ever dereferenced); which device a call runs on, with tensors that have a device and no
memory."""
import ctypes
from types import SimpleNamespace

import pytest
import torch
from torch._subclasses import FakeTensorMode

import xnor_popcount_gemm_gb300 as bt
from mx_reference import quantized, scale_at

E4M3, E2M1 = bt.BT_CODE_E4M3, bt.BT_CODE_E2M1
BAD, ALIGN, WS, NO = bt.BT_ERR_INVALID_ARG, bt.BT_ERR_ALIGNMENT, bt.BT_ERR_WORKSPACE, bt.BT_ERR_UNSUPPORTED


def test_sizes():
    assert [bt.bt_mx_row_bytes(k, E2M1) for k in (1, 256, 257, 4096)] == [128, 128, 256, 2048]
    assert [bt.bt_mx_row_bytes(k, E4M3) for k in (1, 128, 129, 4096)] == [128, 128, 256, 4096]
    assert bt.bt_mx_row_bytes(0, E4M3) == bt.bt_mx_row_bytes(5, bt.BT_CODE_BITS) == bt.bt_mx_row_bytes(1 << 24, E4M3) == 0
    # 512 bytes for 128 rows and 4 blocks; E2M1 rows are whole pairs of those
    assert bt.bt_mx_scale_bytes(1, 32, E4M3) == 512 and bt.bt_mx_scale_bytes(1, 32, E2M1) == 1024
    assert bt.bt_mx_scale_bytes(129, 4096, E4M3) == 2 * 32 * 512 == bt.bt_mx_scale_bytes(129, 4096, E2M1)
    assert bt.bt_mx_scale_bytes(0, 64, E4M3) == 0 == bt.bt_mx_scale_bytes(1 << 24, 64, E4M3)
    # few rows are quantised by the product itself
    assert bt.bt_mx_linear_workspace(16, 4096, 4096, bt.BT_BF16, E2M1) == 0
    assert bt.bt_mx_linear_workspace(200, 4096, 4096, bt.BT_BF16, E2M1) == 200 * 2048 + 2 * 32 * 512
    assert bt.bt_mx_linear_workspace(200, 4096, 4096, bt.BT_PACKED, E2M1) == 0
    assert bt.bt_mx_linear_backward_workspace(7, 9) == 256 and bt.bt_mx_linear_backward_workspace(0, 9) == 0
    assert bt.bt_rms_norm_backward_workspace(0, 64) == 0 and bt.bt_rms_norm_backward_workspace(5, 64) >= 5 * 64 * 4
    assert bt.bt_clip_grads_workspace(0) == 0 and bt.bt_clip_grads_workspace(1) > 0


@pytest.mark.parametrize("code", [E4M3, E2M1])
def test_the_scales_places_are_all_different(code):
    R, K = 300, 700
    n = bt.bt_mx_row_bytes(K, code) // (16 if code == E2M1 else 32)
    at = scale_at(R, n, K, code)
    assert at.unique().numel() == R * n and int(at.max()) < bt.bt_mx_scale_bytes(R, K, code)


@pytest.mark.parametrize("code", [E4M3, E2M1])
def test_the_reference_keeps_what_the_format_holds(code):
    # (of the tests' own reference: values of the format, times powers of two, come back)
    from mx_reference import FORMAT, table
    t = table(code).float()
    x = torch.cat([t, -t, torch.full((1,), 2.0 ** FORMAT[code][2])])
    x = torch.nn.functional.pad(x, (0, -len(x) % 32)).view(-1, 32)
    x[:, 0] = 2.0 ** FORMAT[code][2]
    for e in (-100, 0, 7):
        v = torch.ldexp(x, torch.tensor(e))
        assert torch.equal(quantized(v, code)[0], v.double())


def _quant(**kw):
    a = dict(x=256, dt=bt.BT_BF16, ldx=64, R=4, K=64, code=E4M3, q=512, s=1024, stream=None)
    a.update(kw)
    return bt._c_mx_q(*a.values())


def _dequant(**kw):
    a = dict(q=512, s=1024, R=4, K=64, code=E4M3, out=256, dt=bt.BT_BF16, ldo=64, stream=None)
    a.update(kw)
    return bt._c_mx_dq(*a.values())


def _linear(**kw):
    a = dict(x=256, xt=bt.BT_BF16, ldx=64, xs=None, w=512, ws=1024, code=E2M1, M=40, N=32, K=64, out=2048, ot=bt.BT_BF16, ldo=32,
             work=4096, bytes=1 << 30, stream=None)
    a.update(kw)
    return bt._c_mx_lin(*a.values())


def _transpose(**kw):
    a = dict(q=512, s=1024, R=4, K=64, code=E4M3, ld=8, out=256, stream=None)
    a.update(kw)
    return bt._c_mx_t(*a.values())


def _back(**kw):
    a = dict(g=256, ldg=33, wt=512, ldw=40, M=4, N=33, K=64, gx=1024, t=bt.BT_BF16, work=4096, bytes=1 << 30, stream=None)
    a.update(kw)
    return bt._c_mx_bwd(*a.values())


def _norm(**kw):
    a = dict(x=256, dt=bt.BT_BF16, ldx=64, r=512, ldr=64, w=1024, wt=bt.BT_F32, T=4, N=64, eps=1e-6, sum=2048, lds=64, out=4096, ldo=64,
             code=E4M3, q=8192, s=16384, stream=None)
    a.update(kw)
    return bt._c_rms(*a.values())


def _norm_bwd(**kw):
    a = dict(g=256, dt=bt.BT_BF16, ldg=64, h=512, ldh=64, w=1024, wt=bt.BT_F32, T=4, N=64, eps=1e-6, gs=2048, ldgs=64, gx=4096, ldgx=64,
             gw=8192, work=16384, bytes=1 << 30, stream=None)
    a.update(kw)
    return bt._c_rms_bwd(*a.values())


@pytest.mark.parametrize("call,bad,status", [
    (_quant, dict(dt=bt.BT_I32), BAD), (_quant, dict(R=-1), BAD), (_quant, dict(K=0), BAD), (_quant, dict(ldx=63), BAD),
    (_quant, dict(code=bt.BT_CODE_BITS), BAD), (_quant, dict(x=None), BAD), (_quant, dict(q=None), BAD), (_quant, dict(s=None), BAD),
    (_quant, dict(x=257), ALIGN), (_quant, dict(q=520), ALIGN), (_quant, dict(s=1032), ALIGN), (_quant, dict(K=1 << 24, ldx=1 << 24), NO),
    (_quant, dict(R=1 << 23, K=1 << 20, ldx=1 << 20), NO), (_quant, dict(ldx=1 << 37), NO),
    (_dequant, dict(dt=bt.BT_I32), BAD), (_dequant, dict(ldo=63), BAD), (_dequant, dict(out=None), BAD), (_dequant, dict(q=None), BAD),
    (_dequant, dict(out=257), ALIGN), (_dequant, dict(q=520), ALIGN), (_dequant, dict(R=1 << 24), NO),
    (_linear, dict(xt=bt.BT_I32), BAD), (_linear, dict(ot=bt.BT_I32), BAD), (_linear, dict(code=0), BAD), (_linear, dict(M=-1), BAD),
    (_linear, dict(K=0), BAD), (_linear, dict(ldx=63), BAD), (_linear, dict(ldo=31), BAD), (_linear, dict(x=None), BAD), (_linear, dict(w=None), BAD),
    (_linear, dict(ws=None), BAD), (_linear, dict(out=None), BAD), (_linear, dict(xt=bt.BT_PACKED), BAD), (_linear, dict(x=257), ALIGN),
    (_linear, dict(w=520), ALIGN), (_linear, dict(ws=1032), ALIGN), (_linear, dict(out=2049), ALIGN), (_linear, dict(work=4100), ALIGN),
    (_linear, dict(xt=bt.BT_PACKED, xs=8200), ALIGN), (_linear, dict(work=None), WS), (_linear, dict(bytes=100), WS), (_linear, dict(N=1 << 24, ldo=1 << 24), NO),
    (_linear, dict(M=1 << 24), NO), (_linear, dict(ldo=1 << 37), NO),
    (_transpose, dict(ld=3), BAD), (_transpose, dict(ld=12), BAD), (_transpose, dict(code=0), BAD), (_transpose, dict(out=None), BAD),
    (_transpose, dict(q=None), BAD), (_transpose, dict(out=264), ALIGN), (_transpose, dict(K=65535 * 64 + 1), NO), (_transpose, dict(ld=1 << 24), NO),
    (_back, dict(t=bt.BT_F16), BAD), (_back, dict(M=-1), BAD), (_back, dict(K=0), BAD), (_back, dict(ldg=32), BAD), (_back, dict(ldw=33), BAD),
    (_back, dict(ldw=42), BAD), (_back, dict(g=None), BAD), (_back, dict(wt=None), BAD), (_back, dict(gx=None), BAD), (_back, dict(g=257), ALIGN),
    (_back, dict(wt=520), ALIGN), (_back, dict(gx=1025), ALIGN), (_back, dict(work=None), WS), (_back, dict(bytes=10), WS), (_back, dict(work=4100), ALIGN),
    (_back, dict(K=1 << 24), NO), (_back, dict(ldg=1 << 37), NO),
    (_norm, dict(dt=bt.BT_I32), BAD), (_norm, dict(wt=bt.BT_F16), BAD), (_norm, dict(T=-1), BAD), (_norm, dict(N=0), BAD), (_norm, dict(eps=-1.0), BAD),
    (_norm, dict(eps=float("nan")), BAD), (_norm, dict(eps=float("inf")), BAD), (_norm, dict(code=0), BAD), (_norm, dict(ldx=63), BAD), (_norm, dict(ldr=63), BAD),
    (_norm, dict(lds=63), BAD), (_norm, dict(ldo=63), BAD), (_norm, dict(r=None), BAD), (_norm, dict(q=None), BAD), (_norm, dict(s=None), BAD),
    (_norm, dict(out=None, q=None, s=None), BAD), (_norm, dict(x=None), BAD), (_norm, dict(sum=256, lds=72), BAD), (_norm, dict(out=2048), BAD),
    (_norm, dict(out=256, ldo=72), BAD), (_norm, dict(x=257), ALIGN), (_norm, dict(w=1026), ALIGN), (_norm, dict(q=8200), ALIGN), (_norm, dict(s=16392), ALIGN),
    (_norm, dict(T=1 << 24), NO), (_norm, dict(ldx=1 << 37), NO),
    (_norm_bwd, dict(dt=bt.BT_I32), BAD), (_norm_bwd, dict(wt=bt.BT_F16), BAD), (_norm_bwd, dict(N=0), BAD), (_norm_bwd, dict(eps=-1.0), BAD),
    (_norm_bwd, dict(ldg=63), BAD), (_norm_bwd, dict(ldh=63), BAD), (_norm_bwd, dict(ldgs=63), BAD), (_norm_bwd, dict(ldgx=63), BAD), (_norm_bwd, dict(g=None), BAD),
    (_norm_bwd, dict(h=None), BAD), (_norm_bwd, dict(gx=None), BAD), (_norm_bwd, dict(gx=256, ldgx=72), BAD), (_norm_bwd, dict(gx=2048, ldgx=72), BAD),
    (_norm_bwd, dict(g=257), ALIGN), (_norm_bwd, dict(gw=8194), ALIGN), (_norm_bwd, dict(work=16392), ALIGN), (_norm_bwd, dict(work=None), WS),
    (_norm_bwd, dict(bytes=100), WS), (_norm_bwd, dict(T=1 << 24), NO), (_norm_bwd, dict(ldgx=1 << 37), NO)])
def test_refusals(call, bad, status):
    assert call(**bad) == status


def test_nothing_to_do():
    assert _quant(R=0, x=None) == _dequant(R=0, q=None) == _linear(M=0, x=None) == _linear(N=0, w=None, ldo=0) == bt.BT_OK
    assert _norm(T=0, x=None) == _back(M=0, g=None) == _transpose(R=0, ld=0, out=None) == bt.BT_OK
    assert _norm_bwd(T=0, g=None, gw=None) == bt.BT_OK


def _clip(tensors, max_norm=1.0, eps=1e-6, norm=64, work=256, size=1 << 30, count=None):
    n = len(tensors)
    p = (ctypes.c_void_p * max(n, 1))(*[t[0] for t in tensors])
    m = (ctypes.c_int64 * max(n, 1))(*[t[1] for t in tensors])
    d = (ctypes.c_int32 * max(n, 1))(*[t[2] for t in tensors])
    return bt._c_clip(p, m, d, n if count is None else count, max_norm, eps, norm, work, size, None)


def test_clip_refusals():
    F, H = bt.BT_F32, bt.BT_BF16
    ok = (4096, 100, F)
    assert _clip([ok], max_norm=-1.0) == _clip([ok], max_norm=float("nan")) == _clip([ok], eps=-1.0) == _clip([ok], eps=float("inf")) == BAD
    assert _clip([ok], norm=None) == _clip([(None, 5, F)]) == _clip([(4096, -1, F)]) == _clip([(4096, 5, bt.BT_I32)]) == BAD
    assert _clip([ok], count=-1) == BAD and _clip([ok], norm=66) == ALIGN and _clip([(4098, 5, F)]) == ALIGN and _clip([(4097, 5, H)]) == ALIGN
    assert _clip([ok], work=None) == _clip([ok], size=8) == WS and _clip([ok], work=260) == ALIGN
    assert _clip([(4096, 1 << 41, F)]) == _clip([ok], count=(1 << 20) + 1) == NO
    # an element of two tensors, in any order
    for a, b in (((4096, 100, F), (4096, 100, F)), ((4096, 100, F), (4492, 5, F)), ((8192, 10, H), (8190, 2, H))):
        assert _clip([a, b]) == _clip([b, a]) == _clip([(64, 4, F), b, (1 << 20, 7, H), a]) == BAD


def test_binding_refuses_what_it_cannot_pass_on():
    x = torch.zeros(4, 64)
    for call in (lambda: bt.bt_mx_quantize(x, E4M3), lambda: bt.bt_rms_norm(x), lambda: bt.bt_clip_grads([x], 1.0), lambda: bt.bt_clip_grads([], 1.0),
                 lambda: bt.bt_clip_grads([3.0], 1.0), lambda: bt.bt_mx_dequantize(x), lambda: bt.bt_mx_linear(x, x), lambda: bt.bt_mx_transpose(x)):
        with pytest.raises(ValueError):
            call()


# ---------------------------------------------------------------------------
# devices
# ---------------------------------------------------------------------------
class Entered(Exception):
    pass


@pytest.fixture
def fake(monkeypatch):
    """Device 1 is where the tensors are, device 0 or 1 the current one."""
    if torch.cuda.is_available():
        pytest.skip("for machines without a GPU: a tensor without memory brings up its device all the same")
    state = SimpleNamespace(current=1)
    monkeypatch.setattr(bt, "_current_device", lambda: state.current)

    def device(d):
        raise Entered(f"device {d}")

    monkeypatch.setattr(torch.cuda, "device", device)
    with FakeTensorMode():
        def t(*shape, dtype=torch.bfloat16, on="cuda:1"):
            return torch.empty(*shape, dtype=dtype, device=on)

        def mx(R, K, on="cuda:1"):
            return bt.MxRows(t(R, bt.bt_mx_row_bytes(K, E2M1), dtype=torch.uint8, on=on),
                             t(bt.bt_mx_scale_bytes(R, K, E2M1), dtype=torch.uint8, on=on), K, E2M1)
        state.t, state.mx = t, mx
        yield state


def _calls(s, on=None):
    """(function, arguments, optional ones) of every entry point; `on`: (name, device) of one operand elsewhere."""
    f, big = torch.float32, 1 << 22

    def at(name):
        return on[1] if on is not None and on[0] == name else "cuda:1"

    def t(name, *shape, dtype=torch.bfloat16):
        return s.t(*shape, dtype=dtype, on=at(name))

    def mx(name, R, K):
        return s.mx(R, K, on=at(name))

    u8 = dict(dtype=torch.uint8)
    return [
        (bt.bt_mx_quantize, dict(x=t("x", 4, 64), code=E2M1), dict(out=mx("out", 4, 64))),
        (bt.bt_mx_dequantize, dict(q=mx("q", 4, 64)), dict(out=t("out", 4, 64))),
        (bt.bt_mx_linear, dict(x=t("x", 40, 64), w=mx("w", 24, 64)), dict(out=t("out", 40, 24), workspace=t("workspace", big, **u8))),
        (bt.bt_mx_transpose, dict(w=mx("w", 24, 64)), dict(out=t("out", 64, 64))),
        (bt.bt_mx_linear_backward, dict(g=t("g", 40, 24), wt=t("wt", 64, 64)), dict(grad_x=t("grad_x", 40, 64), workspace=t("workspace", big, **u8))),
        (bt.bt_rms_norm, dict(x=t("x", 4, 64)), dict(weight=t("weight", 64), residual=t("residual", 4, 64), sum=t("sum", 4, 64), out=t("out", 4, 64), q=mx("q", 4, 64))),
        (bt.bt_rms_norm_backward, dict(g=t("g", 4, 64), h=t("h", 4, 64)),
         dict(weight=t("weight", 64), grad_sum=t("grad_sum", 4, 64), grad_x=t("grad_x", 4, 64), grad_weight=t("grad_weight", 64, dtype=f), workspace=t("workspace", big, **u8))),
    ]


def test_the_operands_device_is_made_current(fake, monkeypatch):
    def launching(*_):
        raise Entered("launching")

    for call, args, more in _calls(fake):
        fake.current = 0
        with pytest.raises(Entered, match="device 1"):
            call(**args)
        with pytest.raises(Entered, match="device 1"):
            call(*args.values())
        fake.current = 1
        with monkeypatch.context() as m:
            m.setattr(bt, "_on_stream", launching)
            with pytest.raises((Entered, RuntimeError)):        # (a tensor without memory has no address)
                call(**args, **more)
    fake.current = 0
    for grads in ([fake.t(5), fake.t(7)], (fake.t(5),), iter([fake.t(5)]), {"a": fake.t(5)}.values()):
        with pytest.raises(Entered, match="device 1"):
            bt.bt_clip_grads(grads, 1.0)


def test_operands_of_several_devices_are_refused(fake):
    for i, (call, args, more) in enumerate(_calls(fake)):
        first = next(iter(args))
        for which in [*args, *more]:
            if which in (first, "code"):
                continue
            with pytest.raises(ValueError, match="device|CUDA"):
                call, a, m = _calls(fake, (which, "cuda:0"))[i]
                call(**a, **m)
        with pytest.raises(ValueError, match="stream"):
            call(**args, stream=SimpleNamespace(device=torch.device("cuda:0"), cuda_stream=0))
    with pytest.raises(ValueError, match="device"):
        bt.bt_clip_grads([fake.t(5), fake.t(7, on="cuda:0")], 1.0)
    with pytest.raises(ValueError):
        bt.bt_clip_grads([fake.t(5)], 1.0, norm=fake.t((), dtype=torch.float32, on="cuda:0"))
