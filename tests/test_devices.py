"""CPU: which device the adapters' and the distillation's calls run on, and what they refuse, with tensors that have a
device and no memory. Nothing is launched."""
from types import SimpleNamespace

import pytest
import torch
from torch._subclasses import FakeTensorMode

import xnor_popcount_gemm_gb300 as bt

# (with a GPU, a tensor without memory brings up its device all the same, and there may be only one)
pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="for machines without a GPU")
T, K, N, R, L, V, S = 4, 16, 24, 8, 2, 50, 3


class Entered(Exception):
    pass


@pytest.fixture
def fake(monkeypatch):
    """Device 1 is where the tensors are, device 0 or 1 the current one."""
    state = SimpleNamespace(current=1)
    monkeypatch.setattr(bt, "_current_device", lambda: state.current)

    def device(d):
        raise Entered(f"device {d}")

    monkeypatch.setattr(torch.cuda, "device", device)
    plan = bt.bt_adapter_plan([0, 1, -1, 0], L, device="cpu")
    with FakeTensorMode():
        def t(*shape, dtype=torch.bfloat16, on="cuda:1"):
            return torch.empty(*shape, dtype=dtype, device=on)
        state.t = t
        state.plan = bt.AdapterPlan(t(plan.buffer.numel(), dtype=torch.int32), plan.info)
        f = torch.float32
        state.adapter = dict(x=t(T, K), a=t(L, R, K), b=t(L, N, R), scale=t(L, dtype=f), plan=state.plan)
        state.adapter_more = dict(base=t(T, N), u=t(T, R, dtype=f), out=t(T, N), workspace=t(1 << 20, dtype=torch.uint8))
        state.backward = dict(x=t(T, K), g=t(T, N), u=t(T, R, dtype=f), a=t(L, R, K), b=t(L, N, R), scale=t(L, dtype=f), plan=state.plan)
        state.backward_more = dict(grad_base=t(T, K), grad_x=t(T, K), grad_a=t(L, R, K, dtype=f), grad_b=t(L, N, R, dtype=f),
                                   workspace=t(1 << 20, dtype=torch.uint8))
        teacher = dict(ids=t(T, S, dtype=torch.int32), top=t(T, S, dtype=f))
        more = dict(teacher_lse=t(T, dtype=f))
        state.loss = dict(logits=t(T, V), **teacher)
        state.loss_more = dict(loss=t(T, dtype=f), stats=t(T, 2, dtype=f), **more)
        state.loss_bwd = dict(grad_loss=t(T, dtype=f), logits=t(T, V), **teacher, stats=t(T, 2, dtype=f))
        state.loss_bwd_more = dict(grad=t(T, V), **more)
        state.step = dict(grad_loss=t(T, dtype=f), logits=t(T, V), **teacher)
        state.step_more = dict(loss=t(T, dtype=f), grad=t(T, V), stats=t(T, 2, dtype=f), **more)
        yield state


CALLS = [("bt_adapter_linear", "adapter", "x"), ("bt_adapter_linear_backward", "backward", "x"),
         ("bt_distill_topk", "loss", "logits"), ("bt_distill_topk_backward", "loss_bwd", "logits"),
         ("bt_distill_topk_step", "step", "logits")]


@pytest.mark.parametrize("name,args,first", CALLS)
def test_the_operands_device_is_made_current(fake, name, args, first, monkeypatch):
    def launching(*_):
        raise Entered("launching")

    fake.current = 0
    args, more = getattr(fake, args), getattr(fake, args + "_more")
    with pytest.raises(Entered, match="device 1"):
        getattr(bt, name)(**args)
    with pytest.raises(Entered, match="device 1"):
        getattr(bt, name)(*args.values())
    fake.current = 1
    monkeypatch.setattr(bt, "_on_stream", launching)
    with pytest.raises(Entered, match="launching"):
        getattr(bt, name)(**args, **more)


def test_workspace_sizes_are_of_the_plans_device(fake):
    fake.current = 0
    for call in (bt.bt_adapter_linear_workspace, bt.bt_adapter_linear_backward_workspace):
        with pytest.raises(Entered, match="device 1"):
            call(T, K, N, R, fake.plan)
        with pytest.raises(Entered, match="device 1"):
            call(T, K, N, R, plan=fake.plan)


@pytest.mark.parametrize("name,args,first", CALLS)
def test_operands_of_several_devices_are_refused(fake, name, args, first):
    some, more = getattr(fake, args), getattr(fake, args + "_more")
    for which in [*some, *more]:
        if which == first:
            continue
        for on in ("cuda:0", "cpu"):
            bad = {**some, **more}
            if which == "plan":
                bad["plan"] = bt.AdapterPlan(fake.t(*fake.plan.buffer.shape, dtype=torch.int32, on=on), fake.plan.info)
            else:
                bad[which] = fake.t(*bad[which].shape, dtype=bad[which].dtype, on=on)
            with pytest.raises(ValueError):
                getattr(bt, name)(**bad)
    with pytest.raises(ValueError, match="stream"):
        getattr(bt, name)(**some, stream=SimpleNamespace(device=torch.device("cuda:0"), cuda_stream=0))


def test_a_plans_stream_is_of_its_device():
    with pytest.raises(ValueError, match="stream"):
        bt.bt_adapter_plan([0], 1, device="cuda:1", stream=SimpleNamespace(device=torch.device("cuda:0")))
