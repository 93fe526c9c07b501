"""Calls whose operands lie on the current device do not change it (on the CPU, by tensors without memory)."""
import pytest
import torch

import xnor_popcount_gemm_gb300 as bt
from test_mx import _calls, fake  # noqa: F401


class Launching(Exception):
    pass


def test_the_current_device_is_left_alone(fake, monkeypatch):  # noqa: F811
    entered = []

    class Recorder:
        def __init__(self, device):
            entered.append(device)

        def __enter__(self):
            pass

        def __exit__(self, *_):
            return False

    def launching(*_):
        raise Launching

    monkeypatch.setattr(torch.cuda, "device", Recorder)
    monkeypatch.setattr(bt, "_on_stream", launching)
    for call, args, more in _calls(fake):
        for given in (args, {**args, **more}):
            fake.current = 1
            entered.clear()
            # (a tensor without memory has no address: some calls ask for one before they ask for the stream)
            with pytest.raises((Launching, RuntimeError)):
                call(**given)
            assert entered == []
            # the record works: elsewhere the call does change it
            fake.current = 0
            with pytest.raises((Launching, RuntimeError)):
                call(**given)
            assert entered == [1]
    grads = [fake.t(5), fake.t(7)]
    for current, want in ((1, []), (0, [1])):
        fake.current = current
        entered.clear()
        with pytest.raises((Launching, RuntimeError)):
            bt.bt_clip_grads(grads, 1.0)
        assert entered == want
