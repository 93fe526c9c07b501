"""CPU checks of the distillation entry points: refusals before anything is
launched (no pointer below is ever dereferenced)."""
import pytest
import torch

import xnor_popcount_gemm_gb300 as bt


def _loss(**kw):
    a = dict(z=256, dt=bt.BT_BF16, T=4, V=100, ld=100, ids=512, idb=4, top=768, td=bt.BT_F32, S=8, tlse=None, tau=1.0,
             loss=1024, stats=2048, stream=None)
    a.update(kw)
    return bt._c_distill(*a.values())


def _bwd(**kw):
    a = dict(w=64, z=256, dt=bt.BT_BF16, T=4, V=100, ld=100, ids=512, idb=4, top=768, td=bt.BT_F32, S=8, stats=2048,
             tlse=None, tau=1.0, grad=4096, ldg=100, stream=None)
    a.update(kw)
    return bt._c_distill_bwd(*a.values())


def _step(**kw):
    a = dict(w=64, z=256, dt=bt.BT_BF16, T=4, V=100, ld=100, ids=512, idb=4, top=768, td=bt.BT_F32, S=8, tlse=None,
             tau=1.0, loss=1024, stats=None, grad=4096, ldg=100, stream=None)
    a.update(kw)
    return bt._c_distill_step(*a.values())


@pytest.mark.parametrize("call", [_loss, _bwd, _step])
def test_refusals(call):
    for bad in (dict(dt=bt.BT_I32), dict(td=bt.BT_I32), dict(idb=2), dict(T=-1), dict(V=0), dict(S=0), dict(ld=99),
                dict(tau=0.0), dict(tau=-1.0), dict(tau=float("nan")), dict(tau=float("inf")), dict(tau=1e-45),
                dict(z=None), dict(ids=None), dict(top=None)):
        assert call(**bad) == bt.BT_ERR_INVALID_ARG, bad
    for bad in (dict(S=1025), dict(V=(1 << 28) + 1, ld=1 << 29, ldg=1 << 29), dict(ld=1 << 37), dict(T=(1 << 24) + 1)):
        if call is _loss:
            bad.pop("ldg", None)
        assert call(**bad) == bt.BT_ERR_UNSUPPORTED, bad
    for bad in (dict(z=257), dict(ids=514), dict(idb=8, ids=516), dict(top=770), dict(tlse=6)):
        assert call(**bad) == bt.BT_ERR_ALIGNMENT, bad
    assert call(T=0, z=None, ids=None, top=None) == bt.BT_OK


def test_refusals_of_outputs():
    assert _loss(loss=None) == bt.BT_ERR_INVALID_ARG
    assert _loss(loss=1026) == bt.BT_ERR_ALIGNMENT
    assert _loss(stats=1026) == bt.BT_ERR_ALIGNMENT
    for call in (_bwd, _step):
        assert call(grad=None) == bt.BT_ERR_INVALID_ARG
        assert call(w=None) == bt.BT_ERR_INVALID_ARG
        assert call(ldg=99) == bt.BT_ERR_INVALID_ARG
        assert call(grad=256, ld=104, ldg=112) == bt.BT_ERR_INVALID_ARG      # in place with other rows
        assert call(grad=4097) == bt.BT_ERR_ALIGNMENT
        assert call(w=62) == bt.BT_ERR_ALIGNMENT
    assert _bwd(stats=None) == bt.BT_ERR_INVALID_ARG
    assert _step(loss=None) == bt.BT_ERR_INVALID_ARG


def test_binding_refuses_what_it_cannot_pass_on():
    z, ids, top = torch.zeros(2, 8), torch.zeros(2, 3, dtype=torch.int32), torch.zeros(2, 3)
    with pytest.raises(ValueError, match="CUDA tensor"):
        bt.bt_distill_topk(z, ids, top)
