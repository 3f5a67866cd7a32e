"""What prepared calls and workspaces keep alive and in order, without a GPU (nothing is launched)."""
import gc
import weakref

import pytest
import torch

import sparse_moe_expert_router_amd as moe


def _bank(E=4, H=256, F=128):
    z = lambda *s: torch.zeros(s, dtype=torch.bfloat16)
    return {"fmt": "bf16", "gate": z(E, F, H), "up": z(E, F, H), "down": z(E, H, F)}


def _few(bank, shared):
    return moe.FewTokenLayer(torch.zeros((4, 256), dtype=torch.bfloat16), 2, bank, shared, max_tokens=4,
                             ws=moe.Workspace(torch.device("cpu")))


def _layer(bank, shared):
    return moe.LayerCall(torch.zeros((4, 256), dtype=torch.bfloat16), torch.zeros((4, 256), dtype=torch.bfloat16), 2, bank, shared)


@pytest.mark.parametrize("make", [_few, _layer])
def test_a_prepared_call_keeps_the_weights_it_points_to(make):
    """The caller may put other tensors into the dicts afterwards; the call's own stay where its pointers say."""
    bank, shared = _bank(), _bank(E=1)
    call = make(bank, shared)
    for d, st in ((bank, call.st), (shared, call.sh)):
        for name in ("gate", "up", "down"):
            old, at = weakref.ref(d[name]), d[name].data_ptr()
            d[name] = torch.zeros_like(d[name])
            gc.collect()
            assert old() is not None and old().data_ptr() == at == getattr(st, name).w
