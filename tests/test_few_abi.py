"""What moe_layer_few refuses, before any HIP call (the pointers are never dereferenced)."""
import ctypes

import pytest
import torch

import sparse_moe_expert_router_amd as moe
from sparse_moe_expert_router_amd import _lib

OK, NULL, SHAPE, UNSUP, WS = 0, 1, 2, 3, 4
FAKE = ctypes.c_void_p(256)


def _bank(fmt=0, E=16, H=256, F=128, ptr=256):
    mk = lambda i, o: _lib._Proj(fmt, i, o, ptr, ptr, ptr, ptr, ptr, ptr, ptr, ptr, 1.0)
    return _lib._Experts(E, H, F, mk(H, F), mk(H, F), mk(F, H))


def test_refusals():
    L = moe.lib()
    b, sh = _bank(), _bank(E=1, F=64)
    ref = lambda s: ctypes.byref(s) if s is not None else None
    need = L.moe_layer_few_workspace_bytes(8, 2, ref(b), ref(sh))
    assert need > 0 and L.moe_layer_few_workspace_bytes(16, 2, ref(b), ref(sh)) >= need
    assert L.moe_layer_few_workspace_bytes(8, 2, ref(b), None) < need
    for T in (0, -1, 17):
        assert L.moe_layer_few_workspace_bytes(T, 2, ref(b), None) == 0
    for fmt in (1, 3):
        assert L.moe_layer_few_workspace_bytes(8, 2, ref(_bank(fmt=fmt)), None) == 0

    def call(T=8, k=2, bank=b, shared=sh, scale=None, x=FAKE, r=FAKE, y=FAKE, idx=None, ws=FAKE, n=need):
        return L.moe_layer_few(x, T, r, k, ref(bank), ref(shared), scale, y, idx, ws, n, None)
    assert call(k=0) == SHAPE and call(T=-1) == SHAPE and call(k=17) == SHAPE
    assert call(bank=None) == NULL and call(bank=_bank(H=200)) == UNSUP
    assert call(shared=_bank(E=2)) == SHAPE and call(shared=_bank(E=1, H=512)) == SHAPE
    assert call(shared=None, scale=FAKE) == SHAPE
    assert call(T=17) == UNSUP
    assert call(bank=_bank(fmt=1)) == UNSUP and call(bank=_bank(fmt=3)) == UNSUP
    assert call(shared=_bank(fmt=2, E=1)) == UNSUP
    assert call(bank=_bank(E=100), k=65) == UNSUP
    for name in ("x", "r", "y", "ws"):
        assert call(**{name: None}) == NULL, name
    assert call(x=ctypes.c_void_p(264)) == UNSUP and call(y=ctypes.c_void_p(264)) == UNSUP
    assert call(ws=ctypes.c_void_p(264)) == UNSUP and call(scale=ctypes.c_void_p(258)) == UNSUP
    assert call(n=need - 1) == WS
    assert call(T=0, x=None, y=None, ws=None, n=0) == OK


def test_the_binding_refuses():
    bank = {"fmt": "bf16", "gate": torch.zeros((4, 128, 256), dtype=torch.bfloat16),
            "up": torch.zeros((4, 128, 256), dtype=torch.bfloat16), "down": torch.zeros((4, 256, 128), dtype=torch.bfloat16)}
    router = torch.zeros((4, 256), dtype=torch.bfloat16)
    with pytest.raises(moe.MoeError, match="w_router"):
        moe.FewTokenLayer(router[:3], 2, bank)
    with pytest.raises(moe.MoeError, match="at most 16 tokens"):
        moe.FewTokenLayer(router, 2, bank, max_tokens=17)
    few = moe.FewTokenLayer(router, 2, bank, max_tokens=4, ws=type("W", (), {"get": lambda s, n: (torch.empty(n, dtype=torch.uint8), n)})())
    for x in (torch.zeros((2, 128), dtype=torch.bfloat16), torch.zeros((2, 256)), torch.zeros((2, 512), dtype=torch.bfloat16)[:, ::2]):
        with pytest.raises(moe.MoeError, match="x must be"):
            few(x)
    with pytest.raises(moe.MoeError, match="5 tokens"):
        few(torch.zeros((5, 256), dtype=torch.bfloat16))


def test_refuses_overlap_and_sizes_past_32_bits():
    L = moe.lib()
    b = _bank()
    n = L.moe_layer_few_workspace_bytes(8, 2, ctypes.byref(b), None)

    def call(x, y, bank=b):
        return L.moe_layer_few(ctypes.c_void_p(x), 8, FAKE, 2, ctypes.byref(bank), None, None, ctypes.c_void_p(y), None, FAKE,
                               n, None)
    end = 8 * 256 * 2
    for x, y in ((4096, 4096), (4096, 4096 + end - 16), (4096 + end - 16, 4096)):
        assert call(x, y) == SHAPE
    for big in (_bank(H=(1 << 20) + 128), _bank(F=(1 << 20) + 128)):
        assert call(4096, 1 << 30, big) == UNSUP


def test_the_binding_refuses_other_devices():
    mk = lambda dev: {"fmt": "bf16", "gate": torch.zeros((4, 128, 256), dtype=torch.bfloat16, device=dev),
                      "up": torch.zeros((4, 128, 256), dtype=torch.bfloat16, device=dev),
                      "down": torch.zeros((4, 256, 128), dtype=torch.bfloat16, device=dev)}
    router = torch.zeros((4, 256), dtype=torch.bfloat16)
    with pytest.raises(moe.MoeError, match="different devices"):
        moe.FewTokenLayer(router, 2, mk("meta"))
    few = moe.FewTokenLayer(router, 2, mk("cpu"), max_tokens=4,
                            ws=type("W", (), {"get": lambda s, n: (torch.empty(n, dtype=torch.uint8), n)})())
    x = torch.zeros((2, 256), dtype=torch.bfloat16)
    for kw in ({"y": x.to("meta")}, {"topk_idx": torch.zeros((2, 2), dtype=torch.int32, device="meta")},
               {"shared_scale": torch.zeros(2, device="meta")}):
        with pytest.raises(moe.MoeError, match="different devices"):
            few(x, **kw)
