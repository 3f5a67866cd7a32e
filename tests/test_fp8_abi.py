"""What the FP8 entry points refuse, before any HIP call (the pointers are never dereferenced)."""
import ctypes

import pytest
import torch

import sparse_moe_expert_router_amd as moe
from sparse_moe_expert_router_amd import _lib

OK, NULL, SHAPE, UNSUP, WS = 0, 1, 2, 3, 4
FAKE = ctypes.c_void_p(256)


def test_quantize_refusals():
    q = lambda x=FAKE, dt=0, T=4, n=128, ld=128, c=FAKE, s=FAKE: moe.lib().moe_fp8_quantize(x, dt, T, n, ld, c, s, None)
    assert q(T=-1) == SHAPE and q(n=0) == SHAPE and q(ld=64) == SHAPE
    assert q(dt=2) == UNSUP and q(n=24, ld=24) == UNSUP and q(ld=132) == UNSUP
    assert q(dt=1, ld=130) == UNSUP
    assert q(x=ctypes.c_void_p(258)) == UNSUP and q(c=ctypes.c_void_p(264)) == UNSUP and q(s=ctypes.c_void_p(258)) == UNSUP
    assert q(T=1 << 30) == UNSUP
    assert q(x=None) == NULL and q(c=None) == NULL and q(s=None) == NULL
    assert q(T=0, x=None, c=None, s=None) == OK


def test_matmul_refusals():
    def mm(a=FAKE, sa=FAKE, w=FAKE, sw=FAKE, M=4, N=64, K=128, lda=128, ldw=128, dt=0, y=FAKE, ldy=64):
        return moe.lib().moe_fp8_matmul(a, sa, w, sw, M, N, K, lda, ldw, dt, y, ldy, None)
    assert mm(M=-1) == SHAPE and mm(N=0) == SHAPE and mm(K=0) == SHAPE
    assert mm(lda=112) == SHAPE and mm(ldw=112) == SHAPE and mm(ldy=63) == SHAPE
    assert mm(dt=2) == UNSUP and mm(K=120) == UNSUP and mm(lda=136) == UNSUP and mm(ldw=136) == UNSUP
    assert mm(lda=1 << 23) == UNSUP
    assert mm(a=ctypes.c_void_p(264)) == UNSUP and mm(w=ctypes.c_void_p(264)) == UNSUP
    assert mm(sa=ctypes.c_void_p(258)) == UNSUP and mm(y=ctypes.c_void_p(257)) == UNSUP
    assert mm(dt=1, y=ctypes.c_void_p(258)) == UNSUP
    for name in ("a", "sa", "w", "sw", "y"):
        assert mm(**{name: None}) == NULL
    assert mm(M=0, a=None, sa=None, y=None) == OK


def _bank(fmt=2, E=4, H=256, F=128, ptr=256):
    mk = lambda i, o: _lib._Proj(fmt, i, o, ptr, ptr, ptr, ptr, ptr, ptr)
    return _lib._Experts(E, H, F, mk(H, F), mk(H, F), mk(F, H))


def test_experts_refusals():
    need = moe.workspace_bytes(moe.OP_GROUPED_FFN_A8, 8, 2, 4, 256, 128)
    assert need > 0

    def ffn(b=_bank(), T=8, k=2, x=FAKE, off=FAKE, sp=FAKE, dt=0, rows=FAKE, ws=FAKE, n=need):
        return moe.lib().moe_grouped_ffn_a8(x, T, k, ctypes.byref(b) if b is not None else None, off, sp, dt, rows, ws, n, None)
    assert ffn(b=None) == NULL
    assert ffn(b=_bank(fmt=0)) == UNSUP and ffn(b=_bank(fmt=1)) == UNSUP
    assert ffn(b=_bank(H=320)) == UNSUP and ffn(b=_bank(F=96)) == UNSUP
    assert ffn(T=-1) == SHAPE and ffn(k=0) == SHAPE and ffn(off=None, sp=None) == SHAPE
    assert ffn(off=None) == NULL and ffn(x=None) == NULL and ffn(rows=None) == NULL and ffn(ws=None) == NULL
    assert ffn(n=need - 1) == WS
    assert ffn(ws=ctypes.c_void_p(264)) == UNSUP and ffn(x=ctypes.c_void_p(264)) == UNSUP
    assert ffn(dt=5) == UNSUP
    assert ffn(T=0, x=None, rows=None, ws=None, n=0) == OK
    sizes = [moe.workspace_bytes(moe.OP_GROUPED_FFN_A8, T, 10, 512, 2560, 640) for T in (1, 16, 256, 4096, 32768)]
    assert sizes == sorted(sizes)


def test_the_binding_refuses_what_would_read_out_of_bounds():
    c = torch.zeros((4, 128), dtype=torch.uint8)
    s = torch.ones((4, 1))
    with pytest.raises(moe.MoeError, match="inputs"):
        moe.fp8_matmul(c, s, torch.zeros((8, 144), dtype=torch.uint8), torch.ones((1, 1)))
    with pytest.raises(moe.MoeError, match="scales"):
        moe.fp8_matmul(c, s, torch.zeros((129, 128), dtype=torch.uint8), torch.ones((1, 1)))
    with pytest.raises(moe.MoeError, match="scales"):
        moe.fp8_matmul(c, s[:3], torch.zeros((8, 128), dtype=torch.uint8), torch.ones((1, 1)))
    with pytest.raises(moe.MoeError, match="out_dtype"):
        moe.fp8_matmul(c, s, torch.zeros((8, 128), dtype=torch.uint8), torch.ones((1, 1)), y=torch.zeros((4, 7)))
    with pytest.raises(moe.MoeError, match="GPU tensor"):
        moe.fp8_matmul(c, s, torch.zeros((8, 128), dtype=torch.uint8), torch.ones((1, 1)))
    with pytest.raises(moe.MoeError, match="bf16 or fp32"):
        moe.fp8_quantize(torch.zeros((4, 128), dtype=torch.float16))
    with pytest.raises(moe.MoeError, match="fp8 bank"):
        moe.grouped_ffn_a8(torch.zeros((4, 128), dtype=torch.bfloat16), 1, {"fmt": "bf16"})


def test_the_binding_refuses_other_devices():
    mk = lambda dev: {"fmt": "fp8", "gate_codes": torch.zeros((2, 128, 256), dtype=torch.uint8, device=dev),
                      "up_codes": torch.zeros((2, 128, 256), dtype=torch.uint8, device=dev),
                      "down_codes": torch.zeros((2, 256, 128), dtype=torch.uint8, device=dev),
                      "gate_bscales": torch.ones((2, 1, 2), device=dev), "up_bscales": torch.ones((2, 1, 2), device=dev),
                      "down_bscales": torch.ones((2, 2, 1), device=dev)}
    x = torch.zeros((4, 256), dtype=torch.bfloat16)
    off, sp = torch.zeros(3, dtype=torch.int32), torch.zeros(4, dtype=torch.int32)
    for args in ((mk("meta"), off, sp), (mk("cpu"), off.to("meta"), sp), (mk("cpu"), off, sp.to("meta"))):
        with pytest.raises(moe.MoeError, match="different devices"):
            moe.grouped_ffn_a8(x, 1, *args)
    with pytest.raises(moe.MoeError, match="different devices"):
        moe.fp8_quantize(x, codes=torch.zeros((4, 256), dtype=torch.uint8, device="meta"))
    with pytest.raises(moe.MoeError, match="different devices"):
        moe.fp8_matmul(torch.zeros((4, 128), dtype=torch.uint8), torch.ones((4, 1)),
                       torch.zeros((8, 128), dtype=torch.uint8, device="meta"), torch.ones((1, 1)))


def test_experts_refuse_sizes_past_32_bits():
    def ffn(T, H, F):
        b = _bank(H=H, F=F)
        return moe.lib().moe_grouped_ffn_a8(FAKE, T, 1, ctypes.byref(b), FAKE, FAKE, 0, FAKE, FAKE, 1 << 60, None)
    assert ffn(8, (1 << 20) + 128, 128) == UNSUP and ffn(8, 128, (1 << 20) + 128) == UNSUP
    assert ffn(1 << 22, 1024, 128) == UNSUP


def test_rows_that_share_memory_are_refused():
    """Broadcast rows (stride 0) would be written, or read, as one."""
    q = lambda stride: moe.lib().moe_fp8_quantize(FAKE, 0, 4, 128, stride, FAKE, FAKE, None)
    assert q(0) == SHAPE and q(120) == SHAPE
    mm = lambda lda, ldw, ldy: moe.lib().moe_fp8_matmul(FAKE, FAKE, FAKE, FAKE, 4, 8, 128, lda, ldw, 0, FAKE, ldy, None)
    assert mm(0, 128, 8) == SHAPE and mm(128, 0, 8) == SHAPE and mm(128, 128, 0) == SHAPE


def test_matmul_refuses_more_tiles_than_a_launch_holds():
    """A launch has fewer than 2^32 threads: 2^23 - 8 tiles of 512 (in whole eighths)."""
    mm = lambda M, N: moe.lib().moe_fp8_matmul(FAKE, FAKE, FAKE, FAKE, M, N, 16, 16, 16, 0, FAKE, N, None)
    most = (1 << 31) - 1
    assert mm(1, most) == UNSUP and mm(8, most) == UNSUP and mm(9, most) == UNSUP and mm(64, most) == UNSUP
    assert mm(most, most) == UNSUP and mm(1 << 23, 1 << 20) == UNSUP
    # above 64 rows the largest tiles count: 2^23 - 8 of 256 x 256
    assert mm(256, most) == UNSUP


def test_experts_refuse_more_tiles_than_a_launch_holds():
    """Shallow banks launch one workgroup a tile: 2^23 - 8 of them at most."""
    def ffn(T, k, H, F, dt=0):
        b = _bank(H=H, F=F, E=64)
        return moe.lib().moe_grouped_ffn_a8(FAKE, T, k, ctypes.byref(b), FAKE, FAKE, dt, FAKE, FAKE, 1 << 60, None)
    T = (1 << 25) - 64
    assert ffn(T, 31, 128, 2048) == UNSUP              # gate/up of one block of 128: 4 million tiles of 16 column groups
    assert ffn(T, 4, 128, 2048, 1) == UNSUP            # fp32 rows have tiles of 128 rows at most
    assert ffn(T // 128, 64 * 60, 16384, 256) == UNSUP  # down of two blocks
