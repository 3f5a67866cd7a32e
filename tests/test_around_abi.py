"""What the operators around the layer refuse, before any HIP call (the pointers are never dereferenced)."""
import ctypes

import pytest
import torch

import sparse_moe_expert_router_amd as moe

OK, NULL, SHAPE, UNSUP, WS = 0, 1, 2, 3, 4
BF16, F32 = 0, 1


def P(n):
    return ctypes.c_void_p(n << 32)


X, RES, ROUT, W, Y, CODES, SCALES, RSTD, DX, DW, WSP = (P(n) for n in range(1, 12))


def _norm(x=X, xd=BF16, ldx=256, r=RES, ldr=256, ro=ROUT, ldro=256, rd=BF16, w=W, wd=BF16, off=1.0, eps=1e-6, T=4, H=256,
          y=Y, ldy=256, c=CODES, s=SCALES, rstd=RSTD):
    return moe.lib().moe_add_rmsnorm(x, xd, ldx, r, ldr, ro, ldro, rd, w, wd, off, eps, T, H, y, ldy, c, s, rstd, None)


def test_norm_refusals():
    assert _norm(T=-1) == SHAPE and _norm(H=0) == SHAPE
    for ld in ("ldx", "ldr", "ldro", "ldy"):
        assert _norm(**{ld: 248}) == SHAPE and _norm(**{ld: 0}) == SHAPE and _norm(**{ld: 260}) == UNSUP
    assert _norm(xd=F32, ldx=258) == UNSUP and _norm(rd=F32, ldr=258) == UNSUP
    for eps in (0.0, -1.0, float("nan"), float("inf")):
        assert _norm(eps=eps) == SHAPE
    assert _norm(off=float("inf")) == SHAPE and _norm(off=float("nan")) == SHAPE
    for d in ("xd", "rd", "wd"):
        assert _norm(**{d: 2}) == UNSUP and _norm(**{d: -1}) == UNSUP
    assert _norm(H=252) == UNSUP and _norm(H=248) == UNSUP                      # codes: whole 16-byte rows
    big = dict(ldx=16400, ldr=16400, ldro=16400, ldy=16400, T=1)
    assert _norm(H=16400, **big) == UNSUP
    for p in ("x", "w", "r", "ro", "c", "s"):
        assert _norm(**{p: None}) == NULL
    assert _norm(y=None, c=None, s=None) == NULL
    for p in ("x", "r", "ro", "w", "y", "c"):
        assert _norm(**{p: ctypes.c_void_p((1 << 40) + 8)}) == UNSUP
    assert _norm(s=ctypes.c_void_p((1 << 40) + 2)) == UNSUP and _norm(rstd=ctypes.c_void_p((1 << 40) + 2)) == UNSUP
    assert _norm(T=0, x=None, w=None, r=None, ro=None, y=None, c=None, s=None, rstd=None) == OK


def test_norm_refuses_overlaps():
    at = lambda p, n: ctypes.c_void_p(p.value + n)
    row = 512
    assert _norm(y=RES, rd=F32) == SHAPE and _norm(ro=X, rd=F32) == SHAPE       # another type
    assert _norm(y=at(X, row)) == SHAPE and _norm(y=at(X, -row)) == SHAPE       # shifted by a row
    assert _norm(y=X, ldy=512) == SHAPE                                         # another stride
    assert _norm(y=ROUT) == SHAPE and _norm(c=X) == SHAPE and _norm(c=Y) == SHAPE and _norm(s=Y) == SHAPE
    assert _norm(rstd=SCALES) == SHAPE and _norm(rstd=W) == SHAPE and _norm(y=at(W, -3 * row)) == SHAPE
    # columns that cross
    assert _norm(x=X, ldx=512, y=at(X, 256), ldy=512) == SHAPE and _norm(x=at(X, 256), ldx=512, y=X, ldy=512) == SHAPE


def _bwd(dy=Y, yd=BF16, ldy=256, s=X, lds=256, sd=BF16, r=RSTD, w=W, wd=BF16, off=1.0, dres=RES, ldr=256, T=4, H=256, dx=DX,
         ldx=256, dw=DW, ws=WSP, n=1 << 30):
    return moe.lib().moe_add_rmsnorm_backward(dy, yd, ldy, s, lds, sd, r, w, wd, off, dres, ldr, T, H, dx, ldx, dw, ws, n, None)


def test_norm_backward_refusals():
    assert _bwd(T=-1) == SHAPE and _bwd(H=0) == SHAPE and _bwd(off=float("nan")) == SHAPE
    for ld in ("ldy", "lds", "ldr", "ldx"):
        assert _bwd(**{ld: 248}) == SHAPE and _bwd(**{ld: 260}) == UNSUP
    for d in ("yd", "sd", "wd"):
        assert _bwd(**{d: 2}) == UNSUP
    assert _bwd(H=252) == UNSUP and _bwd(H=16392, ldy=16392, lds=16392, ldr=16392, ldx=16392) == UNSUP
    for p in ("dy", "s", "r", "w", "dx", "dw", "ws"):
        assert _bwd(**{p: None}) == NULL
    for p in ("dy", "s", "w", "dx", "dres", "ws"):
        assert _bwd(**{p: ctypes.c_void_p((1 << 40) + 8)}) == UNSUP
    assert _bwd(r=ctypes.c_void_p((1 << 40) + 2)) == UNSUP and _bwd(dw=ctypes.c_void_p((1 << 40) + 2)) == UNSUP
    need = moe.workspace_bytes(moe.OP_ADD_RMSNORM_BACKWARD, 4, 1, 1, 256)
    assert need > 0 and _bwd(n=need - 1) == WS
    at = lambda p, n: ctypes.c_void_p(p.value + n)
    assert _bwd(dx=Y, yd=F32) == SHAPE and _bwd(dx=at(X, 512)) == SHAPE and _bwd(dx=at(RES, 16)) == SHAPE
    assert _bwd(dw=X) == SHAPE and _bwd(dw=RSTD) == SHAPE and _bwd(dw=DX) == SHAPE and _bwd(dx=W) == SHAPE
    sizes = [moe.workspace_bytes(moe.OP_ADD_RMSNORM_BACKWARD, T, 1, 1, 2560) for T in (1, 7, 500, 4096, 1 << 20)]
    assert sizes == sorted(sizes)
    for H in (0, -8, 1 << 20, (1 << 31) - 1):
        assert moe.workspace_bytes(moe.OP_ADD_RMSNORM_BACKWARD, 4, 1, 1, H) == 0
    assert moe.workspace_bytes(moe.OP_ADD_RMSNORM_BACKWARD, 4, 1, 1, 4) > 0       # (a size that the call refuses)
    for E in (1025, (1 << 31) - 1):
        assert moe.workspace_bytes(moe.OP_BALANCE_LOSS, 4, 1, E, 0) == 0


def test_counts_refusals():
    c = lambda i=X, T=4, k=2, E=8, v=None, acc=0, n=Y: moe.lib().moe_expert_counts(i, T, k, E, v, acc, n, None)
    assert c(T=-1) == SHAPE and c(k=0) == SHAPE and c(E=0) == SHAPE and c(k=9) == SHAPE
    assert c(E=1025) == UNSUP and c(T=1 << 30, k=8) == UNSUP
    assert c(i=None) == NULL and c(n=None) == NULL
    assert c(i=ctypes.c_void_p(258)) == UNSUP and c(n=ctypes.c_void_p(258)) == UNSUP
    assert c(T=0, acc=1, i=None, n=None) == OK


def _bal(l=X, d=F32, ld=64, T=4, E=64, k=2, c=W, coef=0.01, v=None, i=None, g=None, dg=None, loss=SCALES, ps=None, dl=DX, dd=F32,
         ldd=64, ws=WSP, n=1 << 30):
    return moe.lib().moe_balance_loss(l, d, ld, T, E, k, c, coef, v, i, g, dg, loss, ps, dl, dd, ldd, ws, n, None)


def test_balance_refusals():
    assert _bal(T=-1) == SHAPE and _bal(E=0) == SHAPE and _bal(k=0) == SHAPE and _bal(k=65) == SHAPE
    assert _bal(ld=63) == SHAPE and _bal(ldd=63) == SHAPE
    assert _bal(coef=float("nan")) == SHAPE and _bal(coef=float("inf")) == SHAPE
    assert _bal(E=1025, ld=1025, ldd=1025) == UNSUP and _bal(E=128, ld=128, ldd=128, k=65) == UNSUP
    assert _bal(d=2) == UNSUP and _bal(dd=2) == UNSUP and _bal(T=1 << 30, k=8) == UNSUP
    for p in ("l", "c", "loss", "ws"):
        assert _bal(**{p: None}) == NULL
    given = dict(i=Y, g=CODES, dg=RSTD)
    for p in given:                                    # two of the three
        assert _bal(**{q: v for q, v in given.items() if q != p}) == NULL
    assert _bal(dl=None, **given) == NULL
    for p in ("l", "dl", "c", "loss", "ps"):
        assert _bal(**{p: ctypes.c_void_p((1 << 40) + 2)}) == UNSUP
    assert _bal(ws=ctypes.c_void_p((1 << 40) + 8)) == UNSUP
    need = moe.workspace_bytes(moe.OP_BALANCE_LOSS, 4, 2, 64, 0)
    assert need > 0 and _bal(n=need - 1) == WS
    assert _bal(dl=X, dd=BF16) == SHAPE and _bal(dl=X, ldd=128) == SHAPE and _bal(dl=ctypes.c_void_p(X.value + 256)) == SHAPE
    for E, k in ((512, 10), (60, 6), (1, 1)):
        sizes = [moe.workspace_bytes(moe.OP_BALANCE_LOSS, T, k, E, 0) for T in (1, 16, 700, 32768, 1 << 22)]
        assert sizes == sorted(sizes)


def test_awq_refusals():
    def mm(x=X, ldx=256, q=W, z=Y, s=SCALES, M=4, N=64, K=256, g=32, dt=BF16, y=DX, ldy=64, ws=WSP, n=1 << 30):
        return moe.lib().moe_awq_matmul(x, ldx, q, z, s, M, N, K, g, dt, y, ldy, ws, n, None)
    assert mm(M=-1) == SHAPE and mm(N=0) == SHAPE and mm(K=0) == SHAPE and mm(ldx=248) == SHAPE and mm(ldy=63) == SHAPE
    assert mm(g=16) == UNSUP and mm(g=256) == UNSUP and mm(g=0) == UNSUP and mm(dt=2) == UNSUP
    assert mm(N=60) == UNSUP and mm(K=240) == UNSUP and mm(K=224, g=128) == UNSUP and mm(ldx=260) == UNSUP
    assert mm(N=(1 << 24) + 8, ldy=1 << 25) == UNSUP and mm(K=(1 << 24) + 32, ldx=1 << 25) == UNSUP and mm(M=(1 << 20) + 1) == UNSUP
    assert mm(M=1 << 20, N=1 << 20, ldy=1 << 20) == UNSUP
    for p in ("x", "q", "z", "s", "y"):
        assert mm(**{p: None}) == NULL
    assert mm(x=ctypes.c_void_p((1 << 40) + 8)) == UNSUP and mm(s=ctypes.c_void_p((1 << 40) + 8)) == UNSUP
    assert mm(q=ctypes.c_void_p((1 << 40) + 2)) == UNSUP and mm(z=ctypes.c_void_p((1 << 40) + 2)) == UNSUP
    assert mm(y=ctypes.c_void_p((1 << 40) + 1)) == UNSUP and mm(dt=F32, y=ctypes.c_void_p((1 << 40) + 2)) == UNSUP
    assert mm(y=X) == SHAPE
    assert mm(M=0, x=None, y=None) == OK
    need = moe.lib().moe_awq_matmul_workspace_bytes(1, 8192, 8192, 128)
    if need:
        big = dict(M=1, N=8192, K=8192, g=128, ldx=8192, ldy=8192)
        assert mm(n=need - 1, **big) == WS and mm(ws=None, **big) == NULL and mm(ws=ctypes.c_void_p((1 << 40) + 8), **big) == UNSUP
    for N, K in ((8192, 8192), (264, 8192), (16384, 4096), (2560, 16384)):      # one for the largest M serves the smaller
        sizes = [moe.lib().moe_awq_matmul_workspace_bytes(M, N, K, 32) for M in (1, 2, 4, 5, 16, 17, 32, 33, 40, 64, 65, 300, 5000)]
        assert sizes == sorted(sizes)
    for bad in ((0, 64, 64, 32), (4, 60, 64, 32), (4, 64, 48, 32), (4, 64, 64, 0), (-1, 0, 0, 0), (4, 1 << 30, 64, 32)):
        assert moe.lib().moe_awq_matmul_workspace_bytes(*bad) == 0


def test_the_binding_refuses_what_would_read_out_of_bounds():
    f = lambda *s: torch.zeros(s)
    b = lambda *s: torch.zeros(s, dtype=torch.bfloat16)
    i = lambda *s: torch.zeros(s, dtype=torch.int32)
    bad = [
        (lambda: moe.add_rmsnorm(b(4, 64), b(32)), "weight"),
        (lambda: moe.add_rmsnorm(b(4, 64).half(), b(64)), "x must be"),
        (lambda: moe.add_rmsnorm(b(64, 4).t(), b(64)), "contiguous rows"),
        (lambda: moe.add_rmsnorm(b(4, 64), b(64), b(3, 64)), "residual"),
        (lambda: moe.add_rmsnorm(b(4, 64), b(64), residual_out=b(4, 64)), "without a residual"),
        (lambda: moe.add_rmsnorm(b(4, 64), b(64), b(4, 64), residual_out=f(4, 64)), "residual_out"),
        (lambda: moe.add_rmsnorm(b(4, 64), b(64), y=f(4, 64)), "y must be"),
        (lambda: moe.add_rmsnorm(b(4, 64), b(64), codes=torch.zeros((4, 32), dtype=torch.uint8)), "codes"),
        (lambda: moe.add_rmsnorm(b(4, 64), b(64), outputs=("fp8",), scales=f(4, 2)), "scales"),
        (lambda: moe.add_rmsnorm(b(4, 64), b(64), outputs=("z",)), "outputs"),
        (lambda: moe.add_rmsnorm(b(4, 64), b(64), outputs=("rstd",)), "outputs must"),
        (lambda: moe.add_rmsnorm(b(4, 64), b(64), rstd=f(3)), "rstd"),
        (lambda: moe.add_rmsnorm(b(4, 64), b(64)), "GPU tensor"),
        (lambda: moe.add_rmsnorm(b(4, 64), torch.zeros(64, dtype=torch.bfloat16, device="meta")), "different devices"),
        (lambda: moe.add_rmsnorm_backward(b(4, 64), b(4, 64), f(3), b(64)), "rstd"),
        (lambda: moe.add_rmsnorm_backward(b(4, 32), b(4, 64), f(4), b(64)), "dy"),
        (lambda: moe.add_rmsnorm_backward(b(4, 64), b(4, 64), f(4), b(64), dres=f(4, 64)), "dres"),
        (lambda: moe.add_rmsnorm_backward(b(4, 64), b(4, 64), f(4), b(64), dw=f(63)), "dw"),
        (lambda: moe.add_rmsnorm_backward(b(4, 64), b(4, 64), f(4), b(64)), "GPU tensor"),
        (lambda: moe.expert_counts(i(4, 2).long(), 8), "topk_idx"),
        (lambda: moe.expert_counts(i(4, 2), 8, token_valid=f(4)), "token_valid"),
        (lambda: moe.expert_counts(i(4, 2), 8, token_valid=torch.ones(3, dtype=torch.bool)), "token_valid"),
        (lambda: moe.expert_counts(i(4, 2), 8, counts=i(7)), "counts"),
        (lambda: moe.expert_counts(i(4, 2), 8, accumulate=True), "accumulate"),
        (lambda: moe.balance_loss(f(4, 8), i(7), 2, 0.1), "counts"),
        (lambda: moe.balance_loss(f(4, 8).half(), i(8), 2, 0.1), "logits"),
        (lambda: moe.balance_loss(f(4, 8), i(8), 2, 0.1, dlogits=f(4, 7)), "dlogits"),
        (lambda: moe.balance_loss(f(4, 8), i(8), 2, 0.1, topk_idx=i(4, 3), gate=f(4, 2), dgate=f(4, 2)), "topk_idx"),
        (lambda: moe.balance_loss(f(4, 8), i(8), 2, 0.1, topk_idx=i(4, 2), gate=f(4, 2)), "go together"),
        (lambda: moe.awq_matmul(b(4, 64), i(64, 4), i(2, 8), torch.zeros((2, 64)).half()), "qweight"),
        (lambda: moe.awq_matmul(b(4, 64), i(64, 8), i(2, 8), torch.zeros((2, 32)).half()), "scales"),
        (lambda: moe.awq_matmul(b(4, 64), i(64, 8), i(3, 8), torch.zeros((3, 64)).half()), "qzeros"),
        (lambda: moe.awq_matmul(f(4, 64), i(64, 8), i(2, 8), torch.zeros((2, 64)).half()), "x must be bf16"),
        (lambda: moe.awq_matmul(b(4, 64), i(64, 8), i(2, 8), torch.zeros((2, 64)).half(), y=f(4, 32)), "y must be"),
        (lambda: moe.awq_matmul(b(4, 64), i(64, 8), i(2, 8), torch.zeros((2, 64)).half(), out_dtype=moe.OUT_BF16, y=f(4, 64)), "out_dtype"),
        (lambda: moe.awq_matmul(b(4, 64), i(64, 8), i(2, 8), torch.zeros((2, 64)).half()), "GPU tensor"),
    ]
    for call, what in bad:
        with pytest.raises(moe.MoeError, match=what):
            call()
