"""Memory that the operators around the layer refuse to share between an output and anything else, and
workspaces that are too small, before any HIP call (the pointers are never dereferenced)."""
import ctypes

import pytest
import torch

import sparse_moe_expert_router_amd as moe
from tests.test_around_abi import CODES, DW, DX, F32, NULL, P, RES, RSTD, SCALES, SHAPE, UNSUP, W, WS, X, Y, _bal, _bwd, _norm

VALID = P(12)


def at(p, n):
    return ctypes.c_void_p(p.value + n)


def test_norm_small_outputs_are_never_an_inputs_rows():
    """scales and rstd can have an input row's bytes (T values, or T groups, beside H): still another array."""
    sq = dict(T=256, H=256, xd=F32, rd=F32)
    for p in (X, RES):
        assert _norm(rstd=p, **sq) == SHAPE
    deep = dict(T=128, H=256, xd=F32, rd=F32)                       # 128 rows of 2 scales: 256 values
    for p in (X, RES):
        assert _norm(s=p, **deep) == SHAPE
    one = dict(T=1, H=256)
    for name in ("c", "s", "rstd"):
        for p in (X, RES):
            assert _norm(**{name: p}, **one) == SHAPE


def test_norm_backward_sums_are_never_an_inputs_rows():
    for p in (X, Y, RES, RSTD, W):
        assert _bwd(dw=p, T=1, yd=F32, sd=F32) == SHAPE and _bwd(dw=p) == SHAPE


GATES = dict(i=Y, g=CODES, dg=RSTD)


def test_balance_outputs_share_no_memory():
    E, T, k = 64, 4, 2
    inputs = dict(X=(X, 4 * T * E), W=(W, 4 * E), V=(VALID, T), Y=(Y, 4 * T * k), C=(CODES, 4 * T * k), R=(RSTD, 4 * T * k))
    for p, size in inputs.values():
        last = at(p, size - 4)
        assert _bal(loss=p, v=VALID, **GATES) == SHAPE and _bal(loss=last, v=VALID, **GATES) == SHAPE
        assert _bal(ps=p, v=VALID, **GATES) == SHAPE and _bal(ps=last, v=VALID, **GATES) == SHAPE
        assert _bal(ps=at(p, -4 * E + 4), v=VALID, **GATES) == SHAPE
        if p is not X:
            assert _bal(dl=p, v=VALID, **GATES) == SHAPE and _bal(dl=at(p, -4 * T * E + 4), v=VALID, **GATES) == SHAPE
    # each other
    assert _bal(ps=SCALES) == SHAPE and _bal(loss=at(SCALES, 4 * E - 4), ps=SCALES) == SHAPE
    assert _bal(loss=DX) == SHAPE and _bal(loss=at(DX, 4 * T * E - 4)) == SHAPE and _bal(ps=DX) == SHAPE
    # without tokens loss and prob_sum are written all the same, and the counts read
    assert _bal(T=0, loss=W) == SHAPE and _bal(T=0, ps=W) == SHAPE and _bal(T=0, ps=SCALES) == SHAPE


def test_counts_share_no_memory():
    c = lambda i=X, T=4, k=2, E=8, v=VALID, acc=0, n=Y: moe.lib().moe_expert_counts(i, T, k, E, v, acc, n, None)
    for acc in (0, 1):
        assert c(n=X, acc=acc) == SHAPE and c(n=at(X, 28), acc=acc) == SHAPE and c(n=at(X, -28), acc=acc) == SHAPE
        assert c(n=VALID, acc=acc) == SHAPE and c(n=at(VALID, -28), acc=acc) == SHAPE


def test_awq_rows_share_no_memory():
    def mm(x=X, ldx=256, q=W, z=Y, s=SCALES, M=4, N=64, K=256, g=32, dt=F32, y=DX, ldy=64):
        return moe.lib().moe_awq_matmul(x, ldx, q, z, s, M, N, K, g, dt, y, ldy, None, 0, None)
    for p, size in ((X, 2 * 4 * 256), (W, 4 * 256 * 8), (Y, 4 * 8 * 8), (SCALES, 2 * 8 * 64)):
        assert mm(y=p) == SHAPE and mm(y=at(p, size - 4)) == SHAPE and mm(y=at(p, -4 * 4 * 64 + 4)) == SHAPE


def test_awq_large_matrices_need_a_workspace_and_refuse_without():
    need = moe.lib().moe_awq_matmul_workspace_bytes(1, 8192, 8192, 128)
    assert need > 0
    mm = lambda ws, n: moe.lib().moe_awq_matmul(X, 8192, W, Y, SCALES, 1, 8192, 8192, 128, F32, DX, 8192, ws, n, None)
    assert mm(DW, need - 1) == WS and mm(None, need) == NULL and mm(at(DW, 8), need) == UNSUP


def test_a_workspace_of_another_device_is_refused():
    from sparse_moe_expert_router_amd import _lib
    with pytest.raises(moe.MoeError, match="workspace is on cpu"):
        _lib._scratch("call", moe.Workspace("cpu"), torch.device("meta"), 64)
    buf, n = _lib._scratch("call", None, torch.device("cpu"), 64)
    assert buf.device.type == "cpu" and n == 64
    assert _lib._scratch("call", moe.Workspace("cpu"), torch.device("meta"), 0) == (None, 0)
