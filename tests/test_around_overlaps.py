"""Memory that the operators around the layer refuse to share between an output and anything else, before any HIP call (the
pointers are never dereferenced)."""
from tests.test_around_abi import F32, RES, RSTD, SHAPE, W, X, Y, _bwd, _norm


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
