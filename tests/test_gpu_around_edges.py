"""Edges of the operators around the layer: infinite scales beside a run's end, sums of squares near fp32's end."""
import pytest
import torch

import sparse_moe_expert_router_amd as moe
from tests import around_ref as R
from tests.test_gpu_around import BF, DEV, F32, _awq, _randn

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ 4-bit product: infinite scales

# K whose runs of 32 inputs (5, 6 and 9 a wave; 4 or 5 in a large matrix) end inside a step of four
@pytest.mark.parametrize("M", [1, 2, 4, 20])
@pytest.mark.parametrize("N,K,group", [(264, 640, 32), (264, 640, 64), (264, 640, 128), (512, 5152, 32), (8192, 4128, 32)])
def test_awq_infinite_scale(M, N, K, group):
    """The scale multiplies the sums of 32 inputs each.  So an infinite one gives, in its column, an infinity where its group's
    sums have one sign, NaN where they have both (inf - inf), and reaches no other column."""
    q, z, s = _awq(K, N, group, M + K)
    x = _randn(M, K, seed=M, dtype=BF)
    groups, parts = K // group, group // 32
    at = torch.arange(groups, device=DEV)
    col = (at * 13 + 1) % N
    assert len(set(col.tolist())) == groups
    s[at, col] = torch.where(at % 2 == 0, float("inf"), -float("inf")).half()
    d = (R.unpack(q) - R.unpack(z).repeat_interleave(group, 0))[:, col]
    sums = torch.stack([(x[:, 32 * i:32 * i + 32].double() @ d[32 * i:32 * i + 32, i // parts]) for i in range(K // 32)], 1)
    sums = sums.view(M, groups, parts)
    # a sum's own roundings: 72 U of at most 62 |x|, below 1e-2; nearer to 0 its sign is not known
    known = (sums.abs() > 1e-2).all(2)
    assert known.float().mean() > 0.98
    sign = torch.where(at % 2 == 0, 1.0, -1.0).double()[:, None] * torch.sign(sums)
    want = torch.where((sign > 0).all(2), float("inf"), torch.where((sign < 0).all(2), -float("inf"), float("nan")))
    for out in (moe.OUT_F32, moe.OUT_BF16):
        y = moe.awq_matmul(x, q, z, s, out_dtype=out)
        got = y[:, col].double()
        assert not torch.isfinite(got).any()
        assert ((got == want) | (got.isnan() & want.isnan()))[known].all()
        rest = torch.ones(N, dtype=torch.bool, device=DEV)
        rest[col] = False
        fine = s.clone()
        fine[at, col] = 0
        ref, lim = R.awq(x, q, z, fine)
        R.check_rows(y[:, rest], ref[:, rest], 0.0, lim[:, rest])


# ------------------------------------------------------------------ norm: where the sum of squares ends

@pytest.mark.parametrize("H", [8, 128, 640, 8192, 16384])
@pytest.mark.parametrize("dtype", [F32, BF])
def test_norm_up_to_the_largest_sum_of_squares(H, dtype):
    """A row of one magnitude: right while its squares' sum is below fp32's end (2^128), zeros beyond."""
    border = (2.0 ** 128 / H) ** 0.5
    x = torch.where(_randn(6, H, seed=H) > 0, 1.0, -1.0)
    x[0] *= border * 0.97
    x[1] *= border * 1.03
    x[2] *= border * 1e-3
    x[3] *= border * 10
    x = x.to(dtype)
    w = _randn(H, seed=1, scale=0.1)
    r = moe.add_rmsnorm(x, w, outputs=("y", "rstd"))
    fine = [0, 2, 4, 5]
    v, rstd = R.norm(x[fine], w, 1e-6, 1.0)
    R.check_rows(r.y[fine], v)
    assert ((r.rstd[fine].double() - rstd).abs() <= R.NORM_REL * rstd).all()
    assert (r.y[[1, 3]] == 0).all() and (r.rstd[[1, 3]] == 0).all()
    dy, dres = _randn(6, H, seed=2, dtype=dtype), _randn(6, H, seed=3, dtype=dtype)
    dx, _ = moe.add_rmsnorm_backward(dy, x, r.rstd, w, dres=dres)
    assert torch.equal(dx[[1, 3]], dres[[1, 3]])
