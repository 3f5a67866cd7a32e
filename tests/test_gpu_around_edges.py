"""Edges of the operators around the layer: infinite scales beside a run's end, sums of squares near fp32's end,
long sums over tokens, workspaces of exactly the stated size.  Bounds in units of U = 2^-24, half a step of fp32."""
import pytest
import torch

import sparse_moe_expert_router_amd as moe
from tests import around_ref as R
from tests.test_gpu_around import BF, DEV, F32, _awq, _gen, _randn, _routing

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


# ------------------------------------------------------------------ balance loss: long sums

def _teams(T, E, k):
    """The least number of teams that share T tokens; a team adds its tokens' probabilities one after another."""
    lanes = 16 if E <= 64 and k <= 16 else 32 if E <= 256 and k <= 32 else 64
    teams = 8 * 64 // lanes
    need = -(-T // teams)
    return teams * (1 if need <= 4 else min(need, 256 if E > 512 else 768))


def _sums(logits, counts, k, coef):
    """loss and prob_sum in 64 bits with their bounds, in pieces of rows.

    A probability's relative error, x = v - max: the difference's rounding, the product with log2 e and that constant's
    own (0.23 U) come to 2.25 |x| U in the exponent; the exponential, the sum over the experts (at most 16 in a lane, then
    6 steps), the reciprocal and the product below 48 U.  The sum's error is the probabilities' own mean."""
    T, E = logits.shape
    C = float(counts.sum())
    a = coef * E * k / C
    f = counts.double() / C - 1.0 / E
    zero = lambda: torch.zeros(E, dtype=torch.float64, device=DEV)
    S, lim, fp, flim = zero(), zero(), 0.0, 0.0
    for part in logits.split(50000):
        x = part.double()
        x = x - x.amax(1, keepdim=True)
        p = torch.softmax(x, 1)
        rel = (48.0 + 2.25 * x.abs()) * R.U
        err = p * (rel + (p * rel).sum(1, keepdim=True)) + 2.0 ** -126
        S += p.sum(0)
        lim += err.sum(0)
        fp += float((p @ f).sum())
        # f' to fp32 and the fused sums of f' p: 24 U of the magnitudes
        flim += float((err @ f.abs()).sum() + 24 * R.U * (p @ f.abs()).sum())
    # a team's tokens one after another, at most 32 teams of a workgroup, then at most 6 + 7 + 15 additions over workgroups
    lim += (-(-T // _teams(T, E, k)) + 60) * R.U * S
    return a * (fp + T / E), abs(a) * flim, S, lim


@pytest.mark.parametrize("T,E,k,dtype", [(40000, 1000, 5, F32), (40000, 1024, 8, BF), (30001, 516, 4, F32), (2_200_000, 1024, 2, BF),
                                         (300_000, 512, 10, F32), (500_000, 61, 6, BF)])
def test_balance_sums_over_many_tokens(T, E, k, dtype):
    logits = torch.empty((T, E), dtype=dtype, device=DEV)
    for i, part in enumerate(logits.split(200_000)):
        part.copy_(torch.randn(part.shape, generator=_gen(i), device=DEV) * 1.5 + _randn(E, seed=99))
    counts = torch.randint(1, 1000, (E,), generator=_gen(7), device=DEV, dtype=torch.int32)
    loss, prob_sum, d = moe.balance_loss(logits, counts, k, 0.01, want_dlogits=False)
    ref, lim, S, slim = _sums(logits, counts, k, 0.01)
    assert d is None
    assert ((prob_sum.double() - S).abs() <= slim + R.U * S).all(), float(((prob_sum.double() - S).abs() / slim).max())
    assert abs(float(loss) - ref) <= lim + 2 * R.U * abs(ref), (float(loss), ref, lim)


# ------------------------------------------------------------------ workspaces of exactly the stated size

def _guarded(n):
    buf = torch.full((n + 4096,), 0xA5, dtype=torch.uint8, device=DEV)
    return buf, lambda: bool((buf[n:] == 0xA5).all())


def _stream():
    return torch.cuda.current_stream().cuda_stream


@pytest.mark.parametrize("N,K", [(8192, 8192), (8192, 4128), (264, 8192), (4104, 8192)])
def test_awq_workspace_of_the_largest_number_of_rows(N, K):
    q, z, s = _awq(K, N, 32, 21)
    x = _randn(65, K, seed=22, dtype=BF)
    n = moe.lib().moe_awq_matmul_workspace_bytes(65, N, K, 32)
    assert n > 0
    ws, untouched = _guarded(n)
    for M in (65, 64, 48, 33, 32, 20, 17, 16, 5, 4, 3, 1):
        y = torch.empty((M, N), device=DEV)
        assert moe.lib().moe_awq_matmul(x.data_ptr(), K, q.data_ptr(), z.data_ptr(), s.data_ptr(), M, N, K, 32, moe.OUT_F32, y.data_ptr(), N,
                                        ws.data_ptr(), n, _stream()) == 0
        ref, lim = R.awq(x[:M], q, z, s)
        R.check_rows(y, ref, 0.0, lim)
        assert untouched()


@pytest.mark.parametrize("H", [72, 264, 2560, 8200])
def test_norm_backward_workspace_of_the_most_rows(H):
    most = 4100
    s, dy, w = _randn(most, H, seed=23), _randn(most, H, seed=24), _randn(H, seed=25, scale=0.1)
    rstd = moe.add_rmsnorm(s, w, outputs=("y", "rstd")).rstd
    n = moe.workspace_bytes(moe.OP_ADD_RMSNORM_BACKWARD, most, 1, 1, H)
    ws, untouched = _guarded(n)
    for T in (4100, 769, 768, 1):
        dx, dw = torch.empty((T, H), device=DEV), torch.empty(H, device=DEV)
        assert moe.lib().moe_add_rmsnorm_backward(dy.data_ptr(), moe.OUT_F32, H, s.data_ptr(), H, moe.OUT_F32, rstd.data_ptr(), w.data_ptr(),
                                                  moe.OUT_F32, 1.0, None, 0, T, H, dx.data_ptr(), H, dw.data_ptr(), ws.data_ptr(), n, _stream()) == 0
        rx, lx, rw, lw = R.norm_backward(dy[:T], s[:T], rstd[:T], w, 1.0)
        R.check_rows(dx, rx, 0.0, lx)
        assert ((dw.double() - rw).abs() <= lw).all() and untouched()


@pytest.mark.parametrize("E,k", [(61, 6), (200, 8), (512, 10), (1000, 4)])
def test_balance_workspace_of_the_most_tokens(E, k):
    most = 20000
    logits, idx, _ = _routing(most, E, k, F32, 26)
    n = moe.workspace_bytes(moe.OP_BALANCE_LOSS, most, k, E, 0)
    ws, untouched = _guarded(n)
    counts = moe.expert_counts(idx, E)
    for T in (20000, 2000, 65, 1):
        loss, prob_sum, d = torch.empty(1, device=DEV), torch.empty(E, device=DEV), torch.empty((T, E), device=DEV)
        assert moe.lib().moe_balance_loss(logits.data_ptr(), moe.OUT_F32, E, T, E, k, counts.data_ptr(), 0.01, None, None, None, None,
                                          loss.data_ptr(), prob_sum.data_ptr(), d.data_ptr(), moe.OUT_F32, E, ws.data_ptr(), n, _stream()) == 0
        want = moe.balance_loss(logits[:T], counts, k, 0.01)
        assert all(torch.equal(a, b) for a, b in zip((loss, prob_sum, d), want)) and untouched()


def test_workspaces_of_another_device_are_refused():
    cpu = moe.Workspace("cpu")
    x, w = _randn(8, 64, seed=27), _randn(64, seed=28)
    rstd = moe.add_rmsnorm(x, w, outputs=("y", "rstd")).rstd
    counts = torch.ones(64, dtype=torch.int32, device=DEV)
    q, z, s = _awq(8192, 8192, 128, 29)
    for call in (lambda: moe.add_rmsnorm_backward(x, x, rstd, w, ws=cpu), lambda: moe.balance_loss(x, counts, 2, 0.01, ws=cpu),
                 lambda: moe.awq_matmul(_randn(1, 8192, seed=30, dtype=BF), q, z, s, ws=cpu)):
        with pytest.raises(moe.MoeError, match="workspace is on cpu"):
            call()
