"""The operators around the layer on the GPU (add-and-norm and its gradients, counts, balance loss, the 4-bit product) against
their 64-bit forms (around_ref), and a run of them together with the layer."""
import itertools

import pytest
import torch

import sparse_moe_expert_router_amd as moe
import workloads
from tests import around_ref as R

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _randn(*shape, seed, dtype=F32, scale=1.0):
    return (torch.randn(shape, generator=_gen(seed), device=DEV) * scale).to(dtype)


# ------------------------------------------------------------------ add and norm

NORM_SHAPES = [(1, 8), (1, 16), (3, 24), (1, 2560), (2, 144), (5, 520), (7, 688), (33, 1024), (64, 2560), (300, 4104), (17, 8192), (9, 8208),
               (5, 16384), (4097, 640), (20000, 128), (9000, 520), (8193, 2560), (40, 256), (15, 264)]


def _check_norm(x, w, res, r, eps, offset):
    s = x if res is None else (x.float() + res.float()).to(res.dtype)
    if res is not None:
        assert torch.equal(r.residual, s)
    v, rstd = R.norm(s, w, eps, offset)
    if r.y is not None:
        R.check_rows(r.y, v)
    if r.codes is not None:
        R.check_fp8(r.codes, r.scales, v)
    if r.rstd is not None:
        assert ((r.rstd.double() - rstd).abs() <= R.NORM_REL * rstd).all()


@pytest.mark.parametrize("T,H", NORM_SHAPES)
@pytest.mark.parametrize("xd,rd", [(BF, None), (BF, BF), (BF, F32), (F32, BF), (F32, F32)])
def test_norm(T, H, xd, rd):
    x = _randn(T, H, seed=T, dtype=xd, scale=3.0)
    x[:, :4] *= 30
    res = _randn(T, H, seed=H, dtype=rd, scale=5.0) if rd else None
    w = _randn(H, seed=1, dtype=xd, scale=0.2)
    offset = 1.0 if T % 2 else 0.0
    outputs = ("y", "fp8", "rstd") if H % 16 == 0 else ("y", "rstd")
    r = moe.add_rmsnorm(x, w, res, eps=1e-5, gain_offset=offset, outputs=outputs)
    _check_norm(x, w, res, r, 1e-5, offset)
    only = moe.add_rmsnorm(x, w, res, eps=1e-5, gain_offset=offset, outputs=("fp8",) if H % 16 == 0 else None)
    for name in ("y", "codes", "scales", "residual"):
        got = getattr(only, name)
        if got is not None:
            assert torch.equal(got, getattr(r, name)), name
    assert (only.y is None) == (H % 16 == 0)


def test_norm_codes_are_the_quantisers_of_its_own_values():
    """With gain 1 and rows whose r is a power of two v is exact in bf16: codes equal fp8_quantize(y)."""
    x = torch.where(_randn(64, 640, seed=3) > 0, 0.5, -0.5).to(BF)
    r = moe.add_rmsnorm(x, torch.ones(640, device=DEV), gain_offset=0.0, eps=1e-30, outputs=("y", "fp8"))
    assert torch.equal(r.y.float(), 2 * x.float())
    codes, scales = moe.fp8_quantize(r.y)
    assert torch.equal(codes, r.codes) and torch.equal(scales, r.scales)


def test_norm_strided_and_in_place():
    T, H = 37, 688
    wide = _randn(T, 3 * H + 16, seed=4, dtype=BF)
    x, y = wide[:, 8:8 + H], wide[:, 16 + H:16 + 2 * H]          # interleaved columns of one buffer
    big = _randn(T + 2, H + 24, seed=5)
    res = big[1:T + 1, 8:8 + H]
    w = _randn(H, seed=6, scale=0.1)
    x0, res0, big0, wide0 = x.clone(), res.clone(), big.clone(), wide.clone()
    r = moe.add_rmsnorm(x, w, res, residual_out=res, y=y, outputs=("rstd",))
    _check_norm(x0, w, res0, moe.NormResult(r.y, r.residual, None, None, r.rstd), 1e-6, 1.0)
    assert r.residual.data_ptr() == res.data_ptr() and torch.equal(x, x0)
    big0[1:T + 1, 8:8 + H] = res
    wide0[:, 16 + H:16 + 2 * H] = y
    assert torch.equal(big, big0) and torch.equal(wide, wide0)     # nothing else is written
    want = moe.add_rmsnorm(x0, w).y
    got = moe.add_rmsnorm(x, w, y=x).y                              # over its own input
    assert torch.equal(got, want) and torch.equal(x, want)


def test_norm_special_rows():
    H = 640
    x = _randn(8, H, seed=7)
    x[0] = 0
    x[1, 3] = float("inf")
    x[2, 200] = float("nan")
    x[3] = -0.0
    x[4] = 1e-30
    x[5] = 1e15
    x[6] = 0
    x[6, 5] = -1e18
    w = torch.zeros(H, device=DEV)
    r = moe.add_rmsnorm(x, w, outputs=("y", "fp8", "rstd"))
    ok = [0, 3, 4, 5, 6, 7]
    _check_norm(x[ok], w, None, moe.NormResult(r.y[ok], None, r.codes[ok], r.scales[ok], r.rstd[ok]), 1e-6, 1.0)
    assert (r.y[0] == 0).all() and torch.isnan(r.y[1, 3]) and (r.y[1, :3] == 0).all() and torch.isnan(r.y[2]).all()
    assert torch.isnan(r.scales[2]).all()


def test_norm_no_rows():
    e = torch.empty((0, 64), device=DEV)
    w = torch.ones(64, device=DEV)
    r = moe.add_rmsnorm(e, w, e, outputs=("y", "fp8", "rstd"))
    assert r.y.shape == (0, 64) and r.scales.shape == (0, 1) and r.rstd.shape == (0,)
    dw = torch.full((64,), 7.0, device=DEV)
    dx, got = moe.add_rmsnorm_backward(e, e, e[:, 0], w, dw=dw)
    assert dx.shape == (0, 64) and (got == 0).all()


def test_norm_offsets_past_32_bits():
    T, H = 300_000, 8192                       # 2.4e9 values
    x = torch.empty((T, H), dtype=BF, device=DEV)
    x[-3:] = _randn(3, H, seed=8, dtype=BF)
    x[:-3] = 1.0
    w = _randn(H, seed=9, dtype=BF, scale=0.1)
    y = x                                       # over the input
    last = x[-3:].clone()
    r = moe.add_rmsnorm(x, w, y=y, outputs=("rstd",))
    R.check_rows(r.y[-3:], R.norm(last, w, 1e-6, 1.0)[0])
    assert torch.equal(r.y[0], r.y[T // 2]) and torch.equal(r.y[0], r.y[-4])


# ------------------------------------------------------------------ gradients of the norm

@pytest.mark.parametrize("T,H", NORM_SHAPES)
@pytest.mark.parametrize("sd,yd,dres", [(BF, BF, True), (BF, BF, False), (F32, F32, True), (F32, BF, True), (BF, F32, False)])
def test_norm_backward(T, H, sd, yd, dres):
    s = _randn(T, H, seed=T, dtype=sd, scale=3.0)
    w = _randn(H, seed=1, dtype=yd, scale=0.2)
    offset = 1.0 if T % 2 else 0.0
    rstd = moe.add_rmsnorm(s, w, gain_offset=offset, outputs=("y", "rstd")).rstd
    dy = _randn(T, H, seed=2, dtype=yd, scale=1e-3)
    dr = _randn(T, H, seed=3, dtype=sd, scale=1e-3) if dres else None
    dx, dw = moe.add_rmsnorm_backward(dy, s, rstd, w, gain_offset=offset, dres=dr)
    rx, lx, rw, lw = R.norm_backward(dy, s, rstd, w, offset, dr)
    assert dx.dtype == sd and dw.dtype == F32
    R.check_rows(dx, rx, 0.0, lx)
    assert ((dw.double() - rw).abs() <= lw).all()
    assert (dw.double() - rw).norm() <= 2.0 ** -18 * (dy.double() * s.double() * rstd.double()[:, None]).norm(dim=0).norm()
    again = moe.add_rmsnorm_backward(dy, s, rstd, w, gain_offset=offset, dres=dr)
    assert torch.equal(dx, again[0]) and torch.equal(dw, again[1])


@pytest.mark.parametrize("T,H", [(768, 72), (769, 72), (767, 256), (700, 264), (768, 1000), (769, 1000), (513, 8200), (130, 16384), (65, 40)])
@pytest.mark.parametrize("sd,yd", [(BF, BF), (F32, F32), (BF, F32), (F32, BF)])
def test_norm_backward_of_few_and_many_rows(T, H, sd, yd):
    s, dy = _randn(T, H + 8, seed=T, dtype=sd, scale=2.0)[:, 8:], _randn(T, H + 16, seed=2, dtype=yd, scale=1e-2)[:, :H]
    w = _randn(H, seed=1, dtype=sd, scale=0.2)
    rstd = moe.add_rmsnorm(s, w, outputs=("y", "rstd")).rstd
    rx, lx, rw, lw = R.norm_backward(dy, s, rstd, w, 1.0, None)
    dx, dw = moe.add_rmsnorm_backward(dy, s, rstd, w)
    R.check_rows(dx, rx, 0.0, lx)
    assert ((dw.double() - rw).abs() <= lw).all()
    # in place the sums may be taken in another order, and are as good
    on = s.clone()
    dx2, dw2 = moe.add_rmsnorm_backward(dy, on, rstd, w, dx=on)
    assert dx2 is on and torch.equal(dx2, dx)
    assert ((dw2.double() - rw).abs() <= lw).all()


def test_norm_backward_in_place_and_strided():
    T, H = 29, 1288
    wide = _randn(T, 2 * H + 8, seed=11, dtype=BF)
    s, dy = wide[:, :H], wide[:, H + 8:]
    w = _randn(H, seed=12, dtype=BF, scale=0.1)
    rstd = moe.add_rmsnorm(s, w, outputs=("y", "rstd")).rstd
    dres = _randn(T, H, seed=13, dtype=BF)
    want = moe.add_rmsnorm_backward(dy, s, rstd, w, dres=dres)
    for out in ("dres", "dy", "s"):
        a = {"dy": dy.clone(), "s": s.clone(), "dres": dres.clone()}
        dx, dw = moe.add_rmsnorm_backward(a["dy"], a["s"], rstd, w, dres=a["dres"], dx=a[out])
        assert dx.data_ptr() == a[out].data_ptr() and torch.equal(dx, want[0]) and torch.equal(dw, want[1])


def test_norm_backward_against_differences():
    T, H = 6, 64
    x, w = _randn(T, H, seed=14), _randn(H, seed=15, scale=0.1)
    dy = _randn(T, H, seed=16)
    rstd = moe.add_rmsnorm(x, w, outputs=("y", "rstd")).rstd
    dx, dw = moe.add_rmsnorm_backward(dy, x, rstd, w)
    f = lambda x, w: (R.norm(x, w, 1e-6, 1.0)[0] * dy.double()).sum()
    h = 1e-5
    for t, i in itertools.product((0, 5), (0, 31, 63)):
        e = torch.zeros((T, H), dtype=torch.float64, device=DEV)
        e[t, i] = h
        assert abs((f(x.double() + e, w) - f(x.double() - e, w)) / (2 * h) - dx[t, i]) < 1e-4
        assert abs((f(x, w.double() + e[t]) - f(x, w.double() - e[t])) / (2 * h) - dw[i]) < 1e-4


# ------------------------------------------------------------------ counts

@pytest.mark.parametrize("T,k,E", [(1, 1, 1), (1, 10, 512), (16, 10, 512), (300, 8, 60), (4096, 1, 1024), (409, 10, 512), (410, 10, 512),
                                   (8191, 6, 61), (32768, 10, 512), (150000, 3, 7)])
@pytest.mark.parametrize("masked", [False, True])
def test_counts(T, k, E, masked):
    idx = torch.randint(0, E, (T, k), generator=_gen(T), device=DEV, dtype=torch.int32)
    idx[0, 0] = -1
    if T > 3:
        idx[3, k - 1] = E
    valid = torch.rand(T, generator=_gen(1), device=DEV) < 0.6 if masked else None
    want = R.counts(idx, E, valid).int()
    counts = torch.full((E,), 12345, dtype=torch.int32, device=DEV)
    assert torch.equal(moe.expert_counts(idx, E, token_valid=valid, counts=counts), want)
    moe.expert_counts(idx, E, token_valid=valid.to(torch.uint8) if masked else None, counts=counts, accumulate=True)
    assert torch.equal(counts, 2 * want)


@pytest.mark.parametrize("T,k,E", [(128, 8, 100), (1025, 1, 15), (1025, 1, 16), (1000, 5, 17), (3000, 3, 1023), (24576, 2, 8), (24577, 2, 8),
                                   (8192, 6, 61), (8193, 6, 61)])
def test_counts_of_few_and_many_pairs(T, k, E):
    idx = torch.randint(-1, E + 1, (T, k), generator=_gen(T), device=DEV, dtype=torch.int32)
    valid = torch.rand(T, generator=_gen(1), device=DEV) < 0.8
    for v in (None, valid):
        want = R.counts(idx, E, v).int()
        wide = torch.full((E + 2,), 7, dtype=torch.int32, device=DEV)
        counts = wide[1:E + 1]
        assert torch.equal(moe.expert_counts(idx, E, token_valid=v, counts=counts), want)
        for i in (2, 3):
            moe.expert_counts(idx, E, token_valid=v, counts=counts, accumulate=True)
            assert torch.equal(counts, i * want)
        assert wide[0] == 7 and wide[-1] == 7


def test_counts_added_from_two_streams():
    E, parts = 61, [(8000, 6), (9000, 6), (100, 3), (20000, 2)]
    idx = [torch.randint(0, E, p, generator=_gen(i), device=DEV, dtype=torch.int32) for i, p in enumerate(parts)]
    want = sum(R.counts(i, E, None) for i in idx).int() * 20
    counts = torch.zeros(E, dtype=torch.int32, device=DEV)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(20):
        for j, i in enumerate(idx):
            with torch.cuda.stream(streams[j % 2]):
                moe.expert_counts(i, E, counts=counts, accumulate=True)
    torch.cuda.synchronize()
    assert torch.equal(counts, want)


def test_counts_are_the_permutations_groups():
    x, w = _randn(777, 256, seed=1, dtype=BF), _randn(64, 256, seed=2, dtype=BF, scale=0.05)
    idx, _, _, off, _, _ = moe.route_permute(x, w, 4)
    assert torch.equal(moe.expert_counts(idx, 64), off[1:] - off[:-1])


def test_counts_no_tokens():
    e = torch.empty((0, 2), dtype=torch.int32, device=DEV)
    c = torch.full((8,), 3, dtype=torch.int32, device=DEV)
    assert (moe.expert_counts(e, 8, counts=c, accumulate=True) == 3).all() and (moe.expert_counts(e, 8, counts=c) == 0).all()


# ------------------------------------------------------------------ balance loss

BALANCE = [(1, 1, 1), (1, 512, 10), (16, 512, 10), (5, 3, 2), (7, 8, 8), (33, 16, 4), (64, 60, 6), (301, 61, 16), (100, 64, 16), (50, 64, 17),
           (129, 100, 10), (77, 128, 64), (40, 129, 8), (500, 256, 8), (90, 260, 4), (1000, 384, 10), (63, 511, 10), (4099, 512, 10),
           (30, 520, 10), (21, 1000, 5), (19, 1023, 64), (11, 1024, 1), (70000, 8, 2), (20000, 64, 6), (40000, 132, 4), (33, 127, 9), (20, 63, 20), (200, 300, 40), (6, 65, 3)]


def _routing(T, E, k, dtype, seed):
    logits = (_randn(T, E, seed=seed, scale=1.5) + _randn(E, seed=seed + 1)).to(dtype)
    top, idx = torch.sort(logits.float(), dim=1, descending=True, stable=True)
    return logits, idx[:, :k].int().contiguous(), torch.softmax(top[:, :k], 1)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("T,E,k", BALANCE)
def test_balance(T, E, k, dtype):
    logits, idx, gate = _routing(T, E, k, dtype, T + E)
    counts = moe.expert_counts(idx, E)
    got = moe.balance_loss(logits, counts, k, 0.01)
    R.check_balance(got, R.balance(logits, counts, k, 0.01), dtype)
    valid = torch.rand(T, generator=_gen(5), device=DEV) < 0.7
    counts = moe.expert_counts(idx, E, token_valid=valid)
    dgate = _randn(T, k, seed=6, scale=1e-2)
    ref = R.balance(logits, counts, k, 0.01, valid, idx, gate, dgate)
    got = moe.balance_loss(logits, counts, k, 0.01, token_valid=valid, topk_idx=idx, gate=gate, dgate=dgate)
    R.check_balance(got, ref, dtype)
    assert (got[2][~valid] == 0).all()
    again = moe.balance_loss(logits, counts, k, 0.01, token_valid=valid, topk_idx=idx, gate=gate, dgate=dgate)
    assert all(torch.equal(a, b) for a, b in zip(got, again))
    loss, prob_sum, none = moe.balance_loss(logits, counts, k, 0.01, token_valid=valid, want_dlogits=False)
    assert none is None and torch.equal(loss, got[0]) and torch.equal(prob_sum, got[1])


@pytest.mark.parametrize("E", [12, 61, 512, 1001])
def test_balance_masked_experts_and_empty_rows(E):
    T, k = 40, 3
    logits, idx, gate = _routing(T, E, k, F32, E)
    keep = torch.rand((T, E), generator=_gen(1), device=DEV) < 0.5
    keep.scatter_(1, idx.long(), True)
    logits[~keep] = -float("inf")
    logits[5], logits[6] = -float("inf"), torch.finfo(F32).min
    logits[7] = torch.where(keep[7], logits[7], torch.finfo(F32).min)
    logits[8] = 3e38
    logits[8, 0] = -3e38
    valid = torch.ones(T, dtype=torch.uint8, device=DEV)
    valid[9] = 0
    logits[9] = float("nan")
    idx[9], gate[9] = -7, float("nan")
    counts = moe.expert_counts(idx, E, token_valid=valid)
    dgate = _randn(T, k, seed=2)
    dgate[9] = float("inf")
    got = moe.balance_loss(logits, counts, k, 0.5, token_valid=valid, topk_idx=idx, gate=gate, dgate=dgate)
    assert torch.isfinite(got[2]).all() and torch.isfinite(got[0]).all()
    gate[9], dgate[9] = 0, 0
    R.check_balance(got, R.balance(logits, counts, k, 0.5, valid, idx, gate, dgate), F32)
    plain = moe.balance_loss(logits, counts, k, 0.5, token_valid=valid)[2]
    assert (plain[5] == 0).all() and (plain[9] == 0).all() and (plain[~keep & (logits == -float("inf"))] == 0).all()


def test_balance_nan_stays_in_its_row():
    logits, idx, _ = _routing(9, 64, 4, F32, 1)
    counts = moe.expert_counts(idx, 64)
    logits[2, 5], logits[4, 63] = float("nan"), float("inf")
    loss, prob_sum, d = moe.balance_loss(logits, counts, 4, 0.01)
    bad = torch.zeros(9, dtype=torch.bool, device=DEV)
    bad[[2, 4]] = True
    assert torch.isnan(d[bad]).any(1).all() and torch.isfinite(d[~bad]).all() and torch.isnan(loss).all()


@pytest.mark.parametrize("E,k", [(8, 4), (64, 16), (512, 12)])
def test_balance_same_expert_twice_and_foreign_ids(E, k):
    T = 50
    logits, idx, gate = _routing(T, E, k, F32, 3)
    idx[3] = idx[3, 0]                       # all slots one expert
    idx[4, 1] = idx[4, 0]
    idx[5, 2], idx[5, 0] = E, -2 ** 31
    idx[6, 1], idx[6, 3] = idx[6, 2], idx[6, 0]
    counts = moe.expert_counts(idx, E)
    dgate = _randn(T, k, seed=4)
    args = dict(topk_idx=idx, gate=gate, dgate=dgate)
    got = moe.balance_loss(logits, counts, k, 0.01, **args)
    R.check_balance(got, R.balance(logits, counts, k, 0.01, None, idx, gate, dgate), F32)
    assert all(torch.equal(a, b) for a, b in zip(got, moe.balance_loss(logits, counts, k, 0.01, **args)))


@pytest.mark.parametrize("E,k", [(65, 3), (100, 16), (128, 17), (130, 32), (200, 32), (200, 33), (255, 5), (256, 10)])
def test_balance_of_middle_widths(E, k):
    for T in (1, 15, 65, 3001):
        test_balance(T, E, k, F32)
        test_balance(T, E, k, BF)
    test_balance_masked_experts_and_empty_rows(E)
    test_balance_same_expert_twice_and_foreign_ids(E, max(k, 4))


def test_balance_even_load_has_no_gradient():
    T, E = 96, 12
    idx = (torch.arange(T, device=DEV, dtype=torch.int32) % E)[:, None].contiguous()
    logits = _randn(T, E, seed=5)
    loss, _, d = moe.balance_loss(logits, moe.expert_counts(idx, E), 1, 0.25)
    assert (d == 0).all() and abs(float(loss) - 0.25) < 1e-6


def test_balance_no_tokens_and_no_counts():
    c = torch.zeros(8, dtype=torch.int32, device=DEV)
    loss, prob_sum, d = moe.balance_loss(torch.empty((0, 8), device=DEV), c, 2, 0.01)
    assert float(loss) == 0 and (prob_sum == 0).all() and d.shape == (0, 8)
    logits = _randn(5, 8, seed=1)
    loss, prob_sum, d = moe.balance_loss(logits, c, 2, 0.01)
    assert float(loss) == 0 and (d == 0).all() and abs(float(prob_sum.sum()) - 5) < 1e-5
    valid = torch.zeros(5, dtype=torch.uint8, device=DEV)
    loss, prob_sum, d = moe.balance_loss(logits, c + 1, 2, 0.01, token_valid=valid)
    assert float(loss) == 0 and (prob_sum == 0).all() and (d == 0).all()


@pytest.mark.parametrize("E", [60, 62, 512])
def test_balance_strided_in_place_and_other_type(E):
    T, k = 45, 4
    logits, idx, gate = _routing(T, E, k, F32, 8)
    counts = moe.expert_counts(idx, E)
    dgate = _randn(T, k, seed=9)
    args = dict(topk_idx=idx, gate=gate, dgate=dgate)
    want = moe.balance_loss(logits, counts, k, 0.01, **args)
    ref = R.balance(logits, counts, k, 0.01, None, idx, gate, dgate)
    for shift in (0, 1, 4):
        wide = torch.full((T, E + 9), 5.0, device=DEV)
        out = torch.full((T, E + 7), 5.0, dtype=BF, device=DEV)
        wide[:, shift:shift + E] = logits
        view, o = wide[:, shift:shift + E], out[:, 2:2 + E]
        got = moe.balance_loss(view, counts, k, 0.01, dlogits=o, **args)
        R.check_balance(got, ref, BF)
        assert (out[:, :2] == 5).all() and (out[:, 2 + E:] == 5).all()
        got = moe.balance_loss(view, counts, k, 0.01, dlogits=view, **args)
        R.check_balance(got, ref, F32)
        assert (wide[:, :shift] == 5).all() and (wide[:, shift + E:] == 5).all()
    inplace = logits.clone()
    got = moe.balance_loss(inplace, counts, k, 0.01, dlogits=inplace, **args)
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_balance_against_differences():
    T, E, k, coef = 5, 40, 3, 0.7
    logits, idx, gate = _routing(T, E, k, F32, 10)
    counts = moe.expert_counts(idx, E)
    dgate = _randn(T, k, seed=11)
    d = moe.balance_loss(logits, counts, k, coef, topk_idx=idx, gate=gate, dgate=dgate)[2]

    def f(z):
        g = torch.softmax(z.gather(1, idx.long()), 1)
        p = torch.softmax(z, 1).sum(0)
        return coef * E * k / counts.sum() * (counts.double() / counts.sum() * p).sum() + (g * dgate.double()).sum()
    for t, e in ((0, 0), (1, int(idx[1, 0])), (4, int(idx[4, 2])), (3, 39)):
        step = torch.zeros((T, E), dtype=torch.float64, device=DEV)
        step[t, e] = 1e-5
        assert abs((f(logits.double() + step) - f(logits.double() - step)) / 2e-5 - d[t, e]) < 1e-5


def test_balance_shares_of_a_larger_batch():
    T, E, k = 600, 128, 4
    logits, idx, _ = _routing(T, E, k, F32, 12)
    counts = moe.expert_counts(idx[:200], E)
    moe.expert_counts(idx[200:], E, counts=counts, accumulate=True)
    whole = moe.balance_loss(logits, counts, k, 0.1)
    parts = [moe.balance_loss(logits[:200], counts, k, 0.1), moe.balance_loss(logits[200:], counts, k, 0.1)]
    assert torch.equal(torch.cat([p[2] for p in parts]), whole[2])
    assert abs(float(parts[0][0] + parts[1][0] - whole[0])) <= 4 * R.U * float(whole[0])


def test_balance_offsets_past_32_bits():
    T, E, k = 2_200_000, 1024, 2               # 2.25e9 logits
    logits = torch.zeros((T, E), dtype=BF, device=DEV)
    logits[-5:] = _randn(5, E, seed=13, dtype=BF)
    idx = torch.zeros((T, k), dtype=torch.int32, device=DEV)
    idx[:, 1] = 1
    counts = moe.expert_counts(idx, E)
    last = logits[-5:].clone()
    d = moe.balance_loss(logits, counts, k, 0.01, dlogits=logits)[2]
    ref = R.balance(last, counts, k, 0.01)
    R.check_rows(d[-5:], ref["dlogits"], 2 * R.U, ref["lim_dlogits"] + 2.0 ** -126)
    assert torch.equal(d[0], d[T // 2]) and torch.equal(d[0], d[-6])


# ------------------------------------------------------------------ 4-bit product

def _awq(K, N, group, seed):
    g = _gen(seed)
    words = lambda *s: torch.randint(-2 ** 31, 2 ** 31, s, generator=g, device=DEV, dtype=torch.int64).to(torch.int32)
    scales = (torch.randn((K // group, N), generator=g, device=DEV) * 0.01).half()
    return words(K, N // 8), words(K // group, N // 8), scales


def _check_awq(y, x, q, z, s):
    ref, lim = R.awq(x, q, z, s)
    R.check_rows(y, ref, 0.0, lim)
    # the bound is for errors of one sign; with random ones the whole is off by far less
    half = R.HALF[y.dtype] if y.dtype == BF else 2.0 ** -18
    assert (y.double() - ref).norm() <= half * ref.norm()


AWQ = [(1, 8, 32), (1, 128, 64), (3, 136, 96), (16, 1000, 1312), (1, 2560, 2560), (5, 640, 2560), (17, 264, 640), (32, 520, 1024),
       (33, 256, 288), (64, 2560, 640), (65, 384, 320), (130, 72, 4096), (2, 24, 16384), (1, 8192, 2048), (16, 4096, 8192), (7, 16, 30720 // 2),
       # the large matrices' forms: pairs of words (N % 16 == 0) and single ones, split and not, every number of rows
       (1, 8192, 4096), (1, 4112, 8192), (2, 8200, 8192), (4, 16384, 2048), (3, 65536, 512), (5, 8192, 4352), (17, 4096, 8320),
       (40, 8208, 4224), (33, 4104, 8192),
       # wide and shallow
       (1, 20000, 64), (9, 20000, 96), (40, 16392, 64), (1, 10000, 128), (4, 10000, 160), (20, 10000, 128)]


@pytest.mark.parametrize("out", [BF, F32])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("M,N,K", AWQ)
def test_awq(M, N, K, group, out):
    K = -(-K // group) * group
    q, z, s = _awq(K, N, group, M + N + K)
    x = _randn(M, K, seed=M, dtype=BF)
    y = moe.awq_matmul(x, q, z, s, out_dtype=moe.OUT_F32 if out == F32 else None)
    _check_awq(y, x, q, z, s)
    assert torch.equal(y, moe.awq_matmul(x, q, z, s, out_dtype=moe.OUT_F32 if out == F32 else None))


@pytest.mark.parametrize("M", [1, 9, 40])
def test_awq_exact_on_whole_numbers(M):
    """Small whole numbers and scales that are powers of two: every sum is exact."""
    K, N = 640, 264
    q, z, _ = _awq(K, N, 32, 1)
    s = torch.exp2(torch.randint(-3, 3, (K // 32, N), generator=_gen(2), device=DEV).float()).half()
    x = torch.randint(-8, 9, (M, K), generator=_gen(3), device=DEV).to(BF)
    assert torch.equal(moe.awq_matmul(x, q, z, s, out_dtype=moe.OUT_F32).double(), R.awq(x, q, z, s)[0])


def test_awq_strided_and_untouched_surroundings():
    M, N, K = 11, 264, 320
    q, z, s = _awq(K, N, 64, 4)
    big = torch.full((M + 2, K + 24), float("nan"), dtype=BF, device=DEV)
    x = big[1:M + 1, 8:8 + K]
    x.copy_(_randn(M, K, seed=5))
    out = torch.full((M + 2, N + 5), 9.0, dtype=BF, device=DEV)
    y = out[1:M + 1, 3:3 + N]
    moe.awq_matmul(x, q, z, s, y=y)
    _check_awq(y, x, q, z, s)
    assert (out[0] == 9).all() and (out[-1] == 9).all() and (out[:, :3] == 9).all() and (out[:, 3 + N:] == 9).all()


@pytest.mark.parametrize("M", [1, 3, 12, 40])
def test_awq_codes_at_any_word(M):
    """Codes and zeros that begin at an odd word: the same sums as from aligned ones, in both cuts of the columns."""
    N, K = 8192, 4096
    q, z, s = _awq(K, N, 32, 11)
    x = _randn(M, K, seed=12, dtype=BF)
    shift = lambda t: torch.cat([t.new_zeros(1), t.reshape(-1)])[1:].view(t.shape)
    for a, b in ((shift(q), z), (q, shift(z)), (shift(q), shift(z))):
        assert a.data_ptr() % 8 or b.data_ptr() % 8
        _check_awq(moe.awq_matmul(x, a, b, s, out_dtype=moe.OUT_F32), x, q, z, s)


def test_awq_one_workspace_for_every_number_of_rows():
    N, K = 8192, 8192
    q, z, s = _awq(K, N, 128, 13)
    ws = moe.Workspace(DEV)
    x = _randn(65, K, seed=14, dtype=BF)
    moe.awq_matmul(x, q, z, s, ws=ws)
    buf = ws.buf
    for M in (1, 4, 16, 17, 32, 33, 64):
        _check_awq(moe.awq_matmul(x[:M], q, z, s, ws=ws), x[:M], q, z, s)
    assert ws.buf is buf or ws.buf.numel() > buf.numel()


@pytest.mark.parametrize("M", [2, 20, 70])
def test_awq_nan_stays_in_its_row_and_column(M):
    q, z, s = _awq(8192, 264, 32, 6)
    x = _randn(M, 8192, seed=7, dtype=BF)
    x[1, 5000] = float("inf")
    s[3, 17] = float("nan")
    y = moe.awq_matmul(x, q, z, s)
    bad = torch.zeros((M, 264), dtype=torch.bool, device=DEV)
    bad[1], bad[:, 17] = True, True
    assert torch.equal(~torch.isfinite(y), bad)


def test_awq_no_rows():
    q, z, s = _awq(64, 64, 32, 8)
    assert moe.awq_matmul(torch.empty((0, 64), dtype=BF, device=DEV), q, z, s).shape == (0, 64)


def test_awq_codes_past_32_bits():
    K, N, M = 131072, 65664, 3                  # 4.3e9 bytes of codes
    g = _gen(9)
    words = lambda *s: torch.randint(-2 ** 31, 2 ** 31, s, generator=g, device=DEV, dtype=torch.int64).to(torch.int32)
    q, z = words(K, N // 8), words(K // 128, N // 8)
    s = (torch.rand((K // 128, N), generator=g, device=DEV) * 0.01).half()
    x = _randn(M, K, seed=10, dtype=BF)
    y = moe.awq_matmul(x, q, z, s, out_dtype=moe.OUT_F32)
    for w in (0, 4100, N // 8 - 1):
        part = [t[:, w:w + 1].contiguous() for t in (q, z)] + [s[:, 8 * w:8 * w + 8].contiguous()]
        ref, lim = R.awq(x, *part)
        R.check_rows(y[:, 8 * w:8 * w + 8], ref, 0.0, lim)


# ------------------------------------------------------------------ streams, graphs, and the operators together

def _block(d, bank, ws):
    """A decode step's path: 4-bit projection -> add and norm -> the layer -> add and norm to codes."""
    a = moe.awq_matmul(d["attn"], d["q"], d["z"], d["s"], ws=ws[0])
    n1 = moe.add_rmsnorm(a, d["w1"], d["res"])
    y = moe.layer(n1.y, d["router"], d["k"], bank, d["shared"], ws=ws[1])
    n2 = moe.add_rmsnorm(y, d["w2"], n1.residual, outputs=("y", "fp8"))
    return a, n1, y, n2


def _block_inputs(T, seed):
    w = workloads.scaled(workloads.get("decode_awq"), T=T, E=16, k=4)
    g = workloads.generate(w, seed=seed, device=DEV)
    H = g["x"].shape[1]
    q, z, s = _awq(2 * H, H, 32, seed + 1)
    return dict(attn=_randn(T, 2 * H, seed=seed, dtype=BF), q=q, z=z, s=s, res=_randn(T, H, seed=seed + 2, dtype=BF),
                w1=_randn(H, seed=seed + 3, dtype=BF, scale=0.1), w2=_randn(H, seed=seed + 4, dtype=BF, scale=0.1),
                router=g["router"], shared=g["shared"], k=w.k), g["experts"], w


@pytest.mark.parametrize("T", [1, 16])
def test_a_decode_block(T):
    d, bank, w = _block_inputs(T, 3)
    ws = (moe.Workspace(DEV), moe.Workspace(DEV))
    a, n1, y, n2 = _block(d, bank, ws)
    _check_awq(a, d["attn"], d["q"], d["z"], d["s"])
    _check_norm(a, d["w1"], d["res"], n1, 1e-6, 1.0)
    assert torch.equal(y, moe.moe_layer(n1.y, d["router"], d["k"], bank, d["shared"]))
    _check_norm(y, d["w2"], n1.residual, n2, 1e-6, 1.0)
    # captured: every replay equals the eager run, with other eager work between the replays
    want = [t.clone() for t in (a, n1.y, n1.residual, y, n2.y, n2.codes, n2.scales)]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    gws = (moe.Workspace(DEV), moe.Workspace(DEV))
    with torch.cuda.graph(graph):
        ga, g1, gy, g2 = _block(d, bank, gws)
    for _ in range(3):
        _block(d, bank, ws)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(want, (ga, g1.y, g1.residual, gy, g2.y, g2.codes, g2.scales)))


def _router_step(d, k, ws):
    n = moe.add_rmsnorm(d["x"], d["w"], d["res"], outputs=("y", "rstd"))
    idx, _, gate, logits = moe.route(n.y, d["router"], k, want_logits=True, ws=ws)
    counts = moe.expert_counts(idx, d["router"].shape[0], token_valid=d["valid"])
    loss, prob_sum, dlogits = moe.balance_loss(logits, counts, k, 0.02, token_valid=d["valid"], topk_idx=idx, gate=gate, dgate=d["dgate"],
                                               ws=ws)
    dy = d["dy"] if "dy" in d else dlogits @ d["router"].float()
    dx, dw = moe.add_rmsnorm_backward(dy, n.residual, n.rstd, d["w"], dres=d["dres"], ws=ws)
    return n.y, loss, dlogits, dx, dw


@pytest.mark.parametrize("T,H,E,k", [(3, 256, 16, 2), (301, 640, 60, 6), (1000, 2560, 512, 10)])
def test_a_router_training_step(T, H, E, k):
    d = dict(x=_randn(T, H, seed=1, dtype=BF), w=_randn(H, seed=2, scale=0.1), res=_randn(T, H, seed=3), router=_randn(E, H, seed=4, dtype=BF, scale=0.05),
             valid=(torch.rand(T, generator=_gen(5), device=DEV) < 0.8).to(torch.uint8), dgate=_randn(T, k, seed=6, scale=1e-2),
             dres=_randn(T, H, seed=7, scale=1e-2))
    y, loss, dlogits, dx, dw = _router_step(d, k, moe.Workspace(DEV))
    # the same step in 64 bits, from the rows that the norm gave (the routing's decisions are taken on them)
    s = (d["x"].float() + d["res"]).double().requires_grad_()
    w = d["w"].double().requires_grad_()
    v = s / torch.sqrt((s * s).mean(1, keepdim=True) + 1e-6) * (1 + w)
    v.data.copy_(y.double())
    logits = v @ d["router"].double().t()
    idx = torch.sort(logits.float(), dim=1, descending=True, stable=True).indices[:, :k]
    on = d["valid"].double()[:, None]
    c = R.counts(idx, E, d["valid"]).double()
    f = c / c.sum().clamp(min=1)
    ref = 0.02 * E * k / c.sum().clamp(min=1) * (torch.softmax(logits, 1) * on * f).sum()
    total = ref + (torch.softmax(logits.gather(1, idx), 1) * d["dgate"].double() * on).sum() + (s * d["dres"].double()).sum()
    gs, gw = torch.autograd.grad(total, (s, w))
    ref = float(ref.detach())
    assert abs(float(loss) - ref) <= 1e-5 * ref
    # fp32 arithmetic throughout, except that autograd's product has y's own rounding nowhere: 1e-5 of the whole
    assert (dx.double() - gs).norm() <= 1e-5 * gs.norm() and (dw.double() - gw).norm() <= 1e-5 * gw.norm() + 1e-9


def test_router_step_captured():
    T, H, E, k = 200, 640, 64, 4
    mk = lambda o: dict(x=_randn(T, H, seed=1 + o, dtype=BF), w=_randn(H, seed=2 + o, scale=0.1), res=_randn(T, H, seed=3 + o),
                        router=_randn(E, H, seed=4 + o, dtype=BF, scale=0.05), valid=None, dgate=_randn(T, k, seed=6 + o), dres=None,
                        dy=_randn(T, H, seed=7 + o))
    d, other = mk(0), mk(100)
    ws, gws = moe.Workspace(DEV), moe.Workspace(DEV)
    want = [t.clone() for t in _router_step(d, k, ws)]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = _router_step(d, k, gws)
    for _ in range(3):
        _router_step(other, k, ws)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want))


def test_two_streams_without_given_workspaces():
    mk = lambda o: (_randn(2000, 640, seed=o), _randn(640, seed=o + 1, scale=0.1), _randn(2000, 640, seed=o + 2), *_routing(3000, 512, 8, F32, o + 3)[:2],
                    _randn(4, 8192, seed=o + 5, dtype=BF), *_awq(8192, 2560, 32, o + 6))

    def run(s, w, dy, logits, idx, x, q, z, sc):
        rstd = moe.add_rmsnorm(s, w, outputs=("y", "rstd")).rstd
        out = list(moe.add_rmsnorm_backward(dy, s, rstd, w))
        counts = moe.expert_counts(idx, 512)
        return out + [counts] + list(moe.balance_loss(logits, counts, 8, 0.01)) + [moe.awq_matmul(x, q, z, sc)]
    a, b = mk(0), mk(50)
    want = run(*a), run(*b)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(5):
        with torch.cuda.stream(s1):
            ga = run(*a)
        with torch.cuda.stream(s2):
            gb = run(*b)
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(want[0], ga)) and all(torch.equal(p, q) for p, q in zip(want[1], gb))
