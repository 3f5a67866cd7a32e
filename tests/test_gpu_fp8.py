"""FP8 quantisation, block-scaled products and W8A8 experts on the GPU against their 64-bit forms (a8_ref)."""
import pytest
import torch

import sparse_moe_expert_router_amd as moe
from tests import a8_ref as R

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def _gen(seed):
    return torch.Generator().manual_seed(seed)


# ------------------------------------------------------------------ quantiser

@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,n", [(1, 16), (1, 128), (3, 144), (7, 688), (64, 2560), (1025, 640), (2, 8208)])
def test_quantize_is_bit_exact(T, n, dtype):
    x = (torch.randn((T, n), generator=_gen(T * n)) * torch.exp2(torch.randint(-20, 20, (T, 1), generator=_gen(1)).float())).to(dtype)
    x[0, :16] = 0
    codes, s = moe.fp8_quantize(x.to(DEV))
    rc, rs = R.quantize(x.double())
    assert torch.equal(s.cpu().double(), rs)
    assert torch.equal(codes.cpu(), rc)


def test_quantize_every_bf16_magnitude_and_ties():
    # each row: one group whose largest value is a bf16 number, with every bf16 below it in two binades and far below
    amax = torch.arange(0x3F80, 0x4000, dtype=torch.int16).view(torch.bfloat16).double()     # [1, 2)
    below = torch.cat([torch.arange(0x3C00, 0x3F80, dtype=torch.int16).view(torch.bfloat16).double(), torch.zeros(1).double()])
    cols = below.view(-1)
    n = 127
    rows = []
    for i in range(0, cols.numel(), n):
        part = torch.nn.functional.pad(cols[i:i + n], (0, n - cols[i:i + n].numel()))
        rows.append(torch.cat([amax[:, None], part[None].expand(amax.numel(), n)], 1))
    x = torch.cat(rows).bfloat16()
    x[1::2] = -x[1::2]
    codes, s = moe.fp8_quantize(x.to(DEV))
    rc, rs = R.quantize(x.double())
    assert torch.equal(s.cpu().double(), rs) and torch.equal(codes.cpu(), rc)


def test_quantize_special_values():
    x = torch.zeros((6, 256))
    x[1, 0] = 1e-40                      # below the smallest scale's range: codes of a tiny group
    x[2, 5] = float("inf")
    x[3, 200] = float("nan")
    x[4, 0], x[4, 1] = 3e38, -3e38
    x[5, :] = -0.0
    codes, s = moe.fp8_quantize(x.to(DEV))
    codes, s = codes.cpu(), s.cpu()
    v = R.decode(codes) * R.spread(s.double(), 256)
    assert (codes[0] == 0).all() and (s[0] == 2.0 ** -126).all()
    assert torch.isfinite(v[[0, 1, 4, 5]]).all() and (v[1].abs() <= 1e-38).all()
    assert torch.isnan(v[2, :128]).all() and (v[2, 128:] == 0).all()
    assert (v[3, :128] == 0).all() and torch.isnan(v[3, 128:]).all()
    assert v[4, 0] > 2.9e38 and v[4, 1] < -2.9e38


def test_quantize_strided_rows_and_empty():
    wide = torch.randn((9, 512), generator=_gen(3)).bfloat16().to(DEV)
    x = wide[:, 64:64 + 160]
    codes, s = moe.fp8_quantize(x)
    rc, rs = R.quantize(x.cpu().double())
    assert torch.equal(codes.cpu(), rc) and torch.equal(s.cpu().double(), rs)
    c0, s0 = moe.fp8_quantize(torch.empty((0, 128), dtype=torch.bfloat16, device=DEV))
    assert c0.shape == (0, 128) and s0.shape == (0, 1)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_quantize_over_the_range_of_scales(dtype):
    """Rows of every magnitude, down to denormal values and up to the type's largest; codes and scales bit for bit (the
    reference's quotient is a 64-bit one rounded to fp32, which is the fp32 quotient: 53 >= 2 * 24 + 2 bits)."""
    k = torch.arange(-145, 127).repeat_interleave(8)
    x = torch.randn((k.numel(), 512), generator=_gen(9), dtype=torch.float64).clamp(-1.9, 1.9)
    x[:, 128:256] = (torch.randint(-16, 17, (k.numel(), 128), generator=_gen(10)) / 16 * 1.75).double()   # many ties
    x[:, 256:384] *= 2.0 ** -torch.randint(0, 24, (k.numel(), 128), generator=_gen(11)).double()
    x = (x * torch.exp2(k.double())[:, None]).to(dtype)
    codes, s = moe.fp8_quantize(x.to(DEV))
    rc, rs = R.quantize(x.double())
    assert torch.equal(s.cpu().double(), rs) and torch.equal(codes.cpu(), rc)


# ------------------------------------------------------------------ product

def _codes(shape, g):
    c = torch.randint(0, 256, shape, generator=g, dtype=torch.int64)
    return torch.where((c & 127) == 127, c - 1, c).to(torch.uint8)      # every finite code


def _check_product(y, a, sa, w, sw):
    a, sa, w, sw = (t.to(DEV) for t in (a, sa, w, sw))
    K = a.shape[1]
    av = R.decode(a) * R.spread(sa.double(), K)
    wv = R.weights(w, sw)
    ref, bound = R.product(av, wv, K, y.dtype == torch.float32)
    half = torch.finfo(y.dtype).eps / 2
    err = (y.double() - ref).abs()
    lim = bound + half * (ref.abs() + bound)
    assert (err <= lim).all(), f"largest excess {(err - lim).max():.3e} at {(err - lim).argmax()}"
    # signs are random here: the errors of the outputs together (fp32: 128 2^-23 of each, as the products)
    assert err.norm() <= (half + (2.0 ** -16 if y.dtype == torch.float32 else 2.0 ** -10)) * ref.norm()


SHAPES = [(1, 16, 16), (1, 1, 128), (1, 2560, 2560), (5, 33, 144), (16, 128, 640), (17, 130, 1296), (31, 257, 128), (33, 1000, 272),
          (77, 1000, 1296), (128, 256, 256), (129, 300, 384), (200, 640, 2560), (256, 256, 128), (257, 513, 1040), (300, 1280, 512),
          (513, 129, 2064), (1000, 384, 640), (2048, 264, 1152), (4100, 4099, 144), (4097, 4200, 128), (2300, 8200, 1280), (12, 9000, 400), (40, 18000, 272), (1500, 700, 656)]


@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_matmul(M, N, K, out):
    g = _gen(M + 3 * N + 7 * K)
    a, w = _codes((M, K), g), _codes((N, K), g)
    kb = -(-K // 128)
    sa = torch.rand((M, kb), generator=g) + 0.1
    sw = torch.rand((-(-N // 128), kb), generator=g) * 0.01 - 0.005
    y = torch.empty((M, N), dtype=out, device=DEV)
    moe.fp8_matmul(a.to(DEV), sa.to(DEV), w.to(DEV), sw.to(DEV), y=y)
    _check_product(y, a, sa, w, sw)


@pytest.mark.parametrize("M,N,K", [(3, 50, 144), (40, 260, 272), (300, 600, 400)])
def test_matmul_strided_and_untouched_surroundings(M, N, K):
    g = _gen(M)
    A, W = _codes((M + 2, K + 64), g), _codes((N, K + 32), g)
    # what lies between the rows is NaN: it must not be used
    A[:, :16], A[:, 16 + K:], W[:, K:] = 127, 127, 127
    a, w = A.to(DEV)[1:M + 1, 16:16 + K], W.to(DEV)[:, :K]
    kb = -(-K // 128)
    sa, sw = torch.rand((M, kb), generator=g), torch.rand((-(-N // 128), kb), generator=g)
    big = torch.full((M + 2, N + 13), 7.0, dtype=torch.bfloat16, device=DEV)
    y = big[1:M + 1, 3:3 + N]
    moe.fp8_matmul(a, sa.to(DEV), w, sw.to(DEV), y=y)
    _check_product(y, a.cpu(), sa, w.cpu(), sw)
    assert (big[0] == 7).all() and (big[-1] == 7).all() and (big[:, :3] == 7).all() and (big[:, 3 + N:] == 7).all()


@pytest.mark.parametrize("M", [2, 40, 600, 1500, 9000])
def test_matmul_nan_stays_in_its_row_and_column(M):
    N, K = 400, 384
    g = _gen(5)
    a, w = _codes((M, K), g), _codes((N, K), g)
    a[1, 200], w[17, 3] = 127, 255
    sa, sw = torch.rand((M, 3), generator=g), torch.rand((4, 3), generator=g)
    y = moe.fp8_matmul(a.to(DEV), sa.to(DEV), w.to(DEV), sw.to(DEV), out_dtype=moe.OUT_F32).cpu()
    bad = torch.zeros((M, N), dtype=torch.bool)
    bad[1], bad[:, 17] = True, True
    assert torch.equal(torch.isnan(y), bad)


def test_matmul_no_rows():
    y = moe.fp8_matmul(torch.empty((0, 256), dtype=torch.uint8, device=DEV), torch.empty((0, 2), device=DEV),
                       torch.zeros((64, 256), dtype=torch.uint8, device=DEV), torch.ones((1, 2), device=DEV))
    assert y.shape == (0, 64)


# ------------------------------------------------------------------ experts

def _bank(E, H, F, seed):
    g = _gen(seed)
    out = {"fmt": "fp8"}
    for n, o, i in (("gate", F, H), ("up", F, H), ("down", H, F)):
        out[n + "_codes"] = _codes((E, o, i), g)
        out[n + "_bscales"] = (torch.rand((E, o // 128, i // 128), generator=g) + 0.5) * 2e-4
    return out


def _gpu(bank):
    return {k: v if isinstance(v, str) else v.to(DEV) for k, v in bank.items()}


def _check_experts(rows, x, k, bank, off, sp):
    x, sp = x.to(DEV), sp.to(DEV)
    codes, s = R.quantize(x.double())
    xq = R.decode(codes) * R.spread(s, x.shape[1])
    half = torch.finfo(rows.dtype).eps / 2
    got = rows.double()
    total = 0
    for e in range(off.numel() - 1):
        lo, hi = int(off[e]), int(off[e + 1])
        if lo == hi:
            continue
        tok = sp[lo:hi].long() // k
        w = [R.weights(bank[n + "_codes"][e].to(DEV), bank[n + "_bscales"][e].to(DEV)) for n in ("gate", "up", "down")]
        ref, bound = R.expert_a8(xq[tok], *w)
        err = (got[lo:hi] - ref).abs()
        lim = bound + half * (ref.abs() + bound)
        assert (err <= lim).all(), f"expert {e}: largest excess {(err - lim).max():.3e}"
        total = total + torch.stack([(got[lo:hi] - ref).square().sum(), ref.square().sum()])
    # The bound allows for every near tie of h at once.  Together: h is off by about 2^-14 (the cut products of
    # full-range random codes), so a share of 2 * 16 * 2^-14 = 2^-9 of its codes, the steps of E4M3 being 2^-3
    # to 2^-4 apart, is a step off: sqrt(2^-9) 2^-3.5 = 2^-8 of the rows; twice that.  An average over codes a
    # step off: of 768 codes (six rows) 1.5 are expected, and one of them alone can be 2^-3 of the largest term
    # of a row, so it is held only where 2^16 codes (128 expected) make it one.
    if got.shape[0] * w[0].shape[0] >= 1 << 16:
        assert total[0].sqrt() <= (half + 2.0 ** -7) * total[1].sqrt()


def _sorted(idx, E):
    flat = idx.reshape(-1)
    sp = torch.sort(flat, stable=True).indices.int()
    off = torch.cat([torch.zeros(1, dtype=torch.int64), torch.bincount(flat, minlength=E).cumsum(0)]).int()
    return off, sp


FFN = [(1, 256, 128, 4, 2), (5, 128, 256, 16, 3), (16, 384, 128, 8, 2), (40, 256, 384, 3, 2), (70, 512, 128, 2, 1), (300, 256, 256, 4, 2),
       (700, 384, 128, 3, 3), (1100, 128, 128, 2, 2),
       # deep enough for runs of tiles, with one tile a workgroup and with several; 64-, 128- and 256-row tiles
       (70, 2560, 640, 2, 1), (300, 1024, 512, 4, 2), (700, 1152, 640, 3, 3), (260, 1280, 1024, 8, 2), (9000, 1024, 1152, 4, 2),
       (5000, 1152, 512, 64, 2), (2000, 2176, 640, 32, 1)]


@pytest.mark.parametrize("out", [moe.OUT_BF16, moe.OUT_F32])
@pytest.mark.parametrize("T,H,F,E,k", FFN)
def test_experts(T, H, F, E, k, out):
    g = _gen(T + H)
    x = torch.randn((T, H), generator=g).bfloat16()
    bank = _bank(E, H, F, 9)
    idx = torch.rand((T, E), generator=g).topk(k, 1).indices
    off, sp = _sorted(idx, E)
    rows = moe.grouped_ffn_a8(x.to(DEV), k, _gpu(bank), off.to(DEV), sp.to(DEV), out_dtype=out)
    _check_experts(rows, x, k, bank, off, sp)


@pytest.mark.parametrize("T", [64, 700])
def test_experts_all_tokens_on_one_and_empty_experts(T):
    H, F, E = 256, 128, 9
    x = torch.randn((T, H), generator=_gen(2)).bfloat16()
    bank = _bank(E, H, F, 3)
    off, sp = _sorted(torch.full((T, 1), 4), E)
    rows = moe.grouped_ffn_a8(x.to(DEV), 1, _gpu(bank), off.to(DEV), sp.to(DEV))
    _check_experts(rows, x, 1, bank, off, sp)


@pytest.mark.parametrize("T", [1, 20, 513])
def test_experts_identity(T):
    x = torch.randn((T, 384), generator=_gen(4)).bfloat16()
    bank = _bank(1, 384, 256, 5)
    rows = moe.grouped_ffn_a8(x.to(DEV), 1, _gpu(bank))
    _check_experts(rows, x, 1, bank, torch.tensor([0, T]), torch.arange(T).int())


@pytest.mark.parametrize("T", [6, 400])
def test_experts_nan_row_stays_alone(T):
    H, F, E, k = 256, 128, 4, 2
    x = torch.randn((T, H), generator=_gen(6)).bfloat16()
    x[3, 17], x[5, 0] = float("inf"), float("nan")
    bank = _bank(E, H, F, 3)
    idx = torch.rand((T, E), generator=_gen(7)).topk(k, 1).indices
    off, sp = _sorted(idx, E)
    rows = moe.grouped_ffn_a8(x.to(DEV), k, _gpu(bank), off.to(DEV), sp.to(DEV)).cpu()
    tok = sp.long() // k
    bad = (tok == 3) | (tok == 5)
    assert torch.isnan(rows[bad]).all() and torch.isfinite(rows[~bad]).all()


def test_experts_zero_rows_give_zero():
    bank = _bank(2, 128, 128, 1)
    off, sp = _sorted(torch.tensor([[0], [1], [1]]), 2)
    rows = moe.grouped_ffn_a8(torch.zeros((3, 128), dtype=torch.bfloat16, device=DEV), 1, _gpu(bank), off.to(DEV), sp.to(DEV))
    assert (rows == 0).all()


@pytest.mark.parametrize("T", [8, 300])
def test_route_experts_combine_together(T):
    """The layer of separate calls with W8A8 experts: route, permute, experts, combine."""
    H, F, E, k = 512, 256, 32, 4
    g = _gen(T)
    x = torch.randn((T, H), generator=g).bfloat16()
    wr = (torch.randn((E, H), generator=g) * 0.05).bfloat16()
    bank = _bank(E, H, F, 21)
    gb = _gpu(bank)
    idx, tl, gate, off, sp, p2r = moe.route_permute(x.to(DEV), wr.to(DEV), k)
    rows = moe.grouped_ffn_a8(x.to(DEV), k, gb, off, sp)
    y = moe.combine(rows, p2r, gate)
    _check_experts(rows, x, k, bank, off.cpu(), sp.cpu())
    ref = (rows.cpu().double()[p2r.cpu().long()].view(T, k, H) * gate.cpu().double()[..., None]).sum(1)
    bound = (rows.cpu().double()[p2r.cpu().long()].view(T, k, H) * gate.cpu().double()[..., None]).abs().sum(1) * (k + 1) * 2.0 ** -24
    assert ((y.cpu().double() - ref).abs() <= bound + 2.0 ** -8 * (ref.abs() + bound)).all()


@pytest.mark.parametrize("T,E", [(16, 16), (600, 2)])
def test_replays_of_a_captured_call(T, E):
    H, F, k = 256, 128, 2
    bank = _gpu(_bank(E, H, F, 2))
    x = torch.zeros((T, H), dtype=torch.bfloat16, device=DEV)
    off, sp = _sorted(torch.rand((T, E), generator=_gen(8)).topk(k, 1).indices, E)
    off, sp = off.to(DEV), sp.to(DEV)
    ws = moe.Workspace(x.device)
    rows = torch.empty((T * k, H), dtype=torch.bfloat16, device=DEV)
    moe.grouped_ffn_a8(x, k, bank, off, sp, ws=ws, rows=rows)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.grouped_ffn_a8(x, k, bank, off, sp, ws=ws, rows=rows)
    for i in range(4):
        x.copy_(torch.randn((T, H), generator=_gen(i)).bfloat16())
        graph.replay()
        torch.cuda.synchronize()
        got = rows.clone()
        want = moe.grouped_ffn_a8(x, k, bank, off, sp)
        assert torch.equal(got, want)


def test_on_a_side_stream():
    x = torch.randn((33, 256), generator=_gen(1)).bfloat16().to(DEV)
    bank = _gpu(_bank(1, 256, 128, 2))
    want = moe.grouped_ffn_a8(x, 1, bank)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        c, sc = moe.fp8_quantize(x)
        got = moe.grouped_ffn_a8(x, 1, bank, ws=moe.Workspace(x.device))
    s.synchronize()
    assert torch.equal(got, want)
    assert torch.equal(c, moe.fp8_quantize(x)[0])


# ------------------------------------------------------------------ many rows through runs of tiles, and long offsets

@pytest.mark.parametrize("T", [150, 513, 1500])
def test_experts_identity_deep(T):
    x = torch.randn((T, 1024), generator=_gen(4)).bfloat16()
    bank = _bank(1, 1024, 512, 5)
    rows = moe.grouped_ffn_a8(x.to(DEV), 1, _gpu(bank))
    _check_experts(rows, x, 1, bank, torch.tensor([0, T]), torch.arange(T).int())


@pytest.mark.parametrize("T", [300, 1100])
def test_experts_deep_with_empty_experts_and_nan_rows(T):
    H, F, E, k = 1024, 512, 12, 2
    x = torch.randn((T, H), generator=_gen(6)).bfloat16()
    bank = _bank(E, H, F, 3)
    idx = torch.full((T, k), 7)
    idx[:, 1] = 10
    idx[3], idx[-1] = torch.tensor([0, 11]), torch.tensor([7, 0])
    off, sp = _sorted(idx, E)
    args = (k, _gpu(bank), off.to(DEV), sp.to(DEV))
    rows = moe.grouped_ffn_a8(x.to(DEV), *args)
    _check_experts(rows, x, k, bank, off, sp)
    x[3, 17], x[5, 0] = float("inf"), float("nan")
    got = moe.grouped_ffn_a8(x.to(DEV), *args).cpu()
    tok = sp.long() // k
    bad = (tok == 3) | (tok == 5)
    assert torch.isnan(got[bad]).all() and torch.equal(got[~bad], rows.cpu()[~bad])


def test_experts_deep_replays_and_surroundings():
    T, H, F, E, k = 700, 1152, 512, 3, 2
    bank = _gpu(_bank(E, H, F, 2))
    x = torch.zeros((T, H), dtype=torch.bfloat16, device=DEV)
    off, sp = _sorted(torch.rand((T, E), generator=_gen(8)).topk(k, 1).indices, E)
    off, sp = off.to(DEV), sp.to(DEV)
    big = torch.full((T * k + 2, H), 7.0, dtype=torch.bfloat16, device=DEV)
    rows = big[1:-1]
    ws = moe.Workspace(x.device)
    moe.grouped_ffn_a8(x, k, bank, off, sp, ws=ws, rows=rows)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.grouped_ffn_a8(x, k, bank, off, sp, ws=ws, rows=rows)
    for i in range(4):
        x.copy_(torch.randn((T, H), generator=_gen(i)).bfloat16())
        graph.replay()
        torch.cuda.synchronize()
        got = rows.clone()
        assert torch.equal(got, moe.grouped_ffn_a8(x, k, bank, off, sp))
    assert (big[0] == 7).all() and (big[-1] == 7).all()


@pytest.mark.parametrize("M", [60, 1100])
def test_offsets_past_32_bits(M):
    """Rows 4 MiB apart (the most a product takes), 1100 of them (w, and a and y too): 4.6 GB from the first to the
    last."""
    K, N, ld = 256, 1100, 1 << 22
    g = _gen(M)
    a, w = _codes((M, K), g), _codes((N, K), g)
    sa, sw = torch.rand((M, 2), generator=g), torch.rand((-(-N // 128), 2), generator=g)
    buf = [torch.empty(ld * rows, dtype=torch.uint8, device=DEV) for rows in (M, N, M)]
    A, W = (b.as_strided((rows, K), (ld, 1)) for b, rows in ((buf[0], M), (buf[1], N)))
    y = buf[2].view(torch.bfloat16).as_strided((M, N), (ld // 2, 1))
    A.copy_(a), W.copy_(w)
    moe.fp8_matmul(A, sa.to(DEV), W, sw.to(DEV), y=y)
    _check_product(y.contiguous(), a, sa, w, sw)
    x = torch.randn((M, K), generator=g).bfloat16()
    y = buf[2].view(torch.bfloat16).as_strided((M, K), (ld // 2, 1))
    y.copy_(x)
    codes, s = moe.fp8_quantize(y)
    rc, rs = R.quantize(x.double())
    assert torch.equal(codes.cpu(), rc) and torch.equal(s.cpu().double(), rs)


def test_experts_rows_past_32_bits():
    """1.1 million rows of 1024 fp32 outputs, 4.6 GB: those of its first, last and some other tokens."""
    T, H, F = 1_100_003, 1024, 512
    x = torch.randn((T, H), dtype=torch.bfloat16, device=DEV)
    bank = _bank(1, H, F, 5)
    rows = moe.grouped_ffn_a8(x, 1, _gpu(bank), out_dtype=moe.OUT_F32)
    pick = torch.cat([torch.arange(16), torch.arange(1, 33) * 33331, torch.arange(T - 16, T)]).to(DEV)
    _check_experts(rows[pick], x[pick].cpu(), 1, bank, torch.tensor([0, 64]), torch.arange(64).int())


@pytest.mark.parametrize("T,H,F", [(40, 256, 128), (900, 1024, 512)])
def test_experts_offsets_that_overlap_stay_inside_the_workspace(T, H, F):
    """Wrong offsets give wrong rows, but nothing behind the workspace or the rows is written."""
    E = 64
    bank = _gpu(_bank(E, H, F, 1))
    x = torch.randn((T, H), dtype=torch.bfloat16, device=DEV)
    off = torch.tensor([0, T] * 32 + [T], dtype=torch.int32, device=DEV)
    sp = torch.arange(T, dtype=torch.int32, device=DEV)
    n = moe.workspace_bytes(moe.OP_GROUPED_FFN_A8, T, 1, E, H, F)
    buf = torch.full((n + (1 << 20),), 77, dtype=torch.uint8, device=DEV)
    big = torch.full((T + 1, H), 7.0, dtype=torch.bfloat16, device=DEV)
    ws = type("W", (), {"get": lambda s, m: (buf, n)})()
    moe.grouped_ffn_a8(x, 1, bank, off, sp, ws=ws, rows=big[:T])
    assert (buf[n:] == 77).all() and (big[T] == 7).all()


@pytest.mark.parametrize("T", [1, 77, 700])
def test_quantiser_and_products_make_the_expert(T):
    """One expert from the separate calls: quantise, gate and up with fp32 outputs, SwiGLU in torch's fp32 (within the
    bound of the kernel's), quantise, down; against the same 64-bit expert as the grouped call."""
    H, F = 384, 256
    x = torch.randn((T, H), generator=_gen(12)).bfloat16()
    bank = _bank(1, H, F, 13)
    g = _gpu(bank)
    a, sa = moe.fp8_quantize(x.to(DEV))
    gate, up = (moe.fp8_matmul(a, sa, g[n + "_codes"][0], g[n + "_bscales"][0], out_dtype=moe.OUT_F32) for n in ("gate", "up"))
    h, sh = moe.fp8_quantize(torch.nn.functional.silu(gate) * up)
    rows = moe.fp8_matmul(h, sh, g["down_codes"][0], g["down_bscales"][0])
    _check_experts(rows, x, 1, bank, torch.tensor([0, T]), torch.arange(T).int())


def test_experts_without_a_workspace_on_two_streams_and_captured():
    T, H, F, E, k = 300, 1024, 512, 8, 2
    bank = _gpu(_bank(E, H, F, 2))
    x = torch.randn((T, H), generator=_gen(14)).bfloat16().to(DEV)
    off, sp = _sorted(torch.rand((T, E), generator=_gen(15)).topk(k, 1).indices, E)
    off, sp = off.to(DEV), sp.to(DEV)
    want = moe.grouped_ffn_a8(x, k, bank, off, sp)
    streams = [torch.cuda.Stream() for _ in range(2)]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    out = []
    for _ in range(5):
        for s in streams:
            with torch.cuda.stream(s):
                out.append(moe.grouped_ffn_a8(x, k, bank, off, sp))
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in out)
    graphs, rows = [], [torch.empty_like(want) for _ in range(2)]
    for r in rows:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            moe.grouped_ffn_a8(x, k, bank, off, sp, rows=r)
        graphs.append(g)
    for i in range(3):
        x.copy_(torch.randn((T, H), generator=_gen(20 + i)).bfloat16())
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        want = moe.grouped_ffn_a8(x, k, bank, off, sp)
        assert torch.equal(rows[0], want) and torch.equal(rows[1], want)


def test_quantiser_and_product_captured():
    M, N, K = 40, 260, 400
    g = _gen(16)
    x = torch.zeros((M, K), dtype=torch.bfloat16, device=DEV)
    w, sw = _codes((N, K), g).to(DEV), torch.rand((3, 4), generator=g).to(DEV)
    codes, s = moe.fp8_quantize(x)
    y = moe.fp8_matmul(codes, s, w, sw)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.fp8_quantize(x, codes=codes, scales=s)
        moe.fp8_matmul(codes, s, w, sw, y=y)
    for i in range(4):
        x.copy_(torch.randn((M, K), generator=_gen(30 + i)).bfloat16())
        graph.replay()
        torch.cuda.synchronize()
        got = y.clone()
        assert torch.equal(got, moe.fp8_matmul(*moe.fp8_quantize(x), w, sw))


# ------------------------------------------------------------------ large products that cancel

def _code(v):
    """Codes of a tensor of values that E4M3 holds."""
    return R.encode(v.double())


def _cancelling(rows, n, g):
    """[rows, n] with 448 and -448 in the first two places of every 8, small whole numbers in the others."""
    w = torch.randint(-2, 3, (rows, n), generator=g).float()
    w[:, ::8], w[:, 1::8] = 448.0, -448.0
    return w


@pytest.mark.parametrize("M,N,K", [(1, 40, 256), (7, 300, 400), (40, 512, 1024), (300, 260, 640), (1500, 700, 656), (2300, 1000, 384)])
def test_matmul_large_products_that_cancel(M, N, K):
    """448 * 448 and -448 * 448 beside products of at most 4.  Every partial sum of a block of 128 is a whole number
    below 2^24 (16 * 448 * 448 and some), exact in fp32 in any order, and the scales are powers of two: fp32 outputs
    are exact.  bf16 outputs have the FP8 matrix cores' bound, which the largest products set."""
    g = _gen(M + K)
    a, w = torch.randint(-2, 3, (M, K), generator=g).float(), _cancelling(N, K, g)
    a[:, ::8], a[:, 1::8] = 448.0, 448.0
    kb = -(-K // 128)
    sa = torch.exp2(torch.randint(-3, 4, (M, kb), generator=g).float())
    sw = torch.exp2(torch.randint(-3, 4, (-(-N // 128), kb), generator=g).float())
    args = [t.to(DEV) for t in (_code(a), sa, _code(w), sw)]
    av, wv = R.decode(args[0]) * R.spread(args[1].double(), K), R.weights(args[2], args[3])
    ref, bound = R.product(av, wv, K, False)
    y = moe.fp8_matmul(*args, out_dtype=moe.OUT_F32)
    assert ref.abs().max() > 10 and torch.equal(y.double(), ref)
    y = moe.fp8_matmul(*args).double()
    assert ((y - ref).abs() <= bound + 2.0 ** -8 * (ref.abs() + bound)).all()


CANCEL = [(5, 256, 128), (40, 1024, 512), (300, 256, 256), (700, 1024, 512), (5000, 1024, 512), (4200, 896, 512)]


@pytest.mark.parametrize("T,H,F", CANCEL)
def test_experts_fp32_rows_when_gate_and_up_cancel(T, H, F):
    """As in the test of the product: the sums of gate and up are exact in fp32, so the rows have the bound of exact
    sums (their terms of down do not cancel)."""
    g = _gen(T)
    x = torch.randint(-2, 3, (T, H), generator=g).float()
    x[:, ::8], x[:, 1::8] = 448.0, 448.0
    bank = {"fmt": "fp8"}
    for n in ("gate", "up"):
        bank[n + "_codes"] = _code(_cancelling(F, H, g))[None]
        bank[n + "_bscales"] = torch.full((1, F // 128, H // 128), 2.0 ** -6)
    bank["down_codes"] = _codes((1, H, F), g)
    bank["down_bscales"] = torch.full((1, H // 128, F // 128), 2.0 ** -8)
    rows = moe.grouped_ffn_a8(x.bfloat16().to(DEV), 1, _gpu(bank), out_dtype=moe.OUT_F32).double()
    gate, up, down = (R.weights(bank[n + "_codes"][0].to(DEV), bank[n + "_bscales"][0].to(DEV)) for n in ("gate", "up", "down"))
    xq = x.double().to(DEV)                       # 448 is the largest of every group: its scale is 1, every value a code
    zero = torch.zeros((T, F), dtype=torch.float64, device=DEV)
    ref, bound = R.rows_a8(xq @ gate.t(), zero, xq @ up.t(), zero, down, exact=True)
    err = (rows - ref).abs()
    assert ref.abs().mean() > 1e-3 and (err <= bound + 2.0 ** -24 * (ref.abs() + bound)).all()
    # h is off by about 12 units of 2^-23, so a share of 2 * 12 * 2^-23 / 2^-4 = 2^-14.4 of its codes is a step off:
    # 2^-7.2 * 2^-3.5 of the rows.  One such code alone, of the smallest case's five rows of 128: 2^-4 of a term,
    # 2^-4 / sqrt(5 * 128) = 2^-8.7 of the rows.
    assert err.norm() <= 2.0 ** -7 * ref.norm()


@pytest.mark.parametrize("T,H,F", CANCEL)
def test_experts_fp32_rows_when_down_cancels(T, H, F):
    """h is 448 m in two places of every 8 and m or 2 m in the others, up to a sign: codes 448, 1 and 2.  The sum of down
    is a whole number below 2^24 in fp32; what is left are h's scale (swiglu's 8 + |g| units of 2^-23 and a division),
    its product with the weights' scale, and the rounding of each block's share: 8 + |g| + 3 + blocks units."""
    g = _gen(T)
    x = torch.zeros((T, H))
    x[:, 0] = torch.randint(1, 4, (T,), generator=g).float()
    gate, up = torch.zeros((F, H)), torch.zeros((F, H))
    gate[:, 0] = 1.0
    up[:, 0] = torch.randint(-2, 3, (F,), generator=g).float()
    up[::8, 0], up[1::8, 0] = 448.0, 448.0
    bank = {"fmt": "fp8", "gate_codes": _code(gate)[None], "up_codes": _code(up)[None], "down_codes": _code(_cancelling(H, F, g))[None],
            "gate_bscales": torch.ones((1, F // 128, H // 128)), "up_bscales": torch.ones((1, F // 128, H // 128)),
            "down_bscales": torch.ones((1, H // 128, F // 128))}
    rows = moe.grouped_ffn_a8(x.bfloat16().to(DEV), 1, _gpu(bank), out_dtype=moe.OUT_F32).double().cpu()
    v = x[:, :1].double()
    h = torch.sigmoid(v) * v * v * up[:, 0].double()
    ref = h @ R.decode(bank["down_codes"][0]).t()
    size = h.abs() @ R.decode(bank["down_codes"][0]).abs().t()
    size -= 2 * 448 * 448 * (F // 8) * (torch.sigmoid(v) * v * v)      # what does not cancel
    assert ref.abs().mean() > 1 and ((rows - ref).abs() <= (8 + 3 + 3 + F // 128) * 2.0 ** -23 * size).all()


def test_a_captured_call_after_its_workspace_has_grown():
    H, F, E, k = 1024, 512, 8, 2
    bank = _gpu(_bank(E, H, F, 2))
    mk = lambda T, seed: (torch.randn((T, H), generator=_gen(seed)).bfloat16().to(DEV),
                          *(t.to(DEV) for t in _sorted(torch.rand((T, E), generator=_gen(seed)).topk(k, 1).indices, E)))
    x, off, sp = mk(40, 1)
    big = mk(4000, 2)
    ws = moe.Workspace(x.device)
    rows = torch.empty((40 * k, H), dtype=torch.bfloat16, device=DEV)
    moe.grouped_ffn_a8(x, k, bank, off, sp, ws=ws, rows=rows)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.grouped_ffn_a8(x, k, bank, off, sp, ws=ws, rows=rows)
    moe.grouped_ffn_a8(big[0], k, bank, *big[1:], ws=ws)          # grows
    others = [torch.full((1 << 20,), 7, dtype=torch.uint8, device=DEV) for _ in range(64)]
    for i in range(3):
        x.copy_(torch.randn(x.shape, generator=_gen(10 + i)).bfloat16())
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(rows, moe.grouped_ffn_a8(x, k, bank, off, sp)) and all((o == 7).all() for o in others)


@pytest.mark.parametrize("M", [1, 9])
def test_matmul_over_more_outputs_than_streaming_workgroups(M):
    """2^27 + 300 outputs of 16 inputs: more groups of 16 than a launch holds workgroups."""
    N, K = (1 << 27) + 300, 16
    w = torch.randint(0, 120, (N, K), dtype=torch.uint8, device=DEV)
    sw = torch.rand((-(-N // 128), 1), device=DEV) + 0.5
    a, sa = torch.randint(0, 120, (M, K), generator=_gen(1)).to(torch.uint8), torch.rand((M, 1), generator=_gen(2)) + 0.5
    y = moe.fp8_matmul(a.to(DEV), sa.to(DEV), w, sw)
    for lo in (0, (1 << 20) - 128, (1 << 26) + 128 * 77, (1 << 27) - 128 * 16, (1 << 27) + 128):
        n = min(4096, N - lo)
        got = y[:, lo:lo + n].contiguous()
        av = R.decode(a.to(DEV)) * sa.to(DEV).double()
        ref, bound = R.product(av, R.weights(w[lo:lo + n], sw[lo // 128:lo // 128 + -(-n // 128)]), K, False)
        assert ((got.double() - ref).abs() <= bound + 2.0 ** -8 * (ref.abs() + bound)).all()


@pytest.mark.parametrize("out", [moe.OUT_BF16, moe.OUT_F32])
@pytest.mark.parametrize("M,K", [(1, 128), (3, 400), (40, 640), (700, 400), (700, 128), (2000, 400), (2000, 128), (40000, 272)])
def test_matmul_infinite_weight_scale(M, K, out):
    """Positive codes times an infinite scale are infinite: no block behind the last one adds 0 * inf."""
    N, kb = 300, -(-K // 128)
    g = _gen(K)
    a, w = (torch.randint(1, 120, s, generator=g).to(torch.uint8) for s in ((M, K), (N, K)))
    sa, sw = torch.rand((M, kb), generator=g) + 0.5, torch.rand((3, kb), generator=g) + 0.5
    clean = moe.fp8_matmul(*(t.to(DEV) for t in (a, sa, w, sw)), out_dtype=out)
    sw[1, kb - 1] = float("inf")
    y = moe.fp8_matmul(*(t.to(DEV) for t in (a, sa, w, sw)), out_dtype=out)
    assert (y[:, 128:256] == float("inf")).all()
    assert torch.equal(y[:, :128], clean[:, :128]) and torch.equal(y[:, 256:], clean[:, 256:])
