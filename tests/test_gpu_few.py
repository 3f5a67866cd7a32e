"""moe_layer_few on the GPU against the 64-bit layer (few_ref)."""
import pytest
import torch

import sparse_moe_expert_router_amd as moe
import workloads
from tests import few_ref as R

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def _make(T, H, E, k, F, Fs, fmt, seed=0):
    """Inputs of the tiny recipe at the given sizes, on the GPU."""
    w = workloads.Workload("few", T=T, H=H, E=E, k=k, F=F, Fs=max(Fs, 32), fmt="awq" if fmt == "awq_om" else fmt)
    d = workloads.generate(w, seed=seed, device=DEV, with_shared=Fs > 0)
    bank = moe.awq_to_output_major(d["experts"]) if fmt == "awq_om" else d["experts"]
    return d["x"], d["router"], bank, d.get("shared")


def _check(y, idx, ref):
    want, bound, ridx = ref
    assert torch.equal(idx, ridx.to(idx.device))
    err = (y.double() - want).abs()
    lim = bound + 2.0 ** -8 * (want.abs() + bound)
    assert (err <= lim).all(), f"largest excess {(err - lim).max():.3e}"


CASES = [  # T, H, E, k, F, Fs
    (1, 256, 16, 2, 128, 128), (1, 256, 4, 4, 128, 0), (2, 512, 1, 1, 256, 64), (3, 768, 40, 5, 384, 96),
    (4, 2560, 24, 10, 640, 640), (7, 256, 600, 3, 128, 32), (11, 1024, 1000, 10, 128, 0), (16, 256, 8, 8, 256, 256),
    (16, 512, 64, 10, 128, 128), (5, 4096, 6, 2, 1152, 160), (2, 256, 70, 64, 128, 32)]


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "awq_om"])
@pytest.mark.parametrize("T,H,E,k,F,Fs", CASES)
def test_layer(T, H, E, k, F, Fs, fmt):
    x, router, bank, shared = _make(T, H, E, k, F, Fs, fmt, seed=T)
    y, idx = moe.layer_few(x, router, k, bank, shared)
    _check(y, idx, R.layer(x, router, k, bank, shared))


@pytest.mark.parametrize("H,F", [(192, 32), (320, 96), (64, 160), (2624, 672)])
def test_sizes_only_bf16_takes(H, F):
    x, router, bank, shared = _make(6, H, 12, 3, F, 96, "bf16")
    y, idx = moe.layer_few(x, router, 3, bank, shared)
    _check(y, idx, R.layer(x, router, 3, bank, shared))


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "awq_om"])
def test_every_token_on_the_same_experts(fmt):
    x, router, bank, shared = _make(16, 512, 32, 4, 256, 64, fmt)
    x[1:] = x[0]
    y, idx = moe.layer_few(x, router, 4, bank, shared)
    assert (idx == idx[0]).all()
    _check(y, idx, R.layer(x, router, 4, bank, shared))
    assert (y == y[0]).all()


def test_ties_go_to_the_lowest_expert():
    x, router, bank, shared = _make(3, 256, 48, 6, 128, 32, "bf16")
    router[:] = router[0]
    _, idx = moe.layer_few(x, router, 6, bank, shared)
    assert (idx.cpu() == torch.arange(6)).all()


def test_shared_scale_and_given_outputs():
    x, router, bank, shared = _make(9, 512, 20, 3, 128, 96, "fp8")
    scale = torch.linspace(-1, 2, 9, device=DEV)
    few = moe.FewTokenLayer(router, 3, bank, shared)
    y, idx = torch.full((9, 512), 7.0, dtype=torch.bfloat16, device=DEV), torch.full((9, 3), -1, dtype=torch.int32, device=DEV)
    a, b = few(x, shared_scale=scale, y=y, topk_idx=idx)
    assert a is y and b is idx
    _check(y, idx, R.layer(x, router, 3, bank, shared, scale))


@pytest.mark.parametrize("T", [1, 5, 16])
def test_only_the_calls_rows_are_written(T):
    x, router, bank, shared = _make(16, 256, 16, 2, 128, 128, "bf16")
    big = torch.full((18, 256), 7.0, dtype=torch.bfloat16, device=DEV)
    moe.layer_few(x[:T], router, 2, bank, shared, y=big[1:1 + T])
    assert (big[0] == 7).all() and (big[1 + T:] == 7).all() and (big[1:1 + T] != 7).any()


def test_one_object_for_every_number_of_tokens_and_repeats():
    x, router, bank, shared = _make(16, 512, 64, 4, 128, 64, "awq_om")
    few = moe.FewTokenLayer(router, 4, bank, shared)
    few.ws_buf.fill_(0xFF)                      # any content will do
    for T in (16, 1, 7, 2, 16, 3):
        y, idx = few(x[:T])
        for _ in range(5):
            y2, idx2 = few(x[:T])
            assert torch.equal(y, y2) and torch.equal(idx, idx2)
        one = torch.cat([few(x[t:t + 1])[0] for t in range(T)])
        # the experts' order of a token's sum differs with the other tokens: fp32 sums, then the bf16 rounding
        assert ((one.double() - y.double()).abs() <= 2.0 ** -7 * y.double().abs() + 2.0 ** -12 * y.double().abs().max()).all()
    y, idx = few(x[:0])
    assert y.shape == (0, 512) and idx.shape == (0, 4)


def test_nan_token_stays_alone():
    x, router, bank, shared = _make(6, 256, 16, 2, 128, 32, "bf16")
    clean, _ = moe.layer_few(x, router, 2, bank, shared)
    x2 = x.clone()
    x2[2, 5] = float("nan")
    y, idx = moe.layer_few(x2, router, 2, bank, shared)
    assert torch.isnan(y[2]).all() and ((idx >= 0) & (idx < 16)).all()
    keep = [0, 1, 3, 4, 5]
    assert torch.isfinite(y[keep]).all()
    assert ((y[keep].double() - clean[keep].double()).abs() <= 2.0 ** -7 * clean[keep].double().abs() + 2.0 ** -12 * clean.double().abs().max()).all()


@pytest.mark.parametrize("T,fmt", [(1, "awq_om"), (16, "fp8"), (4, "bf16")])
def test_replays_of_a_captured_call(T, fmt):
    x, router, bank, shared = _make(T, 512, 32, 4, 128, 64, fmt)
    few = moe.FewTokenLayer(router, 4, bank, shared, max_tokens=T)
    other = moe.FewTokenLayer(router, 4, bank, shared, max_tokens=T)
    y, idx = few(x)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        few(x, y=y, topk_idx=idx)
    for i in range(5):
        x.copy_(torch.randn(x.shape, generator=torch.Generator().manual_seed(i)).bfloat16())
        graph.replay()
        torch.cuda.synchronize()
        want, widx = other(x)
        assert torch.equal(y, want) and torch.equal(idx, widx)


def test_two_streams_at_once():
    """Calls on two streams with workspaces of their own; each waits only for what it started itself."""
    x, router, bank, shared = _make(16, 2560, 128, 10, 640, 640, "fp8")
    few = [moe.FewTokenLayer(router, 10, bank, shared) for _ in range(2)]
    want, widx = few[0](x)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    out = [[], []]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for i in range(10):
        for j in range(2):
            with torch.cuda.stream(streams[j]):
                out[j].append(few[j](x))
    torch.cuda.synchronize()
    for j in range(2):
        for y, idx in out[j]:
            assert torch.equal(y, want) and torch.equal(idx, widx)


def test_every_list_at_its_largest():
    """16 tokens of 64 among 1024 experts: the most pairs, touched experts and LDS of a call."""
    x, router, bank, shared = _make(16, 256, 1024, 64, 128, 32, "bf16")
    y, idx = moe.layer_few(x, router, 64, bank, shared)
    _check(y, idx, R.layer(x, router, 64, bank, shared))


def test_calls_without_a_workspace_on_two_streams():
    x, router, bank, shared = _make(16, 1024, 64, 6, 256, 64, "fp8")
    want, widx = moe.layer_few(x, router, 6, bank, shared)
    made_here = moe.FewTokenLayer(router, 6, bank, shared)
    streams = [torch.cuda.Stream() for _ in range(2)]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    out = []
    for i in range(10):
        for s in streams:
            with torch.cuda.stream(s):
                out.append(moe.layer_few(x, router, 6, bank, shared))
    with torch.cuda.stream(streams[1]):
        out.append(made_here(x))
    del made_here
    torch.cuda.synchronize()
    for y, idx in out:
        assert torch.equal(y, want) and torch.equal(idx, widx)


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "awq_om"])
def test_agrees_with_the_layer_of_separate_kernels(fmt):
    """moe_layer rounds h and the experts' rows to bf16: three roundings of 2^-8 on the way, of terms that
    add up to at most the sum of their magnitudes."""
    T, H, E, k, F = 8, 512, 64, 6, 256
    x, router, bank, shared = _make(T, H, E, k, F, 256, fmt)
    idx0 = torch.empty((T, k), dtype=torch.int32, device=DEV)
    y0 = moe.layer(x, router, k, bank, shared, topk_idx=idx0)
    y, idx = moe.layer_few(x, router, k, bank, shared)
    assert torch.equal(idx, idx0)
    a, b = y.double(), y0.double()
    assert (a - b).norm() <= 3 * 2.0 ** -8 * a.norm()


@pytest.mark.parametrize("name", ["gate", "up", "down"])
@pytest.mark.parametrize("bad", ["nan", "inf"])
@pytest.mark.parametrize("T,fmt", [(4, "bf16"), (4, "fp8"), (4, "awq_om"), (16, "bf16"), (16, "fp8"), (16, "awq_om")])
def test_weights_that_are_no_numbers_reach_only_their_tokens(T, fmt, bad, name):
    """A NaN or an infinity in one expert's weights or scales shows in the tokens routed to it; the others keep their
    bits (the expert's share of them is no part of their sums, not zero times its weights)."""
    x, router, bank, shared = _make(T, 512, 32, 2, 256, 64, fmt, seed=T)
    clean, idx = moe.layer_few(x, router, 2, bank, shared)
    e = int(idx[0, 0])
    hit = (idx == e).any(1)
    assert hit.any() and not hit.all()
    if fmt == "bf16":
        bank[name][e, 3, 5] = float(bad)
    elif fmt == "fp8" and bad == "nan":
        bank[name + "_codes"][e, 3, 5] = 0x7F
    elif fmt == "fp8":
        bank[name + "_bscales"][e, 0, 0] = float(bad)
    else:
        bank[name + "_scales"][e, 0, 3] = float(bad)
    y, idx2 = moe.layer_few(x, router, 2, bank, shared)
    assert torch.equal(idx, idx2)
    assert (~torch.isfinite(y[hit])).any(1).all()
    assert torch.equal(y[~hit], clean[~hit])


def test_the_workspace_of_a_layer_made_behind_pending_work():
    """The workspace takes memory that work on the current stream still reads; the first call, on another stream,
    leaves that work its values."""
    x, router, bank, shared = _make(16, 512, 32, 4, 128, 64, "fp8")
    want, _ = moe.layer_few(x, router, 4, bank, shared)
    n = moe.FewTokenLayer(router, 4, bank, shared).ws_buf.numel()
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    m = torch.randn((4096, 4096), device=DEV)
    torch.cuda.synchronize()
    for _ in range(3):
        with torch.cuda.stream(a):
            old = torch.full((n,), 5, dtype=torch.uint8, device=DEV)
            for _ in range(20):
                m = (m @ m).clamp(-1, 1)           # some ms of work
            kept = old.clone()
            del old
            few = moe.FewTokenLayer(router, 4, bank, shared)
        with torch.cuda.stream(b):
            y, _ = few(x)
        torch.cuda.synchronize()
        assert (kept == 5).all() and torch.equal(y, want)


def test_one_layer_on_two_streams_in_turn():
    x, router, bank, shared = _make(16, 1024, 64, 6, 256, 64, "fp8")
    xs = [x, x.flip(0).contiguous()]
    few = moe.FewTokenLayer(router, 6, bank, shared)
    want = [moe.layer_few(v, router, 6, bank, shared) for v in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    out = []
    for i in range(20):
        with torch.cuda.stream(streams[i % 2]):
            out.append(few(xs[i % 2]))
    torch.cuda.synchronize()
    for i, (y, idx) in enumerate(out):
        assert torch.equal(y, want[i % 2][0]) and torch.equal(idx, want[i % 2][1])
