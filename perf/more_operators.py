"""Cases of the operators around the routed layer: what is timed, on which inputs, and the plain form of each operator.

  norm:      residual addition and root-mean-square norm, to bf16 rows and / or E4M3 codes with one scale per 128 values
  norm_bwd:  its gradients: of the rows (those of the residual added) and of the gain
  balance:   per-expert counts of a routed batch, its balance loss, and the gradient of the router's logits (through the
             gates too, where their gradient is given)
  awq:       the product of few bf16 rows with a 4-bit AWQ matrix, scales and zeros per group of inputs

`own` selects the framework's kernels; otherwise run() computes the same with elementary torch operations in fp32.
"""
import math

import torch

own = False

E4M3 = torch.float8_e4m3fn
TINY = 448.0 * 2.0 ** -126      # smallest largest-magnitude a group of 128 is scaled by
COLUMN = (0, 2, 4, 6, 1, 3, 5, 7)  # column of nibble j of a packed AWQ word
EPS = 1e-6
DTYPE = {"bf16": torch.bfloat16, "f32": torch.float32}
LARGEST = {"norm": 32768 * 2560, "norm_bwd": 32768 * 2560, "balance": 32768 * 512, "awq": 16 * 16384 * 16384}


def listed():
    return [
        # one token's hidden state between two blocks of a decode step: latency
        {"name": "norm_1x2560", "op": "norm", "T": 1, "H": 2560, "x": "bf16", "res": "bf16", "out": "y"},
        # an odd number of rows, an fp32 residual stream, a last group of 48 values, bf16 rows and codes both
        {"name": "norm_4097x688_f32", "op": "norm", "T": 4097, "H": 688, "x": "bf16", "res": "f32", "out": "both"},
        # one packed row of prefill at full width, straight to codes
        {"name": "norm_32768x2560_fp8", "op": "norm", "T": 32768, "H": 2560, "x": "bf16", "res": "bf16", "out": "fp8"},
        # a small ragged training batch in fp32, no other gradient of the residual
        {"name": "norm_bwd_515x688_f32", "op": "norm_bwd", "T": 515, "H": 688, "dtype": "f32", "dres": False},
        # a packed row of training at full width, with the gradient that the residual stream brings
        {"name": "norm_bwd_32768x2560", "op": "norm_bwd", "T": 32768, "H": 2560, "dtype": "bf16", "dres": True},
        # a decode-sized batch: latency
        {"name": "balance_16_of_512", "op": "balance", "T": 16, "E": 512, "k": 10, "dtype": "f32", "valid": 1.0, "gates": False},
        # few experts, an odd number of them, bf16 logits, padded tokens, and the gates' gradient
        {"name": "balance_8191_of_61_bf16", "op": "balance", "T": 8191, "E": 61, "k": 6, "dtype": "bf16", "valid": 0.9, "gates": True},
        # a packed row of training over all experts, the whole gradient of the router's logits
        {"name": "balance_32768_of_512", "op": "balance", "T": 32768, "E": 512, "k": 10, "dtype": "f32", "valid": 1.0, "gates": True},
        # one token through a hidden x hidden projection: latency
        {"name": "awq_1x2560x2560", "op": "awq", "M": 1, "N": 2560, "K": 2560, "group": 32, "out": "bf16"},
        # a ragged decode batch, an output width that ends inside a tile, fp32 sums
        {"name": "awq_13x1000x1312_f32", "op": "awq", "M": 13, "N": 1000, "K": 1312, "group": 32, "out": "f32"},
        # one token through a large projection: the weights' bytes count
        {"name": "awq_1x8192x8192", "op": "awq", "M": 1, "N": 8192, "K": 8192, "group": 128, "out": "bf16"},
        # a decode batch through the largest projection
        {"name": "awq_16x16384x16384", "op": "awq", "M": 16, "N": 16384, "K": 16384, "group": 32, "out": "bf16"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    while True:
        op = rng.choice(["norm", "norm_bwd", "balance", "awq"])
        if op == "norm":
            c = {"op": op, "T": _log(rng, 1, 32768), "H": 16 * _log(rng, 1, 1024), "x": rng.choice(["bf16", "f32"]),
                 "res": rng.choice(["none", "bf16", "f32"]), "out": rng.choice(["y", "fp8", "both"])}
            size = c["T"] * c["H"] * (2 if "f32" in (c["x"], c["res"]) else 1)
        elif op == "norm_bwd":
            c = {"op": op, "T": _log(rng, 1, 32768), "H": 8 * _log(rng, 1, 2048), "dtype": rng.choice(["bf16", "f32"]),
                 "dres": rng.choice([False, True])}
            size = c["T"] * c["H"] * (2 if c["dtype"] == "f32" else 1)
        elif op == "balance":
            E = _log(rng, 1, 1024)
            c = {"op": op, "T": _log(rng, 1, 65536), "E": E, "k": rng.randint(1, min(16, E)), "dtype": rng.choice(["bf16", "f32"]),
                 "valid": rng.choice([1.0, 0.9, 0.3]), "gates": rng.choice([False, True])}
            size = c["T"] * E
        else:
            group = rng.choice([32, 64, 128])
            c = {"op": op, "M": _log(rng, 1, 64), "N": 8 * _log(rng, 1, 2048), "K": group * _log(rng, 1, 16384 // group),
                 "group": group, "out": rng.choice(["bf16", "f32"])}
            size = c["M"] * c["N"] * c["K"]
        if size <= LARGEST[op]:
            return c


# ------------------------------------------------------------------ inputs

def _gen(seed, tid):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 1_000_003 + tid)
    return g


def _activations(T, n, seed, tid, dtype):
    """N(0, 1) with a few channels of larger magnitude, as hidden states have them."""
    g = _gen(seed, tid)
    x = torch.randn((T, n), generator=g, device="cuda")
    x *= 1.0 + 7.0 * (torch.rand(n, generator=g, device="cuda") > 0.98)
    return x.to(dtype)


def _words(shape, g):
    return torch.randint(-2 ** 31, 2 ** 31, shape, generator=g, device="cuda", dtype=torch.int64).to(torch.int32)


def prepare(case, seed):
    op = case["op"]
    st = {"op": op}
    if op == "norm":
        T, H = case["T"], case["H"]
        st["x"] = _activations(T, H, seed, 1, DTYPE[case["x"]])
        st["residual"] = st["residual_out"] = None
        if case["res"] != "none":
            st["residual"] = _activations(T, H, seed, 2, DTYPE[case["res"]]) * 4
            st["residual_out"] = torch.empty_like(st["residual"])
        st["weight"] = (torch.randn(H, generator=_gen(seed, 3), device="cuda") * 0.1).bfloat16()
        # the buffers that the next call reads
        st["y"] = torch.empty((T, H), dtype=torch.bfloat16, device="cuda") if case["out"] != "fp8" else None
        fp8 = case["out"] != "y"
        st["codes"] = torch.empty((T, H), dtype=torch.uint8, device="cuda") if fp8 else None
        st["scales"] = torch.empty((T, -(-H // 128)), device="cuda") if fp8 else None
    elif op == "norm_bwd":
        T, H = case["T"], case["H"]
        dt = DTYPE[case["dtype"]]
        st["s"] = _activations(T, H, seed, 1, dt)
        st["rstd"] = 1.0 / torch.sqrt(st["s"].float().square().mean(1) + EPS)
        st["weight"] = (torch.randn(H, generator=_gen(seed, 3), device="cuda") * 0.1).to(dt)
        st["dy"] = (torch.randn((T, H), generator=_gen(seed, 4), device="cuda") * 1e-3).to(dt)
        st["dres"] = (torch.randn((T, H), generator=_gen(seed, 5), device="cuda") * 1e-3).to(dt) if case["dres"] else None
        st["dx"] = torch.empty_like(st["s"])
        st["dw"] = torch.empty(H, device="cuda")
        if own:  # the workspace that a training program keeps
            import sparse_moe_expert_router_amd as moe
            st["ws"] = moe.Workspace(st["s"].device)
    elif op == "balance":
        T, E, k = case["T"], case["E"], case["k"]
        g = _gen(seed, 1)
        # logits of a router that prefers some experts
        logits = torch.randn((T, E), generator=g, device="cuda") + 0.5 * torch.randn(E, generator=g, device="cuda")
        st["logits"], st["k"], st["coef"] = logits.to(DTYPE[case["dtype"]]), k, 1e-2
        st["valid"] = None
        if case["valid"] < 1.0:
            st["valid"] = (torch.rand(T, generator=g, device="cuda") < case["valid"]).to(torch.uint8)
        top, idx = torch.sort(st["logits"].float(), dim=1, descending=True, stable=True)
        st["idx"] = idx[:, :k].int().contiguous()
        st["gate"] = st["dgate"] = None
        if case["gates"]:
            p = torch.exp(top[:, :k] - top[:, :1])
            st["gate"] = (p / p.sum(1, keepdim=True)).contiguous()
            st["dgate"] = torch.randn((T, k), generator=g, device="cuda") / T
        st["counts"] = torch.empty(E, dtype=torch.int32, device="cuda")
        st["dlogits"] = torch.empty_like(st["logits"])
        if own:
            import sparse_moe_expert_router_amd as moe
            st["ws"] = moe.Workspace(st["logits"].device)
    else:
        M, N, K, group = case["M"], case["N"], case["K"], case["group"]
        st["x"] = _activations(M, K, seed, 1, torch.bfloat16)
        g = _gen(seed, 2)
        st["qweight"] = _words((K, N // 8), g)
        st["qzeros"] = _words((K // group, N // 8), g)
        st["scales"] = (torch.randn((K // group, N), generator=g, device="cuda") * 0.002).abs().add(1e-4).half()
        st["y"] = torch.empty((M, N), dtype=DTYPE[case["out"]], device="cuda")
        if own:
            import sparse_moe_expert_router_amd as moe
            st["ws"] = moe.Workspace(st["x"].device)
    return st


# ------------------------------------------------------------------ plain forms

def _plain_norm(st):
    x, res = st["x"].float(), st["residual"]
    out = {}
    if res is not None:
        out["residual"] = (x + res.float()).to(res.dtype)
        x = out["residual"].float()
    v = x / torch.sqrt((x * x).mean(1, keepdim=True) + EPS) * (1.0 + st["weight"].float())
    if st["y"] is not None:
        out["y"] = v.bfloat16()
    if st["codes"] is not None:
        T, n = v.shape
        nb = -(-n // 128)
        b = torch.nn.functional.pad(v, (0, nb * 128 - n)).view(T, nb, 128)
        amax = b.abs().amax(-1).clamp(min=TINY)
        scales = amax / torch.full_like(amax, 448.0)
        out["values"] = (b / scales[..., None]).to(E4M3).view(T, nb * 128)[:, :n].contiguous()
        out["scales"] = scales
    return out


def _plain_norm_bwd(st):
    r = st["rstd"][:, None]
    h, dy = st["s"].float() * r, st["dy"].float()
    u = dy * (1.0 + st["weight"].float())
    dx = r * (u - h * (u * h).mean(1, keepdim=True))
    if st["dres"] is not None:
        dx = dx + st["dres"].float()
    return {"dx": dx.to(st["dx"].dtype), "dw": (dy * h).sum(0)}


def _plain_balance(st):
    logits, k = st["logits"].float(), st["k"]
    T, E = logits.shape
    valid = torch.ones(T, device=logits.device) if st["valid"] is None else st["valid"].float()
    chosen = (st["idx"].long()[..., None] == torch.arange(E, device=logits.device)) & (valid[:, None, None] > 0)
    counts = chosen.sum((0, 1))
    total = counts.sum().clamp(min=1)
    f = counts.float() / total.float()
    p = torch.exp(logits - logits.amax(1, keepdim=True))
    p = p / p.sum(1, keepdim=True) * valid[:, None]
    prob_sum = p.sum(0)
    a = st["coef"] * E * k / total.float()
    d = a * p * (f - (f * p).sum(1, keepdim=True))
    if st["dgate"] is not None:
        g, dg = st["gate"], st["dgate"]
        v = g * (dg - (g * dg).sum(1, keepdim=True))
        d = d + (chosen * v[..., None]).sum(1)
    return {"counts": counts.int(), "loss": (a * (f * prob_sum).sum()).view(1), "prob_sum": prob_sum, "dlogits": d.to(st["logits"].dtype)}


def _plain_awq(st):
    qw, qz, s = st["qweight"], st["qzeros"], st["scales"].float()
    K, group = qw.shape[0], qw.shape[0] // qz.shape[0]
    shift = torch.tensor([4 * COLUMN.index(c) for c in range(8)], device=qw.device, dtype=torch.int32)
    q = (qw[..., None] >> shift & 15).flatten(1)
    z = (qz[..., None] >> shift & 15).flatten(1)
    w = (q - z.repeat_interleave(group, 0)).float() * s.repeat_interleave(group, 0)
    return (st["x"].float() @ w).to(st["y"].dtype)


def run(st):
    op = st["op"]
    if not own:
        return {"norm": _plain_norm, "norm_bwd": _plain_norm_bwd, "balance": _plain_balance, "awq": _plain_awq}[op](st)
    import sparse_moe_expert_router_amd as moe
    if op == "norm":
        r = moe.add_rmsnorm(st["x"], st["weight"], st["residual"], eps=EPS, gain_offset=1.0, residual_out=st["residual_out"],
                            y=st["y"], codes=st["codes"], scales=st["scales"])
        out = {}
        if st["residual"] is not None:
            out["residual"] = r.residual
        if st["y"] is not None:
            out["y"] = r.y
        if st["codes"] is not None:
            out["values"], out["scales"] = r.codes.view(E4M3), r.scales
        return out
    if op == "norm_bwd":
        dx, dw = moe.add_rmsnorm_backward(st["dy"], st["s"], st["rstd"], st["weight"], gain_offset=1.0, dres=st["dres"],
                                          dx=st["dx"], dw=st["dw"], ws=st["ws"])
        return {"dx": dx, "dw": dw}
    if op == "balance":
        counts = moe.expert_counts(st["idx"], st["logits"].shape[1], token_valid=st["valid"], counts=st["counts"])
        loss, prob_sum, dlogits = moe.balance_loss(st["logits"], counts, st["k"], st["coef"], token_valid=st["valid"],
                                                   topk_idx=st["idx"] if st["dgate"] is not None else None, gate=st["gate"],
                                                   dgate=st["dgate"], dlogits=st["dlogits"], ws=st["ws"])
        return {"counts": counts, "loss": loss, "prob_sum": prob_sum, "dlogits": dlogits}
    return moe.awq_matmul(st["x"], st["qweight"], st["qzeros"], st["scales"], y=st["y"], ws=st["ws"])


def work(case):
    op = case["op"]
    size = {"none": 0, "bf16": 2, "f32": 4}
    if op == "norm":
        T, H = case["T"], case["H"]
        each = size[case["x"]] + 2 * size[case["res"]] + {"y": 2, "fp8": 1, "both": 3}[case["out"]]
        return {"bytes": T * H * each + 2 * H + (0 if case["out"] == "y" else 4 * T * -(-H // 128)), "flops": 6 * T * H}
    if op == "norm_bwd":
        T, H, n = case["T"], case["H"], size[case["dtype"]]
        return {"bytes": T * H * n * (4 if case["dres"] else 3) + 4 * T + (n + 4) * H, "flops": 10 * T * H}
    if op == "balance":
        T, E, k, n = case["T"], case["E"], case["k"], size[case["dtype"]]
        return {"bytes": 2 * n * T * E + 4 * T * k * (3 if case["gates"] else 1) + (T if case["valid"] < 1.0 else 0) + 8 * E,
                "flops": 8 * T * E}
    M, N, K, group = case["M"], case["N"], case["K"], case["group"]
    return {"bytes": K * N // 2 + K // group * N * 5 // 2 + 2 * M * K + size[case["out"]] * M * N, "flops": 2 * M * N * K}


# ------------------------------------------------------------------ from the definitions, in 64 bits

def _round_e4m3(q):
    """Nearest E4M3 value of |q| <= 448, ties to even: the step is 2^(exponent - 3), at least 2^-9."""
    step = torch.exp2(torch.frexp(q)[1].sub(4).clamp(min=-9).double())
    return torch.round(q / step) * step


def _exact_norm(st):
    s = st["x"].double()
    out = {}
    if st["residual"] is not None:
        out["residual"] = s = s + st["residual"].double()
        s = s.to(st["residual"].dtype).double()  # what is normalised is the residual as it is stored
    H = s.shape[1]
    r = torch.rsqrt(s.pow(2).sum(1) / H + EPS)
    v = torch.einsum("th,t,h->th", s, r, st["weight"].double() + 1.0)
    if st["y"] is not None:
        out["y"] = v
    if st["codes"] is not None:
        values, scales = torch.empty_like(v), []
        for i in range(0, H, 128):
            part = v[:, i:i + 128]
            scale = part.abs().max(1).values.clamp(min=TINY) / 448.0
            values[:, i:i + 128] = _round_e4m3(part / scale[:, None])
            scales.append(scale)
        out["values"], out["scales"] = values, torch.stack(scales, 1)
    return out


def _exact_norm_bwd(st):
    s, dy, r = st["s"].double(), st["dy"].double(), st["rstd"].double()[:, None]
    gain = st["weight"].double() + 1.0
    H = s.shape[1]
    # d/ds of s r(s): the identity times r, less the part along s
    along = (dy * gain * s).sum(1, keepdim=True) / H
    dx = r * dy * gain - r ** 3 * s * along
    if st["dres"] is not None:
        dx += st["dres"].double()
    return {"dx": dx, "dw": torch.einsum("th,th,to->h", dy, s, r)}


def _exact_balance(st):
    logits, k, idx = st["logits"].double(), st["k"], st["idx"].long()
    T, E = logits.shape
    keep = torch.ones(T, dtype=torch.bool, device=idx.device) if st["valid"] is None else st["valid"] != 0
    counts = torch.bincount(idx[keep].reshape(-1), minlength=E)
    total = float(counts.sum())
    p = torch.softmax(logits, 1)
    p[~keep] = 0
    d = torch.zeros_like(p)
    loss = torch.zeros(1, dtype=torch.float64, device=idx.device)
    if total:
        f = counts.double() / total
        a = st["coef"] * E * k / total
        loss += a * (f @ p.sum(0))
        d += a * (p * f - p * (p @ f)[:, None])
    if st["dgate"] is not None:
        g, dg = st["gate"].double(), st["dgate"].double()
        v = g * dg - g * (g * dg).sum(1, keepdim=True)
        d.scatter_add_(1, idx, v * keep[:, None])
    return {"counts": counts.int(), "loss": loss, "prob_sum": p.sum(0), "dlogits": d}


def _exact_awq(st):
    qw, qz, s, x = st["qweight"].long(), st["qzeros"].long(), st["scales"].double(), st["x"].double()
    K, N = qw.shape[0], qw.shape[1] * 8
    groups = qz.shape[0]
    n = K // groups
    y = torch.zeros((x.shape[0], N), dtype=torch.float64, device=x.device)
    step = max(1, (1 << 25) // (n * N))
    for g in range(0, groups, step):
        m = min(step, groups - g)
        w = torch.empty((m, n, N), dtype=torch.float64, device=x.device)
        for j, c in enumerate(COLUMN):
            z = qz[g:g + m] >> 4 * j & 15
            w[..., c::8] = ((qw[g * n:(g + m) * n].view(m, n, -1) >> 4 * j & 15) - z[:, None]).double()
        w *= s[g:g + m, None]
        y += x[:, g * n:(g + m) * n] @ w.view(m * n, N)
    return y


def exact(case, seed):
    st = prepare(case, seed)
    return {"norm": _exact_norm, "norm_bwd": _exact_norm_bwd, "balance": _exact_balance, "awq": _exact_awq}[st["op"]](st)
