"""Cases of the FP8 products and of the few-token layer: what is timed, on which inputs, and the plain form of each operator.

Four operators, all of them forward passes of a serving path:
  quantize: rows of activations to E4M3 codes with one fp32 scale per 128 values
  matmul:   the product of two E4M3 matrices, scales per 128 inputs (rows) and per 128 x 128 block (weights)
  ffn_a8:   grouped SwiGLU experts on those products, activations quantised before each of them
  few:      a whole routed layer (router, top-k, experts, shared expert, weighted sum) for at most 16 tokens

`own` selects the framework's kernels; otherwise run() computes the same with elementary torch operations in fp32.
"""
import math

import torch

own = False

E4M3 = torch.float8_e4m3fn
TINY = 448.0 * 2.0 ** -126      # smallest largest-magnitude a group of 128 is scaled by
NIBBLE = (0, 2, 4, 6, 1, 3, 5, 7)  # column of nibble j of a packed AWQ zero word
LARGEST = {"quantize": 32768 * 2560, "matmul": 8192 ** 3, "ffn_a8": 32768 * 10 * 2560 * 640, "few": 16 * 10 * 3 * 2560 * 640}


def listed():
    return [
        # one token's hidden state before a projection: latency
        {"name": "quantize_1x2560", "op": "quantize", "T": 1, "n": 2560, "dtype": "bf16"},
        # an odd number of rows whose last group holds 48 values, from an fp32 intermediate
        {"name": "quantize_4097x688_f32", "op": "quantize", "T": 4097, "n": 688, "dtype": "f32"},
        # one packed row of prefill at full width
        {"name": "quantize_32768x2560", "op": "quantize", "T": 32768, "n": 2560, "dtype": "bf16"},
        # one token through a hidden x hidden projection: the weights' bytes count
        {"name": "matmul_1x2560x2560", "op": "matmul", "M": 1, "N": 2560, "K": 2560, "out": "bf16"},
        # a ragged decode batch, an output width and a depth that end inside a block
        {"name": "matmul_77x1000x1296_f32", "op": "matmul", "M": 77, "N": 1000, "K": 1296, "out": "f32"},
        # gate and up of the shared expert over a prefill batch
        {"name": "matmul_4096x1280x2560", "op": "matmul", "M": 4096, "N": 1280, "K": 2560, "out": "bf16"},
        # a large square product: the matrix cores' rate
        {"name": "matmul_8192x8192x8192", "op": "matmul", "M": 8192, "N": 8192, "K": 8192, "out": "bf16"},
        # a decode step: few rows per expert, the touched experts' bytes count
        {"name": "ffn_a8_16_of_512", "op": "ffn_a8", "T": 16, "H": 2560, "F": 640, "E": 512, "k": 10, "skew": 0.0},
        # a prefill batch, 80 rows per expert on average, some experts with several times that
        {"name": "ffn_a8_4096_of_512", "op": "ffn_a8", "T": 4096, "H": 2560, "F": 640, "E": 512, "k": 10, "skew": 0.5},
        # one packed row over a pruned bank, 1280 rows per expert on average
        {"name": "ffn_a8_32768_of_256", "op": "ffn_a8", "T": 32768, "H": 2560, "F": 640, "E": 256, "k": 10, "skew": 0.0},
        # one user's token on 4-bit experts: latency
        {"name": "few_1_awq", "op": "few", "T": 1, "H": 2560, "F": 640, "E": 512, "k": 10, "Fs": 640, "fmt": "awq_om"},
        # the largest few-token batch on FP8 experts
        {"name": "few_16_fp8", "op": "few", "T": 16, "H": 2560, "F": 640, "E": 512, "k": 10, "Fs": 640, "fmt": "fp8"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    while True:
        op = rng.choice(["quantize", "matmul", "ffn_a8", "few"])
        if op == "quantize":
            c = {"op": op, "T": _log(rng, 1, 32768), "n": 16 * _log(rng, 1, 512), "dtype": rng.choice(["bf16", "f32"])}
            size = c["T"] * c["n"]
        elif op == "matmul":
            c = {"op": op, "M": _log(rng, 1, 32768), "N": _log(rng, 1, 8192), "K": 16 * _log(rng, 1, 512),
                 "out": rng.choice(["bf16", "f32"])}
            size = c["M"] * c["N"] * c["K"]
        elif op == "ffn_a8":
            E = _log(rng, 1, 512)
            c = {"op": op, "T": _log(rng, 1, 32768), "H": 128 * rng.randint(1, 20), "F": 128 * rng.randint(1, 5), "E": E,
                 "k": rng.randint(1, min(10, E)), "skew": rng.choice([0.0, 0.5, 1.0])}
            size = c["T"] * c["k"] * c["H"] * c["F"]
        else:
            E = _log(rng, 2, 512)
            c = {"op": op, "T": rng.randint(1, 16), "H": 256 * rng.randint(1, 10), "F": 128 * rng.randint(1, 5), "E": E,
                 "k": rng.randint(1, min(10, E)), "Fs": 128 * rng.randint(0, 5), "fmt": rng.choice(["bf16", "fp8", "awq_om"])}
            size = c["T"] * c["k"] * 3 * c["H"] * c["F"]
        if size <= LARGEST[op]:
            return c


# ------------------------------------------------------------------ inputs

def _gen(seed, tid):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 1_000_003 + tid)
    return g


def _activations(T, n, seed):
    """N(0, 1) with a few channels of larger magnitude, as hidden states have them."""
    g = _gen(seed, 1)
    x = torch.randn((T, n), generator=g, device="cuda")
    x *= 1.0 + 7.0 * (torch.rand(n, generator=g, device="cuda") > 0.98)
    return x


def _fp8_matrix(E, O, I, seed, tid):
    """N(0, 0.02) weights as E4M3 codes with one fp32 scale per 128 x 128 block (codes uint8 [E, O, I])."""
    g = _gen(seed, tid)
    codes = torch.empty((E, O, I), dtype=torch.uint8, device="cuda")
    ob, ib = -(-O // 128), -(-I // 128)
    scales = torch.empty((E, ob, ib), device="cuda")
    step = max(1, (1 << 28) // (O * I))
    for e in range(0, E, step):
        n = min(step, E - e)
        w = torch.randn((n, ob * 128, ib * 128), generator=g, device="cuda") * 0.02
        w[:, O:] = 0
        w[:, :, I:] = 0
        b = w.view(n, ob, 128, ib, 128)
        s = b.abs().amax(dim=(2, 4)) / 448.0
        q = (b / s[:, :, None, :, None]).view(n, ob * 128, ib * 128)[:, :O, :I]
        codes[e:e + n] = q.to(E4M3).view(torch.uint8)
        scales[e:e + n] = s
    return codes, scales


def _normal(shape, seed, tid):
    g = _gen(seed, tid)
    out = torch.empty(shape, dtype=torch.bfloat16, device="cuda")
    step = max(1, (1 << 28) // max(1, out[0].numel()))
    for e in range(0, shape[0], step):
        out[e:e + step] = torch.randn(out[e:e + step].shape, generator=g, device="cuda") * 0.02
    return out


def _words(shape, g):
    return torch.randint(-2 ** 31, 2 ** 31, shape, generator=g, device="cuda", dtype=torch.int64).to(torch.int32)


def _bank(fmt, E, H, F, seed):
    out = {"fmt": fmt}
    for j, (name, o, i) in enumerate((("gate", F, H), ("up", F, H), ("down", H, F))):
        if fmt == "bf16":
            out[name] = _normal((E, o, i), seed, 10 + j)
        elif fmt == "fp8":
            out[name + "_codes"], out[name + "_bscales"] = _fp8_matrix(E, o, i, seed, 20 + j)
        else:  # 4-bit codes, eight consecutive inputs of a column in a word
            g = _gen(seed, 30 + j)
            out[name + "_qweight"] = _words((E, o, i // 8), g)
            out[name + "_qzeros"] = _words((E, i // 32, o // 8), g)
            out[name + "_scales"] = (torch.randn((E, i // 32, o), generator=g, device="cuda") * 0.002).abs().add(1e-4).half()
    return out


def prepare(case, seed):
    op = case["op"]
    st = {"op": op}
    if op == "quantize":
        T, n = case["T"], case["n"]
        st["x"] = _activations(T, n, seed).to(torch.float32 if case["dtype"] == "f32" else torch.bfloat16)
        st["codes"] = torch.empty((T, n), dtype=torch.uint8, device="cuda")
        st["scales"] = torch.empty((T, -(-n // 128)), device="cuda")
    elif op == "matmul":
        M, N, K = case["M"], case["N"], case["K"]
        st["a"], st["sa"] = _quantize(_activations(M, K, seed).bfloat16())
        w, sw = _fp8_matrix(1, N, K, seed, 2)
        st["w"], st["sw"] = w[0], sw[0]
        st["dtype"] = torch.float32 if case["out"] == "f32" else torch.bfloat16
        st["y"] = torch.empty((M, N), dtype=st["dtype"], device="cuda")
    elif op == "ffn_a8":
        T, H, F, E, k = (case[v] for v in ("T", "H", "F", "E", "k"))
        st["x"], st["k"] = _activations(T, H, seed).bfloat16(), k
        st["bank"] = _bank("fp8", E, H, F, seed)
        # the routing that comes before: `skew` spreads the experts' loads
        g = _gen(seed, 3)
        score = torch.randn((T, E), generator=g, device="cuda") + case["skew"] * torch.randn(E, generator=g, device="cuda")
        idx = score.topk(k, dim=1).indices.reshape(-1)
        st["sorted_pair"] = torch.sort(idx, stable=True).indices.int()
        count = torch.bincount(idx, minlength=E)
        st["offsets"] = torch.cat([count.new_zeros(1), count.cumsum(0)]).int()
        st["cap"] = int(count.max())
        st["rows"] = torch.empty((T * k, H), dtype=torch.bfloat16, device="cuda")
        if own:  # the workspace that a serving program keeps
            import sparse_moe_expert_router_amd as moe
            st["ws"] = moe.Workspace(st["x"].device)
    else:
        T, H, F, E, k, Fs = (case[v] for v in ("T", "H", "F", "E", "k", "Fs"))
        st["x"], st["k"] = torch.randn((T, H), generator=_gen(seed, 1), device="cuda").bfloat16(), k
        st["router"] = _normal((E, H), seed, 2)
        st["bank"] = _bank(case["fmt"], E, H, F, seed)
        st["shared"] = _bank("bf16", 1, H, Fs, seed + 500_000) if Fs else None
        if own:  # the handle of the layer: its weights' addresses and its workspace
            import sparse_moe_expert_router_amd as moe
            st["layer"] = moe.FewTokenLayer(st["router"], k, st["bank"], st["shared"])
    return st


# ------------------------------------------------------------------ plain forms

def _quantize(x):
    """E4M3 codes (uint8) and fp32 scales of the rows of x, per 128 values."""
    T, n = x.shape
    nb = -(-n // 128)
    b = torch.nn.functional.pad(x.float(), (0, nb * 128 - n)).view(T, nb, 128)
    amax = b.abs().amax(-1).clamp(min=TINY)
    scales = amax / torch.full_like(amax, 448.0)  # by a tensor: torch multiplies by the rounded reciprocal of a number
    codes = (b / scales[..., None]).to(E4M3).view(torch.uint8).view(T, nb * 128)[:, :n]
    return codes.contiguous(), scales


def _rows32(codes, scales):
    """fp32 values of quantised rows."""
    n = codes.shape[-1]
    return codes.view(E4M3).float() * scales.repeat_interleave(128, -1)[..., :n]


def _blocks32(codes, scales):
    """fp32 values of [.., O, I] codes with 128 x 128 block scales."""
    O, I = codes.shape[-2:]
    s = scales.repeat_interleave(128, -2)[..., :O, :].repeat_interleave(128, -1)[..., :I]
    return codes.view(E4M3).float() * s


def _silu(a):
    return a / (1.0 + torch.exp(-a))


def _plain_ffn_a8(st):
    x, k, bank, off, cap = st["x"], st["k"], st["bank"], st["offsets"].long(), st["cap"]
    P, H = x.shape[0] * k, x.shape[1]
    E = off.numel() - 1
    xq = _rows32(*_quantize(x))
    codes, scales = ({n: bank[n + v] for n in ("gate", "up", "down")} for v in ("_codes", "_bscales"))
    if P < E:  # few rows: each row with its own expert's weights, the other experts are not read
        r = torch.arange(P, device=x.device)[:, None]
        valid = torch.ones_like(r, dtype=torch.bool)
        e = torch.bucketize(r[:, 0], off[1:], right=True)
        codes, scales = ({n: v[e] for n, v in d.items()} for d in (codes, scales))
        E, cap = P, 1
    else:  # every expert's rows, padded to the largest expert's number
        r = off[:-1, None] + torch.arange(cap, device=x.device)
        valid = r < off[1:, None]
    token = st["sorted_pair"].long()[r.clamp(max=P - 1)] // k
    a = xq[token] * valid[..., None]
    w = {n: _blocks32(codes[n], scales[n]) for n in codes}
    g = torch.matmul(a, w["gate"].transpose(1, 2).contiguous())
    u = torch.matmul(a, w["up"].transpose(1, 2).contiguous())
    h = _silu(g) * u
    F = h.shape[-1]
    hq = _rows32(*_quantize(h.view(E * cap, F))).view(E, cap, F)
    o = torch.matmul(hq, w["down"].transpose(1, 2).contiguous())
    rows = torch.zeros((P + 1, H), dtype=torch.bfloat16, device=x.device)
    rows[torch.where(valid, r, P)] = o.bfloat16()
    return rows[:P]


def _weights32(bank, name, e):
    """fp32 [.., O, I] weights of the experts e (any index tensor)."""
    if bank["fmt"] == "bf16":
        return bank[name][e].float()
    if bank["fmt"] == "fp8":
        return _blocks32(bank[name + "_codes"][e], bank[name + "_bscales"][e])
    shift = torch.arange(0, 32, 4, device=e.device, dtype=torch.int32)
    q = (bank[name + "_qweight"][e][..., None] >> shift & 15).flatten(-2)                  # [.., O, I]
    order = torch.tensor([NIBBLE.index(c) for c in range(8)], device=e.device)
    z = (bank[name + "_qzeros"][e][..., None] >> shift[order] & 15).flatten(-2)            # [.., I/32, O]
    s = bank[name + "_scales"][e].float()
    z, s = (v.transpose(-1, -2).repeat_interleave(32, -1) for v in (z, s))
    return (q - z).float() * s


def _plain_few(st):
    x, k = st["x"], st["k"]
    # logits: the rounded fp32 of the exact sums, which fp32 sums would not give
    logits = (x.double() @ st["router"].double().t()).float()
    top, idx = torch.sort(logits, dim=1, descending=True, stable=True)
    top, idx = top[:, :k], idx[:, :k]
    p = torch.exp(top - top[:, :1])
    gate = p / p.sum(1, keepdim=True)
    xf = x.float()
    g = (_weights32(st["bank"], "gate", idx) * xf[:, None, None, :]).sum(-1)
    u = (_weights32(st["bank"], "up", idx) * xf[:, None, None, :]).sum(-1)
    h = _silu(g) * u * gate[..., None]
    y = (_weights32(st["bank"], "down", idx) * h[:, :, None, :]).sum((-1, 1))
    if st["shared"] is not None:
        one = {n: st["shared"][n][0].float() for n in ("gate", "up", "down")}
        y = y + (_silu(xf @ one["gate"].t()) * (xf @ one["up"].t())) @ one["down"].t()
    return {"y": y.bfloat16(), "idx": idx.int()}


def run(st):
    op = st["op"]
    if op == "quantize":
        if own:
            import sparse_moe_expert_router_amd as moe
            moe.fp8_quantize(st["x"], codes=st["codes"], scales=st["scales"])
            return {"values": st["codes"].view(E4M3), "scales": st["scales"]}
        codes, scales = _quantize(st["x"])
        return {"values": codes.view(E4M3), "scales": scales}
    if op == "matmul":
        if own:
            import sparse_moe_expert_router_amd as moe
            return moe.fp8_matmul(st["a"], st["sa"], st["w"], st["sw"], y=st["y"])
        return (_rows32(st["a"], st["sa"]) @ _blocks32(st["w"], st["sw"]).t()).to(st["dtype"])
    if op == "ffn_a8":
        if own:
            import sparse_moe_expert_router_amd as moe
            return moe.grouped_ffn_a8(st["x"], st["k"], st["bank"], st["offsets"], st["sorted_pair"], ws=st["ws"],
                                      rows=st["rows"])
        return _plain_ffn_a8(st)
    if own:
        y, idx = st["layer"](st["x"])
        return {"y": y, "idx": idx}
    return _plain_few(st)


def work(case):
    op = case["op"]
    if op == "quantize":
        T, n = case["T"], case["n"]
        return {"bytes": T * n * (5 if case["dtype"] == "f32" else 3) + 4 * T * -(-n // 128), "flops": 3 * T * n}
    if op == "matmul":
        M, N, K = case["M"], case["N"], case["K"]
        kb = -(-K // 128)
        return {"bytes": M * K + N * K + 4 * kb * (M + -(-N // 128)) + M * N * (4 if case["out"] == "f32" else 2),
                "flops": 2 * M * N * K}
    T, H, F, E, k = (case[v] for v in ("T", "H", "F", "E", "k"))
    touched = E * (1.0 - (1.0 - k / E) ** T)  # of uniform routing
    n = 3 * H * F
    if op == "ffn_a8":
        return {"bytes": int(touched * (n + 4 * n / 16384) + 2 * T * H + 2 * T * k * H), "flops": 2 * T * k * n}
    each = {"bf16": 2 * n, "fp8": n + 4 * n / 16384, "awq_om": n / 2 + 2 * n / 32 + n / 64}[case["fmt"]]
    ns = 3 * H * case["Fs"]
    return {"bytes": int(touched * each + 2 * ns + 2 * E * H + 4 * T * H + 4 * T * k), "flops": 2 * T * (k * n + ns + E * H)}


# ------------------------------------------------------------------ from the definitions, in 64 bits

def _decode64(codes):
    """Values of E4M3 codes from their bits: sign, 4 exponent bits (bias 7), 3 mantissa bits."""
    c = codes.long()
    ex, m = c >> 3 & 15, (c & 7).double()
    v = torch.where(ex == 0, m * 2.0 ** -9, (8.0 + m) * torch.exp2((ex - 10).double()))
    return torch.where(c >= 128, -v, v)


def _round_e4m3(q):
    """Nearest E4M3 value of |q| <= 448, ties to even: the step is 2^(exponent - 3), at least 2^-9."""
    step = torch.exp2(torch.frexp(q)[1].sub(4).clamp(min=-9).double())
    return torch.round(q / step) * step


def _quantized64(x):
    """The values the quantiser's codes stand for, and its scales.  The scale and the quotient are fp32 numbers by definition."""
    x = x.double()
    T, n = x.shape
    values, scales = torch.empty_like(x), []
    for i in range(0, n, 128):
        part = x[:, i:i + 128]
        s = (part.abs().max(1).values.clamp(min=TINY) / 448.0).float().double()
        values[:, i:i + 128] = _round_e4m3((part / s[:, None]).float().double())
        scales.append(s)
    return values, torch.stack(scales, 1)


def _times(values, scales):
    out = values.clone()
    for i in range(scales.shape[-1]):
        out[:, 128 * i:128 * i + 128] *= scales[:, i:i + 1]
    return out


def _block64(codes, scales):
    """[O, I] codes to values, block by block."""
    out = _decode64(codes)
    for o in range(scales.shape[0]):
        out[128 * o:128 * o + 128] = _times(out[128 * o:128 * o + 128], scales[o:o + 1].double().expand(out[128 * o:128 * o + 128].shape[0], -1))
    return out


def _swiglu64(g, u):
    return g * torch.sigmoid(g) * u


def _expert64(bank, e):
    out = []
    for name in ("gate", "up", "down"):
        if bank["fmt"] == "bf16":
            out.append(bank[name][e].double())
        elif bank["fmt"] == "fp8":
            out.append(_block64(bank[name + "_codes"][e], bank[name + "_bscales"][e]))
        else:
            qw, qz, s = (bank[name + v][e].long() if v != "_scales" else bank[name + v][e].double()
                         for v in ("_qweight", "_qzeros", "_scales"))
            O, I = qw.shape[0], qw.shape[1] * 8
            q = torch.empty((O, I), dtype=torch.float64, device=qw.device)
            z = torch.empty((I // 32, O), dtype=torch.float64, device=qw.device)
            for j in range(8):
                q[:, j::8] = (qw >> 4 * j & 15).double()
                z[:, NIBBLE[j]::8] = (qz >> 4 * j & 15).double()
            for b in range(I // 32):
                q[:, 32 * b:32 * b + 32] = (q[:, 32 * b:32 * b + 32] - z[b, :, None]) * s[b, :, None]
            out.append(q)
    return out


def exact(case, seed):
    st = prepare(case, seed)
    op = st["op"]
    if op == "quantize":
        values, scales = _quantized64(st["x"])
        return {"values": values, "scales": scales}
    if op == "matmul":
        return _times(_decode64(st["a"]), st["sa"].double()) @ _block64(st["w"], st["sw"]).t()
    if op == "ffn_a8":
        xq = _times(*_quantized64(st["x"]))
        off = st["offsets"].tolist()
        rows = torch.zeros((st["rows"].shape[0], xq.shape[1]), dtype=torch.float64, device=xq.device)
        for e in range(len(off) - 1):
            if off[e] == off[e + 1]:
                continue
            a = xq[st["sorted_pair"][off[e]:off[e + 1]].long() // st["k"]]
            gate, up, down = _expert64(st["bank"], e)
            h = _swiglu64(a @ gate.t(), a @ up.t())
            rows[off[e]:off[e + 1]] = _times(*_quantized64(h)) @ down.t()
        return rows
    x, k = st["x"].double(), st["k"]
    logits = (x @ st["router"].double().t()).float().double()
    y = torch.zeros_like(x)
    chosen = []
    for t in range(x.shape[0]):
        order = sorted(range(logits.shape[1]), key=lambda e, v=logits[t].tolist(): (-v[e], e))[:k]
        chosen.append(order)
        gate = torch.softmax(logits[t, order], 0)
        for j, e in enumerate(order):
            wg, wu, wd = _expert64(st["bank"], e)
            y[t] += gate[j] * (wd @ _swiglu64(wg @ x[t], wu @ x[t]))
    if st["shared"] is not None:
        wg, wu, wd = _expert64(st["shared"], 0)
        y += _swiglu64(x @ wg.t(), x @ wu.t()) @ wd.t()
    return {"y": y, "idx": torch.tensor(chosen, dtype=torch.int32, device=x.device)}
