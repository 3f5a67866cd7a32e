"""Plain 64-bit forms of the FP8 quantiser, the block-scaled product and the W8A8 experts, with bounds on
how far fp32 arithmetic may be from them.  Shares no code with the library.

Bounds.  A product of two E4M3 values has at most 8 significant bits, exact in fp32.

fp32 sums (fp32 outputs): at most 128 roundings per block of 128 products, each off by at most 2^-23 of the
running sum of magnitudes (2^-24 rounded to nearest, twice that truncated); then, per block, the product of
the two scales, the multiplication and the addition, 2^-24 each, and one more addition per block:
  |y - exact| <= (128 + blocks + 3) 2^-23 * sum |p|,   p = a_i w_i sa sw.
FP8 matrix cores (everything else): the 8 products of 8 consecutive inputs are cut below 2^-13 of the
largest one's power of two, so all but that one are off by at most 2^-13 max |p|; their sums are added in fp32:
  |y - exact| <= 7 2^-13 * sum over groups of 8 of max |p|  +  the bound above.
The cuts follow the products' signs; where these are random, the errors of one output add up like the
products themselves: |error| <= 7 2^-13 |y| < 2^-10 |y| in the 2-norm over the outputs.
The final rounding adds |y| eps / 2.
"""
import torch

BLOCK = 128
TINY = 448.0 * 2.0 ** -126


def _values():
    out = []
    for c in range(256):
        ex, m = (c >> 3) & 15, c & 7
        v = m * 2.0 ** -9 if ex == 0 else (8 + m) * 2.0 ** (ex - 10)
        if (c & 127) == 127:
            v = float("nan")
        out.append(-v if c & 128 else v)
    return torch.tensor(out, dtype=torch.float64)


VALUES = _values()
POS = VALUES[:127]                       # 0 .. 448, ascending
MID = (POS[1:] + POS[:-1]) / 2           # ties between neighbours


def decode(codes):
    return VALUES.to(codes.device)[codes.long()]


def encode(q):
    """Codes of the fp32 quotients q (float64 tensor of fp32 values): nearest, ties to the even code."""
    a, mid = q.abs(), MID.to(q.device)
    c = torch.bucketize(a, mid, right=False)          # number of midpoints below a
    tie = (c < mid.numel()) & (a == mid[c.clamp(max=mid.numel() - 1)])
    c = torch.where(tie & (c % 2 == 1), c + 1, c)
    c = torch.where(torch.isnan(q), torch.full_like(c, 127), c)
    return torch.where(torch.signbit(q), c + 128, c).to(torch.uint8)


def scales(x):
    """fp32 scales (as float64) of x [T, n] (float64 of bf16 or fp32 values)."""
    T, n = x.shape
    nb = -(-n // BLOCK)
    out = torch.empty((T, nb), dtype=torch.float64, device=x.device)
    for b in range(nb):
        g = x[:, BLOCK * b:BLOCK * (b + 1)].abs()
        m = torch.where(torch.isnan(g).any(1), torch.full_like(g[:, 0], float("nan")), g.nan_to_num(posinf=float("inf")).amax(1))
        m = torch.where(m < TINY, torch.full_like(m, TINY), m)
        out[:, b] = (m / 448.0).float().double()
    return out


def spread(s, n):
    return s.repeat_interleave(BLOCK, -1)[..., :n]


def quantize(x):
    """(codes uint8, scales float64) of x [T, n]."""
    s = scales(x)
    return encode((x / spread(s, x.shape[1])).float().double()), s


def weights(codes, s):
    """float64 values of codes [O, I] with block scales."""
    O, I = codes.shape
    return decode(codes) * s.double().repeat_interleave(BLOCK, 0)[:O].repeat_interleave(BLOCK, 1)[:, :I]


def product(a, w, K, exact):
    """(a w^T, bound of the sums' error) of float64 values; exact: the fp32 sums' bound."""
    blocks = -(-K // BLOCK)
    bound = (128 + blocks + 3) * 2.0 ** -23 * (a.abs() @ w.abs().t())
    if not exact:
        for i in range(0, K, 8):
            bound += 7 * 2.0 ** -13 * (a[:, None, i:i + 8].abs() * w[None, :, i:i + 8].abs()).amax(2)
    return a @ w.t(), bound


def swiglu(g, dg, u, du):
    """silu(g) u and the bound of its error for errors dg, du of its inputs: silu' lies in [-0.1, 1.1]; the
    kernel's exponential and reciprocal are each within 2 ulp, its three other operations within half of one,
    and e^-g carries the rounding of its argument, |g| 2^-23 relative: 8 + |g| units of 2^-23 in all."""
    s = g * torch.sigmoid(g)
    h = s * u
    return h, 1.1 * dg * u.abs() + s.abs() * du + 1.1 * dg * du + (8 + g.abs()) * 2.0 ** -23 * h.abs()


def expert_a8(xq, gate, up, down, exact=False):
    """Rows of one W8A8 expert on dequantised rows xq (float64): (rows, bound before the final rounding); exact:
    products with the fp32 sums' bound."""
    H = gate.shape[1]
    g, dg = product(xq, gate, H, exact)
    u, du = product(xq, up, H, exact)
    return rows_a8(g, dg, u, du, down, exact)


def rows_a8(g, dg, u, du, down, exact=False):
    """The rows from the sums of gate and up and the bounds dg, du of their errors."""
    F = g.shape[1]
    h, dh = swiglu(g, dg, u, du)
    codes, s = quantize(h)
    sx = spread(s, F)
    v = decode(codes)
    # relative error of a group's scale: that of its largest value, and two roundings
    T = h.shape[0]
    grp = lambda t: t.view(T, F // BLOCK, BLOCK)
    ds = (grp(dh).amax(2) / grp(h).abs().amax(2).clamp(min=TINY) + 2.0 ** -23).repeat_interleave(BLOCK, 1)
    # a quotient this near a tie may take the neighbouring code, a step away
    q = h / sx
    dq = dh / sx + q.abs() * (ds + 2.0 ** -23)
    near = (q.abs()[..., None] - MID.to(q.device)).abs().amin(-1) <= dq
    step = torch.exp2(torch.floor(torch.log2(q.abs().clamp(min=2.0 ** -6))) - 3) * 1.0
    dhq = (near * 2 * step + v.abs() * ds) * sx * (1 + ds)
    y, dy = product(v * sx, down, F, exact)
    return y, dy * 1.2 + dhq @ down.abs().t()
