"""Plain 64-bit forms of the operators around the layer (add-and-norm and its gradients, counts, balance loss and router
gradient, the 4-bit product) with bounds on how far fp32 arithmetic may be from them.  Shares no code with the library.

u = 2^-24 is half a step of fp32.  A sum of n terms in any order is off by at most n u times the sum of magnitudes (first
order; the constants below leave room for the second).  HALF[t] is half a step of type t, relative.
"""
import torch

from tests import a8_ref

U = 2.0 ** -24
HALF = {t: torch.finfo(t).eps / 2 for t in (torch.bfloat16, torch.float32)}

# ------------------------------------------------------------------ add and norm

# A row's sum of squares: at most 16 terms in a thread, 6 steps in a wave, 16 waves: 38 u relative (all terms are positive),
# half of it after the root; the mean, the root, the quotient, two products and the gain's addition 6 u more: below 32 u.
NORM_REL = 32 * U


def norm(s, weight, eps, offset):
    """(v, r) in 64 bits of the rows s as they are stored."""
    s = s.double()
    r = 1.0 / torch.sqrt((s * s).mean(1) + eps)
    return s * r[:, None] * (offset + weight.double()), r


def check_rows(y, v, rel=NORM_REL, extra=0.0):
    """y, rounded once, against v that fp32 arithmetic may miss by rel |v| + extra."""
    miss = rel * v.abs() + extra
    err = (y.double() - v).abs()
    lim = miss + HALF[y.dtype] * (v.abs() + miss)
    if y.dtype == torch.bfloat16:
        lim = lim + 2.0 ** -134  # half of the smallest denormal step
    bad = ~(err <= lim)
    assert not bad.any(), f"{int(bad.sum())} values off, largest excess {(err - lim).max():.3e}"


def check_fp8(codes, scales, v):
    """Codes and scales of v: the scale carries v's error and its own rounding, and a code is the rounding of some quotient
    within twice that of the exact one."""
    n = v.shape[1]
    exact = a8_ref.scales(v)
    err = (scales.double() - exact).abs()
    assert (err <= (NORM_REL + 2 * U) * exact).all(), "scales"
    q = v / a8_ref.spread(exact, n)
    d = 2 * (NORM_REL + 2 * U)
    lo = a8_ref.decode(a8_ref.encode((q.abs() * (1 - d)).clamp(max=448.0)))
    hi = a8_ref.decode(a8_ref.encode((q.abs() * (1 + d)).clamp(max=448.0)))
    got = a8_ref.decode(codes)
    assert ((got.abs() >= lo) & (got.abs() <= hi)).all(), "codes"
    assert (torch.signbit(got) == torch.signbit(v))[got != 0].all(), "signs"


def norm_backward(dy, s, rstd, weight, offset, dres=None):
    """(dx, its bound, dw, its bound) in 64 bits, from the rstd that is given."""
    dy, s, r = dy.double(), s.double(), rstd.double()[:, None]
    T, H = s.shape
    h = s * r
    u = dy * (offset + weight.double())
    mean = (u * h).mean(1, keepdim=True)
    mag = (u * h).abs().mean(1, keepdim=True)
    dx = r * (u - h * mean)
    # u and h: 3 roundings; the sum over a row as in the norm 38 u of its magnitudes, and the products' own 3; then 4 operations
    lim = r * (4 * U * u.abs() + h.abs() * 48 * U * mag + 4 * U * (u.abs() + (h * mean).abs()))
    if dres is not None:
        dx = dx + dres.double()
        lim = lim + U * dx.abs()
    # dw: any order of T terms of two roundings each
    return dx, lim, (dy * h).sum(0), (T + 4) * U * (dy * h).abs().sum(0)


# ------------------------------------------------------------------ balance

def counts(idx, E, valid=None):
    idx = idx.long()
    if valid is not None:
        idx = idx[valid.bool()]
    idx = idx[(idx >= 0) & (idx < E)]
    return torch.bincount(idx.reshape(-1), minlength=E)


def balance(logits, c, k, coef, valid=None, idx=None, gate=None, dgate=None):
    """dict of loss, prob_sum, dlogits in 64 bits and, under "lim_*", their bounds before the last rounding."""
    z = logits.double()
    T, E = z.shape
    on = torch.ones(T, dtype=torch.bool, device=z.device) if valid is None else valid.bool()
    z = torch.where(on[:, None], z, torch.full_like(z, -float("inf")))
    m = z.amax(1, keepdim=True) if E else z
    full = (z == -float("inf")).all(1, keepdim=True)
    x = torch.where(full, torch.full_like(z, -float("inf")), z - torch.where(full, torch.zeros_like(m), m))
    e = torch.exp(x)
    p = torch.where(full, torch.zeros_like(e), e / e.sum(1, keepdim=True))
    C = float(c.sum())
    a = coef * E * k / C if C else 0.0
    f = c.double() / C - 1.0 / E if C else torch.zeros(E, dtype=torch.float64, device=z.device)
    q = p @ f
    rows = float((~full).sum())
    # a probability: the difference's rounding |x| u, the exponential 4 u, the sum over the experts 40 u, two operations
    rel = (48.0 + x.abs().clamp(max=104.0)) * U
    top = torch.where(p > 0, rel, torch.zeros_like(rel)).amax(1, keepdim=True)
    mag = (p @ f.abs())[:, None]
    d = a * p * (f - q[:, None])
    # flushed below fp32's normal range: 2^-126 of a probability
    lim = abs(a) * (p + 2.0 ** -126) * (2 * top + 48 * U) * (f.abs() + mag) + abs(a) * 2.0 ** -126 * (f.abs() + mag)
    if dgate is not None:
        g, dg = gate.double(), dgate.double()
        ok = on[:, None] & (idx >= 0) & (idx < E)
        gd = g * dg
        v = g * (dg - gd.sum(1, keepdim=True))
        lv = 80 * U * (gd.abs() + g * gd.abs().sum(1, keepdim=True))  # at most 64 terms in 16 steps, four operations
        at = torch.where(ok, idx.long(), torch.zeros_like(idx.long()))
        zero = torch.zeros_like(v)
        d = d.scatter_add(1, at, torch.where(ok, v, zero))
        lim = lim.scatter_add(1, at, torch.where(ok, lv + 4 * U * v.abs(), zero)) + U * d.abs()
    tm = float(torch.nan_to_num(top).amax()) if T else 0.0
    loss = a * (float(q.sum()) + rows / E)
    return {"loss": loss, "lim_loss": (tm + 64 * U) * abs(a) * (float(mag.sum()) + rows / E), "prob_sum": p.sum(0),
            # at most T / 4096 tokens a team one after another, then 32 teams and 80 steps over workgroups
            "lim_prob_sum": (tm + (T / 4096 + 116) * U) * p.sum(0) + T * 2.0 ** -126, "dlogits": d, "lim_dlogits": lim}


def check_balance(got, ref, dtype):
    loss, prob_sum, d = got
    assert abs(float(loss) - ref["loss"]) <= ref["lim_loss"] + U * abs(ref["loss"]) + 1e-45, (float(loss), ref["loss"])
    assert ((prob_sum.double() - ref["prob_sum"]).abs() <= ref["lim_prob_sum"]).all()
    if d is not None:
        assert d.dtype == dtype
        check_rows(d, ref["dlogits"], 2 * U, ref["lim_dlogits"] + 2.0 ** -126)  # (fp32 results below its normal range are flushed)


# ------------------------------------------------------------------ 4-bit product

COLUMN = (0, 2, 4, 6, 1, 3, 5, 7)


def unpack(words):
    """[R, n/8] words in GEMM packing -> [R, n] numbers."""
    w = words.long()
    out = torch.empty((w.shape[0], w.shape[1] * 8), dtype=torch.float64, device=w.device)
    for j, c in enumerate(COLUMN):
        out[:, c::8] = ((w >> 4 * j) & 15).double()
    return out


def awq(x, qweight, qzeros, scales):
    """(y, bound) in 64 bits."""
    K = qweight.shape[0]
    group = K // qzeros.shape[0]
    q = unpack(qweight)
    z = unpack(qzeros).repeat_interleave(group, 0)
    s = scales.double().repeat_interleave(group, 0)
    x = x.double()
    # per 32 inputs two sums of 32 exact products x (16 + q), x (16 + z) on the matrix cores, 33 roundings of 2 u each, and two
    # operations; then the sums over K / 32 steps, 8 waves and the splits, of magnitudes x |q - z| s
    lim = 2 * 36 * U * (x.abs() @ ((32 + q + z) * s.abs())) + (K / 32 + 80) * U * (x.abs() @ ((q - z) * s).abs())
    return x @ ((q - z) * s), lim
