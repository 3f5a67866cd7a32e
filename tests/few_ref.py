"""The whole layer in 64 bits for few tokens, with a bound on how far fp32 arithmetic may be from it.

Bound.  A sum of products in fp32, however split over lanes, meets fewer than 128 roundings on any path here
(at most 90 additions in a lane, 6 levels of lanes, a scale), each off by at most 2^-23 of the magnitudes
summed (2^-24 rounded to nearest, twice that truncated): error <= 128 2^-23 A, A the sum of the magnitudes of
what is added.  For 4-bit codes that is s (128 + q) x and s (128 + z) x in the first two projections, s q h
and s z h in the last.  h is rounded to bf16, half a step of 2^-8.  Gates: an exponential (2 ulp), a sum and a division, 2^-20 relative.
"""
import torch

from tests import a8_ref as R

ORDER = (0, 2, 4, 6, 1, 3, 5, 7)      # column (mod 8) of nibble j of an AWQ zero word


def matrices(bank, name, e):
    """(w, m1, m2): float64 weights [O, I] of expert e, and the magnitudes that sums of the first two / of the
    last projection add up per unit of input."""
    if bank["fmt"] == "bf16":
        w = bank[name][e].double()
        return w, w.abs(), w.abs()
    if bank["fmt"] == "fp8":
        w = R.weights(bank[name + "_codes"][e], bank[name + "_bscales"][e])
        return w, w.abs(), w.abs()
    qw, qz, s = (bank[name + t][e] for t in ("_qweight", "_qzeros", "_scales"))
    O, I = qw.shape[0], qw.shape[1] * 8
    q = torch.stack([(qw >> (4 * j)) & 15 for j in range(8)], -1).reshape(O, I).double()
    z = torch.zeros((I // 32, O), dtype=torch.float64, device=qw.device)
    for j in range(8):
        z[:, ORDER[j]::8] = ((qz >> (4 * j)) & 15).double()
    z, s = (t.t().repeat_interleave(32, 1) for t in (z, s.double()))
    return (q - z) * s, (256 + q + z) * s, (q + z) * s


def expert(bank, e, x):
    """(output, bound) of expert e on x [H] float64."""
    eps = 128 * 2.0 ** -23
    (wg, mg, _), (wu, mu, _), (wd, _, md) = (matrices(bank, n, e) for n in ("gate", "up", "down"))
    g, u = wg @ x, wu @ x
    h, dh = R.swiglu(g, eps * (mg @ x.abs()), u, eps * (mu @ x.abs()))
    dh = dh + 2.0 ** -8 * (h.abs() + dh)      # rounded to bf16 (with the gate, a factor)
    return wd @ h, wd.abs() @ dh + eps * (md @ (h.abs() + dh))


def layer(x, router, k, bank, shared=None, scale=None):
    """(y float64 [T, H], bound before the final rounding, topk_idx [T, k])."""
    x = x.double()
    logits = (x @ router.double().t()).float()
    top, idx = torch.sort(logits, dim=1, descending=True, stable=True)
    top, idx = top[:, :k].double(), idx[:, :k]
    gate = torch.softmax(top, 1)
    y, dy = torch.zeros_like(x), torch.zeros_like(x)
    for t in range(x.shape[0]):
        for j in range(k):
            o, d = expert(bank, int(idx[t, j]), x[t])
            y[t] += gate[t, j] * o
            dy[t] += gate[t, j] * (d + 2.0 ** -20 * (o.abs() + d))
        if shared is not None:
            s = 1.0 if scale is None else float(scale[t])
            o, d = expert(shared, 0, x[t])
            y[t] += s * o
            dy[t] += abs(s) * (d + 2.0 ** -22 * o.abs())
    return y, dy * (1 + 2.0 ** -16), idx.int()
