"""The 64-bit forms of the operators around the layer: their gradients against differences, their parts against each other."""
import torch

from tests import around_ref as R

G = lambda seed: torch.Generator().manual_seed(seed)


def test_norm_gradients_are_those_of_the_norm():
    T, H, eps, off = 5, 24, 1e-6, 1.0
    s = torch.randn((T, H), generator=G(1), dtype=torch.float64)
    w = torch.randn(H, generator=G(2), dtype=torch.float64)
    dy = torch.randn((T, H), generator=G(3), dtype=torch.float64)
    dres = torch.randn((T, H), generator=G(4), dtype=torch.float64)
    f = lambda s, w: (R.norm(s, w, eps, off)[0] * dy).sum() + (s * dres).sum()
    dx, _, dw, _ = R.norm_backward(dy, s, R.norm(s, w, eps, off)[1], w, off, dres)
    h = 1e-6
    for t, i in ((0, 0), (2, 7), (4, 23)):
        e = torch.zeros_like(s)
        e[t, i] = h
        assert abs((f(s + e, w) - f(s - e, w)) / (2 * h) - dx[t, i]) < 1e-7
    for i in (0, 11, 23):
        e = torch.zeros_like(w)
        e[i] = h
        assert abs((f(s, w + e) - f(s, w - e)) / (2 * h) - dw[i]) < 1e-7


def test_balance_gradients_are_those_of_loss_and_gates():
    T, E, k, coef = 6, 12, 3, 0.3
    z = torch.randn((T, E), generator=G(5), dtype=torch.float64)
    z[1, 4] = -float("inf")
    z[2] = -float("inf")
    valid = torch.tensor([1, 1, 1, 0, 1, 1])
    idx = torch.stack([torch.randperm(E, generator=G(t))[:k] for t in range(T)]).int()
    idx[1] = torch.tensor([0, 5, 7])
    c = R.counts(idx, E, valid)
    dg = torch.randn((T, k), generator=G(6), dtype=torch.float64)
    gates = lambda z: torch.softmax(z.gather(1, idx.long()), 1)

    def f(z):
        g = torch.where(((valid > 0) & torch.isfinite(z).any(1))[:, None], gates(z), torch.zeros((T, k), dtype=torch.float64))
        return R.balance(z, c, k, coef, valid)["loss"] + float((g * dg).nan_to_num(0.0).sum())

    g = gates(z)
    g[2] = 0
    d = R.balance(z, c, k, coef, valid, idx, g, dg)["dlogits"]
    h = 1e-6
    for t, e in ((0, 0), (0, int(idx[0, 1])), (1, 5), (3, 2), (4, int(idx[4, 0])), (5, 11)):
        step = torch.zeros_like(z)
        step[t, e] = h
        assert abs((f(z + step) - f(z - step)) / (2 * h) - d[t, e]) < 1e-7
    assert (d[2] == 0).all() and (d[3] == 0).all() and d[1, 4] == 0


def test_shares_of_a_larger_batch_add_up():
    T, E, k = 20, 9, 2
    z = torch.randn((T, E), generator=G(7), dtype=torch.float64)
    idx = z.topk(k, 1).indices.int()
    c = R.counts(idx, E)
    whole = R.balance(z, c, k, 0.1)
    parts = [R.balance(z[:7], c, k, 0.1), R.balance(z[7:], c, k, 0.1)]
    assert abs(sum(p["loss"] for p in parts) - whole["loss"]) < 1e-12
    assert torch.allclose(torch.cat([p["dlogits"] for p in parts]), whole["dlogits"], atol=1e-15)


def test_unpack_is_the_inverse_of_the_packing():
    codes = torch.randint(0, 16, (3, 16), generator=G(8))
    words = torch.zeros((3, 2), dtype=torch.int64)
    for c in range(2):
        for j, col in enumerate(R.COLUMN):
            words[:, c] |= codes[:, 8 * c + col] << (4 * j)
    assert torch.equal(R.unpack(words), codes.double())
