"""The experts' gated MLP in 64 bits with the bound that the call's contract gives: h kept within 2^-17 of its value (and
2^-134, half of bf16's last place), everything else in fp32. picked.experts has the same form with a wider bound.

A sum is off by at most a last place (2^-23) of the sum of magnitudes for each addition of a term that is not zero (adding
zero is exact)."""
import torch

from tests.picked import ADD, HALF


def experts(x, ids, weights, w13, w2, parts=2):
    """(y, bound) in float64; w13 [E, 2I, H] and w2 [E, H, I] float64; ids outside [0, E) left out. With parts=1 y is what an
    h of one bf16 part would give, which the bound must not admit."""
    T, H = x.shape
    E, I = w13.shape[0], w2.shape[2]
    y = torch.zeros(T, H, dtype=torch.float64, device=x.device)
    off, size = torch.zeros_like(y), torch.zeros_like(y)
    x = x.double()
    for e in range(E):
        t, j = torch.nonzero(ids == e, as_tuple=True)
        if not t.numel():
            continue
        w = weights[t, j].double()[:, None]
        gu = x[t] @ w13[e].t()
        gu_off = (w13[e] != 0).sum(dim=1) * ADD * (x[t].abs() @ w13[e].abs().t())
        g, u, dg, du = gu[:, :I], gu[:, I:], gu_off[:, :I], gu_off[:, I:]
        s = g * torch.sigmoid(g)
        h = w * s * u
        # |silu'| < 1.1; exp (two), 1 +, quotient and two products: within 8 fp32 half steps
        ds = 1.1 * dg + 8 * 2.0 ** -24 * s.abs()
        dh = w.abs() * (ds * (u.abs() + du) + s.abs() * du)
        dh = dh + 2.0 ** -17 * (h.abs() + dh) + 2.0 ** -134
        mag = (h.abs() + dh) @ w2[e].abs().t()
        if parts == 1:
            h = h.bfloat16().double()
        y.index_add_(0, t, h @ w2[e].t())
        # two parts: twice the terms
        off.index_add_(0, t, dh @ w2[e].abs().t() + 2 * (w2[e] != 0).sum(dim=1) * ADD * mag)
        size.index_add_(0, t, mag)
    off = off + ids.shape[1] * ADD * size  # the pairs' sum
    return y, off + HALF[torch.bfloat16] * (y.abs() + off) + 2.0 ** -134
