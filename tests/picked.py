"""Plain forms in 64 bits of the products whose weight is picked row by row, with bounds of what the kernels may be off.

Each bound is elementwise: the roundings that the kernels make, carried through the formulas. A sum of n fp32 products is
within n * 2^-23 of the sum of the products' magnitudes, whatever its order (a last place for each addition, which also
covers a matrix instruction that truncates)."""
import math

import torch

E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0]
ADD = 2.0 ** -23
HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}  # half a step, relative


def dequantised(codes, scales):
    """fp4x2 [..., K/2] and E8M0 [..., K/32] uint8 -> float64 [..., K]."""
    table = torch.tensor(E2M1, dtype=torch.float64, device=codes.device)
    v = table[torch.stack([codes & 15, codes >> 4], dim=-1).long()].flatten(-2)
    s = torch.exp2(scales.double() - 127)
    return (v.unflatten(-1, (-1, 32)) * s[..., None]).flatten(-2)


def experts(x, ids, weights, w13, w2):
    """(y, bound) in float64; w13 [E, 2I, H] and w2 [E, H, I] float64; ids outside [0, E) left out."""
    T, H = x.shape
    E, I = w13.shape[0], w2.shape[2]
    y = torch.zeros(T, H, dtype=torch.float64, device=x.device)
    off = torch.zeros_like(y)
    size = torch.zeros_like(y)
    x = x.double()
    for e in range(E):
        t, j = torch.nonzero(ids == e, as_tuple=True)
        if not t.numel():
            continue
        w = weights[t, j].double()[:, None]
        gu = x[t] @ w13[e].t()
        gu_off = H * ADD * (x[t].abs() @ w13[e].abs().t())
        g, u, dg, du = gu[:, :I], gu[:, I:], gu_off[:, :I], gu_off[:, I:]
        s = g * torch.sigmoid(g)
        h = s * u
        # |silu'| < 1.1; exp, quotient and product take 8 fp32 half steps; a bf16 half step when h is kept
        ds = 1.1 * dg + 8 * 2.0 ** -24 * s.abs()
        dh = ds * (u.abs() + du) + s.abs() * du + 2.0 ** -8 * (h.abs() + ds * u.abs() + s.abs() * du)
        one = (h @ w2[e].t()) * w
        mag = ((h.abs() + dh) @ w2[e].abs().t()) * w.abs()
        y.index_add_(0, t, one)
        off.index_add_(0, t, (dh @ w2[e].abs().t()) * w.abs() + I * ADD * mag)
        size.index_add_(0, t, mag)
    off = off + (ids.shape[1] + 4) * ADD * size  # the pairs' sum, and their weights
    return y, off + HALF[torch.bfloat16] * (y.abs() + off) + 2.0 ** -130


def adapters(y, x, a, b, index, scale):
    """(y, bound) in float64."""
    out, off = y.double(), torch.zeros(y.shape, dtype=torch.float64, device=y.device)
    n, R, K = a.shape
    held = {torch.float32: 2.0 ** -23}.get(y.dtype, 2.0 ** -16)
    for i in range(n):
        t = torch.nonzero(index == i)[:, 0]
        if not t.numel():
            continue
        A, B, X = a[i].double(), b[i].double(), x[t].double()
        s = 1.0 if scale is None else scale[i].double()
        u = X @ A.t()
        # fp16 pieces: the row's largest value is brought to 2^14, a piece's last bit is at least 2^-24 there
        du = K * ADD * (X.abs() @ A.abs().t()) + held * u.abs() + 2.0 ** -38 * u.abs().amax(dim=1, keepdim=True)
        d = u @ B.t()
        mag = (u.abs() + du) @ B.abs().t()
        dd = du @ B.abs().t() + 3 * max(R, 32) * ADD * mag
        out.index_add_(0, t, s * d)
        off.index_add_(0, t, abs(s) * (dd + 2 * 2.0 ** -24 * (d.abs() + dd)))
    off = torch.where(((index >= 0) & (index < n))[:, None], off + 2.0 ** -24 * (out.abs() + off), off)
    return out, off + torch.where(off > 0, HALF[y.dtype] * (out.abs() + off) + 2.0 ** -25 * (y.dtype is torch.float16), 0.0)


def route(logits, k, bias, score, renormalize, scale):
    """(weights float64, ids) by the definition, row by row in plain Python; NaN weights for a row that is not finite."""
    weights, ids = [], []
    for row in logits.double().tolist():
        none = [v == -math.inf for v in row]
        top = max((v for v in row if v == v), default=-math.inf)
        if any(v != v or v == math.inf for v in row):
            weights.append([math.nan] * k)
            ids.append(list(range(k)))
            continue
        if score == "sigmoid":
            p = [1 / (1 + math.exp(-v)) if v > -700 else 0.0 for v in row]
        else:
            p = [0.0 if z else math.exp(v - top) for v, z in zip(row, none)]
            total = math.fsum(p)
            p = [q / total if total else 0.0 for q in p]
        rank = row if bias is None else [-math.inf if z else q + float(c) for q, z, c in zip(p, none, bias.double().tolist())]
        if any(r != r or r == math.inf for r in rank):
            weights.append([math.nan] * k)
            ids.append(list(range(k)))
            continue
        order = sorted((e for e in range(len(row)) if rank[e] > -math.inf), key=lambda e: (-rank[e], e))[:k]
        chosen = [p[e] for e in order]
        total = math.fsum(chosen)
        if renormalize:
            chosen = [q / total if total > 0 else 0.0 for q in chosen]
        weights.append([scale * q for q in chosen] + [0.0] * (k - len(order)))
        ids.append(order + [-1] * (k - len(order)))
    return torch.tensor(weights, dtype=torch.float64), torch.tensor(ids, dtype=torch.int32)
