"""Cases of the products whose weight is picked row by row: a router's choice of experts, the experts' gated MLP on
MXFP4 weights for a few tokens, and low-rank adapters beside a shared projection. `own` selects the library's calls or
plain torch."""
import math

import torch

own = False

_T = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
_BYTES = {"bf16": 2, "fp16": 2, "fp32": 4}
_E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0]
_ELEMENTS = 64 * 7168 * 2048      # E * H * I of the largest listed layer
_PAIRS = 64 * 8 * 7168 * 2048     # T * k * H * I of it


def listed():
    return [
        # a layer with few, small experts and two tokens: latency
        dict(name="experts_tiny", op="experts", T=2, H=512, I=256, E=8, k=2, absent=0.0),
        # one token of one request: eight experts are read, nothing else
        dict(name="experts_one_token", op="experts", T=1, H=7168, I=2048, E=32, k=8, absent=0.0),
        # odd extents (H and I end inside a tile), and pairs whose expert another rank holds
        dict(name="experts_ragged", op="experts", T=37, H=2112, I=1056, E=24, k=3, absent=0.15),
        # a decode batch of 64 requests: every expert is read once
        dict(name="experts_batch64", op="experts", T=64, H=7168, I=2048, E=64, k=8, absent=0.0),
        # a larger batch on smaller experts, 32 rows for each
        dict(name="experts_batch256", op="experts", T=256, H=2048, I=1024, E=32, k=4, absent=0.0),
        # the choice for a decode batch: sigmoid scores with a balancing bias
        dict(name="route_decode", op="route", T=16, E=256, k=8, dtype="fp32", score="sigmoid", bias=True, renormalize=True),
        # odd extents, bf16 logits with many ties, experts masked out, rows of padding with nothing left
        dict(name="route_ragged", op="route", T=777, E=60, k=3, dtype="bf16", score="softmax", bias=False, renormalize=False),
        # a prompt
        dict(name="route_prompt", op="route", T=4096, E=256, k=8, dtype="fp32", score="softmax", bias=False, renormalize=True),
        # one token with its adapter
        dict(name="adapters_one_token", op="adapters", T=1, K=7168, N=2112, R=16, n=8, dtype="bf16", out="bf16", spans=False),
        # a decode batch: any request has any adapter, or none
        dict(name="adapters_decode", op="adapters", T=64, K=7168, N=4096, R=32, n=24, dtype="bf16", out="bf16", spans=False),
        # odd extents, fp16 with an fp32 projection
        dict(name="adapters_ragged", op="adapters", T=777, K=2064, N=2113, R=24, n=5, dtype="fp16", out="fp32", spans=True),
        # prompts of a few requests in one batch
        dict(name="adapters_prompt", op="adapters", T=4096, K=7168, N=4096, R=64, n=8, dtype="bf16", out="bf16", spans=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["experts", "experts", "route", "adapters", "adapters"])
    if op == "route":
        E = _log(rng, 4, 512)
        return dict(op=op, T=_log(rng, 1, 4096), E=E, k=rng.randint(1, min(E, 12)), dtype=rng.choice(["fp32", "fp32", "bf16", "fp16"]),
                    score=rng.choice(["softmax", "sigmoid"]), bias=rng.random() < 0.4, renormalize=rng.random() < 0.7)
    if op == "experts":
        H, I = 32 * _log(rng, 8, 224), 32 * _log(rng, 4, 64)
        E = max(2, min(_log(rng, 4, 128), _ELEMENTS // (H * I)))
        k = rng.randint(1, min(E, 8))
        T = min(_log(rng, 1, 256), max(1, _PAIRS // (k * H * I)))
        return dict(op=op, T=T, H=H, I=I, E=E, k=k, absent=rng.choice([0.0, 0.0, 0.2]))
    n, R = _log(rng, 1, 32), 8 * _log(rng, 1, 16)
    K, N = 8 * _log(rng, 32, 896), _log(rng, 64, 8192)
    T = min(_log(rng, 1, 4096), max(1, 4096 * (7168 + 2 * 4096 + 8 * 64) // (K + 2 * N + n * R)))
    dtype = rng.choice(["bf16", "bf16", "fp16"])
    return dict(op=op, T=T, K=K, N=N, R=R, n=n, dtype=dtype, out=rng.choice([dtype, dtype, "fp32"]), spans=rng.random() < 0.5)


def _packed(codes, scales):
    """Codes [E, N, K/2] and scales [E, N, K/32] as the library's packed weights, one row of bytes for each expert: units
    of 32 columns x 64 k and after them scales of 32 columns x 256 k (N is a multiple of 32 here; K is padded with zeros)."""
    E, N, half = codes.shape
    KU, KG = -(-half // 32), -(-half // 128)
    pad = torch.nn.functional.pad
    units = pad(codes, (0, 32 * KU - half)).view(E, N // 32, 32, KU, 2, 16).permute(0, 1, 3, 4, 2, 5)
    words = pad(scales, (0, 8 * KG - half // 16), value=127).view(E, N // 32, 32, KG, 4, 2).permute(0, 1, 3, 5, 2, 4)
    return torch.cat([units.reshape(E, -1), words.reshape(E, -1)], dim=1)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    def uniform(*shape):
        return torch.rand(*shape, generator=g, device="cuda")

    def weight(E, N, K):
        # every code as likely as any other; scales that give a row's product about the size of its activations
        codes = torch.randint(0, 256, (E, N, K // 2), generator=g, device="cuda", dtype=torch.uint8)
        low = 127 - 3 - round(0.5 * math.log2(K))
        return codes, torch.randint(low, low + 3, (E, N, K // 32), generator=g, device="cuda", dtype=torch.uint8)

    state = dict(case)
    T = case["T"]
    if case["op"] == "experts":
        H, I, E, k = case["H"], case["I"], case["E"], case["k"]
        x = normal(T, H)
        x[:, :: max(1, H // 5)] *= 12.0  # a few outlier channels
        state["x"] = x.bfloat16()
        state["w13"], state["w2"] = weight(E, 2 * I, H), weight(E, H, I)  # gate and up rows; down
        state["w13_packed"], state["w2_packed"] = _packed(*state["w13"]), _packed(*state["w2"])  # kept by a program
        score, ids = torch.topk(normal(T, E), k, dim=1)
        state["ids"] = torch.where(uniform(T, k) < case["absent"], -1, ids).int()
        state["weights"] = torch.softmax(score, dim=1)
        return state
    if case["op"] == "route":
        E = case["E"]
        logits = (1.5 * normal(T, E)).masked_fill_(uniform(1, E) < 0.05, -math.inf)  # experts taken out of use
        logits = logits.masked_fill_(uniform(T, 1) < 0.02, -math.inf)                # rows of padding
        state["logits"] = logits.to(_T[case["dtype"]])
        state["bias_values"] = 0.1 * normal(E) if case["bias"] else None
        return state
    K, N, R, n = case["K"], case["N"], case["R"], case["n"]
    D = _T[case["dtype"]]
    state["x"] = normal(T, K).to(D)
    state["a"] = (normal(n, R, K) / math.sqrt(K)).to(D)
    state["b"] = (normal(n, N, R) / math.sqrt(R)).to(D)
    state["y"] = normal(T, N).to(_T[case["out"]])  # the shared projection's product
    state["scale"] = 0.1 + 0.2 * uniform(n)
    index = torch.randint(-1, n, (T,), generator=g, device="cuda")  # -1: no adapter
    if case["spans"]:  # the tokens of a request are neighbours and share its adapter
        at = torch.randint(0, T, (2 * n,), generator=g, device="cuda").sort().values
        index = torch.randint(-1, n, (2 * n + 1,), generator=g, device="cuda")[torch.searchsorted(at, torch.arange(T, device="cuda"))]
    state["index"] = index.int()
    return state


def _dequantised(codes, scales, T):
    table = torch.tensor([[_E2M1[b & 15], _E2M1[b >> 4]] for b in range(256)], dtype=T, device=codes.device)
    w = table.index_select(0, codes.reshape(-1).int()).view(*scales.shape, 32)
    return w.mul_(torch.exp2(scales.to(T) - 127)[..., None]).view(*codes.shape[:-1], -1)


def _experts(s):
    x, ids, weights = s["x"].float(), s["ids"], s["weights"]
    (T, k), E, I = ids.shape, s["E"], s["I"]
    here = ids >= 0
    if T * k <= E:  # each pair with its own expert's weights
        e = ids.clamp_min(0).reshape(-1)
        w13 = _dequantised(s["w13"][0][e], s["w13"][1][e], torch.float32)
        w2 = _dequantised(s["w2"][0][e], s["w2"][1][e], torch.float32)
        gu = torch.bmm(w13, x.repeat_interleave(k, dim=0)[:, :, None])
        pair = torch.where(here, weights, 0.0).reshape(-1, 1, 1)
    else:           # each expert with every token
        w13, w2 = _dequantised(*s["w13"], torch.float32), _dequantised(*s["w2"], torch.float32)
        gu = (w13.view(E * 2 * I, -1) @ x.t().contiguous()).view(E, 2 * I, T)
        pair = torch.zeros(T, E, device=x.device).scatter_add_(1, ids.clamp_min(0).long(), torch.where(here, weights, 0.0))
        pair = pair.t()[:, None, :]
    g, u = gu[:, :I], gu[:, I:]
    y = torch.bmm(w2, g / (1.0 + torch.exp(-g)) * u) * pair
    y = y.view(T, k, -1).sum(dim=1) if T * k <= E else y.sum(dim=0).t()
    return y.to(torch.bfloat16)


def _route(s):
    k = s["k"]
    l = s["logits"].double()  # in 64 bits: a last bit of a score would change the choice
    top = l.amax(dim=1, keepdim=True)
    p = torch.exp(l - torch.where(top > -math.inf, top, 0.0))
    p = 1.0 / (1.0 + torch.exp(-l)) if s["score"] == "sigmoid" else p / p.sum(dim=1, keepdim=True)
    rank = l if s["bias_values"] is None else torch.where(l > -math.inf, p + s["bias_values"].double(), -math.inf)
    rank, ids = torch.sort(rank, dim=1, descending=True, stable=True)
    chosen = rank[:, :k] > -math.inf
    ids = torch.where(chosen, ids[:, :k], -1)
    p = torch.where(chosen, p.gather(1, ids.clamp_min(0)), 0.0)
    if s["renormalize"]:
        total = p.sum(dim=1, keepdim=True)
        p = torch.where(total > 0, p / total, 0.0)
    return p.float(), ids.int()


def _adapters(s):
    n, N, R = s["b"].shape
    index = s["index"].long()
    u = (s["x"].float() @ s["a"].float().view(n * R, -1).t()).view(-1, n, R)
    mine = index[:, None] == torch.arange(n, device=index.device)
    u = torch.where(mine[:, :, None], u * s["scale"][:, None], 0.0).view(-1, n * R)
    s["y"].copy_(s["y"].float() + u @ s["b"].float().transpose(1, 2).reshape(n * R, N))
    return s["y"]


def run(state):
    """The adapters' sum is written where the projection's product is."""
    op = state["op"]
    if own:
        from mxfp4_block_scaled_02_amd import ops
        if op == "experts":
            return ops.moe_a16w4(state["x"], state["ids"], state["weights"], state["w13_packed"], state["w2_packed"], state["I"])
        if op == "route":
            return ops.moe_route(state["logits"], state["k"], bias=state["bias_values"], score=state["score"],
                                 renormalize=state["renormalize"])
        return ops.lora_add(state["y"], state["x"], state["a"], state["b"], state["index"], scale=state["scale"])
    return _experts(state) if op == "experts" else _route(state) if op == "route" else _adapters(state)


def work(case):
    T = case["T"]
    if case["op"] == "experts":
        H, I, E, k = case["H"], case["I"], case["E"], case["k"]
        there = 1.0 - case["absent"]
        read = E * (1.0 - (1.0 - there * k / E) ** T)  # experts that any token takes, on average
        return {"bytes": int(read * 3 * H * I * 17 / 32) + 4 * T * H + 8 * T * k, "flops": int(6 * there * T * k * H * I)}
    if case["op"] == "route":
        E, k = case["E"], case["k"]
        return {"bytes": T * E * _BYTES[case["dtype"]] + (4 * E if case["bias"] else 0) + 8 * T * k, "flops": 4 * T * E}
    K, N, R, n = case["K"], case["N"], case["R"], case["n"]
    some = T * n / (n + 1)  # tokens with an adapter, on average
    read = n * (1.0 - (1.0 - 1.0 / (n + 1)) ** min(T, 2 * n + 1 if case["spans"] else T))  # adapters that any token takes
    return {"bytes": int(some * (2 * K + 2 * N * _BYTES[case["out"]]) + read * 2 * R * (K + N)) + 4 * T + 4 * n,
            "flops": int(2 * some * R * (K + N))}


def exact(case, seed):
    """In 64 bits, expert by expert, row by row of the choice, adapter by adapter."""
    s = prepare(case, seed)
    if case["op"] == "experts":
        x, I = s["x"].double(), case["I"]
        y = torch.zeros_like(x)
        for e in range(case["E"]):
            row, slot = torch.nonzero(s["ids"] == e, as_tuple=True)
            if not row.numel():
                continue
            w13 = _dequantised(s["w13"][0][e], s["w13"][1][e], torch.float64)
            w2 = _dequantised(s["w2"][0][e], s["w2"][1][e], torch.float64)
            gu = torch.matmul(x[row], w13.t())
            h = torch.sigmoid(gu[:, :I]) * gu[:, :I] * gu[:, I:]
            y.index_add_(0, row, s["weights"][row, slot, None].double() * torch.matmul(h, w2.t()))
        return y
    if case["op"] == "route":
        l = s["logits"].cpu().double()
        p = torch.sigmoid(l) if case["score"] == "sigmoid" else torch.softmax(l, dim=1).nan_to_num(0.0)
        rank = l.clone() if s["bias_values"] is None else p + s["bias_values"].cpu().double()
        rank[l == -math.inf] = -math.inf
        weights, ids = [], []
        for _ in range(case["k"]):
            best, at = rank.max(dim=1)
            at = (rank == best[:, None]).int().argmax(dim=1)  # the lowest index of the largest
            none = best == -math.inf
            weights.append(p.gather(1, at[:, None])[:, 0].masked_fill(none, 0.0))
            ids.append(at.masked_fill(none, -1))
            rank.scatter_(1, at[:, None], -math.inf)
        w = torch.stack(weights, dim=1)
        if case["renormalize"]:
            w = (w / w.sum(dim=1, keepdim=True)).nan_to_num(0.0)
        return w, torch.stack(ids, dim=1).int()
    y = s["y"].double()
    for i in range(case["n"]):
        row = torch.nonzero(s["index"] == i)[:, 0]
        u = torch.matmul(s["x"][row].double(), s["a"][i].double().t())
        y.index_add_(0, row, s["scale"][i].double() * torch.matmul(u, s["b"][i].double().t()))
    return y
