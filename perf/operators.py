"""Cases of the 8-bit integer path: row quantisation, RMS norm with the residual's addition and quantisation, and the
integer matrix product with a scale for each token and channel. `own` selects the library's calls or plain torch."""
import math

import torch

own = False

_T = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
_BYTES = {"bf16": 2, "fp16": 2, "fp32": 4}
_EPS = 2.0 ** -20           # an epsilon that fp32 holds exactly
_MIN_SCALE = 2.0 ** -126    # the smallest scale: the smallest normal fp32
_CAP = 4096 * 4096 * 7168   # multiply-adds of the largest listed product
_CAP_ELEMENTS = 4096 * 7168


def listed():
    return [
        # one token of a decode step against a projection of 4096 channels
        dict(name="gemm_one_token", op="gemm", M=1, N=4096, K=7168, out="bf16", bias=False),
        # the smallest product: latency
        dict(name="gemm_tiny", op="gemm", M=4, N=256, K=512, out="bf16", bias=False),
        # a small decode batch, bound by reading the weight
        dict(name="gemm_decode", op="gemm", M=16, N=2112, K=7168, out="bf16", bias=False),
        # a larger decode batch, a projection with a bias
        dict(name="gemm_batch64", op="gemm", M=64, N=7168, K=2048, out="fp16", bias=True),
        # a short prompt or a mixed batch
        dict(name="gemm_mid", op="gemm", M=256, N=4096, K=7168, out="bf16", bias=False),
        # odd extents: a prompt of 777 tokens, an odd share of the channels, K that ends inside a tile, fp32 logits
        dict(name="gemm_ragged", op="gemm", M=777, N=2113, K=2064, out="fp32", bias=True),
        # a prefill
        dict(name="gemm_prefill", op="gemm", M=4096, N=4096, K=7168, out="bf16", bias=False),
        # the norm before a projection: a decode batch, an odd prompt without a residual (first layer), a prefill
        dict(name="norm_decode", op="norm", M=16, K=7168, dtype="bf16", residual=True),
        dict(name="norm_ragged", op="norm", M=777, K=2064, dtype="fp16", residual=False),
        dict(name="norm_prefill", op="norm", M=4096, K=7168, dtype="bf16", residual=True),
        # activations between two products; a weight in fp32, quantised by channel
        dict(name="quant_prefill", op="quant", M=4096, K=7168, dtype="bf16"),
        dict(name="quant_weight", op="quant", M=2112, K=7168, dtype="fp32"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["gemm", "gemm", "norm", "quant"])
    K = 16 * _log(rng, 4, 512)
    if op == "gemm":
        N = _log(rng, 16, 8192)
        M = min(_log(rng, 1, 4096), max(1, _CAP // (N * K)))
        return dict(op=op, M=M, N=N, K=K, out=rng.choice(["bf16", "fp16", "fp32"]), bias=rng.random() < 0.4)
    K = rng.choice([K, 16 * _log(rng, 512, 1024)])
    dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    M = min(_log(rng, 1, 4096), _CAP_ELEMENTS * 2 // (_BYTES[dtype] * K))
    case = dict(op=op, M=M, K=K, dtype=dtype)
    if op == "norm":
        case["residual"] = rng.random() < 0.7
    return case


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    M, K = case["M"], case["K"]
    state = dict(case)
    if case["op"] == "gemm":
        N, T = case["N"], _T[case["out"]]
        # codes as a row quantiser leaves them: the row's largest value is 127, most lie within a third of it
        state["aq"] = (normal(M, K) * 32).round_().clamp_(-127, 127).to(torch.int8)
        state["bq"] = (normal(N, K) * 32).round_().clamp_(-127, 127).to(torch.int8)
        state["a_scale"] = torch.rand(M, generator=g, device="cuda") * 0.04 + 0.01
        state["b_scale"] = torch.rand(N, generator=g, device="cuda") * 8e-4 + 2e-4
        state["bias_values"] = normal(N).to(T) if case["bias"] else None
        return state
    x = normal(M, K)
    x[:, :: max(1, K // 5)] *= 12.0  # a few outlier channels
    state["x"] = x.to(_T[case["dtype"]])
    if case["op"] == "norm":
        state["w"] = (1.0 + 0.2 * normal(K)).to(_T[case["dtype"]])
        state["r"] = (2.0 * normal(M, K)).to(_T[case["dtype"]]) if case["residual"] else None
    return state


def _row_codes(y):
    """Rows of fp32 values to (int8 codes, fp32 scales)."""
    s = (y.abs().amax(dim=1) * (1.0 / 127.0)).clamp_min(_MIN_SCALE)
    inverse = s.double().reciprocal().float()  # 1 / s, rounded once to fp32
    return torch.round(y * inverse[:, None]).to(torch.int8), s


def run(state):
    """The codes are whole numbers and are returned as such, beside the scales."""
    op = state["op"]
    if own:
        from mxfp4_block_scaled_02_amd import ops
        if op == "gemm":
            return ops.gemm_a8w8(state["aq"], state["a_scale"], state["bq"], state["b_scale"],
                                 bias=state["bias_values"], out_dtype=_T[state["out"]])
        if op == "norm":
            return ops.int8_rmsnorm_quant(state["x"], state["w"], _EPS, residual=state["r"])
        return ops.int8_quant(state["x"])
    if op == "gemm":
        c = state["aq"].float() @ state["bq"].float().t()
        c = c * state["a_scale"][:, None] * state["b_scale"][None, :]
        if state["bias_values"] is not None:
            c = c + state["bias_values"].float()
        return c.to(_T[state["out"]])
    if op == "norm":
        h = state["x"]
        if state["r"] is not None:
            h = (h.float() + state["r"].float()).to(h.dtype)
        # the squares' sum in 64 bits: a last bit of the norm would move codes that lie next to a border
        mean = h.double().square().mean(dim=1)
        inv = (1.0 / torch.sqrt(mean + _EPS)).float()
        q, s = _row_codes(h.float() * inv[:, None] * state["w"].float())
        return (q, s) if state["r"] is None else (q, s, h)
    return _row_codes(state["x"].float())


def work(case):
    M, K = case["M"], case["K"]
    if case["op"] == "gemm":
        N, t = case["N"], _BYTES[case["out"]]
        return {"bytes": M * K + N * K + t * M * N + 4 * (M + N) + (t * N if case["bias"] else 0), "flops": 2 * M * N * K}
    e = _BYTES[case["dtype"]]
    if case["op"] == "norm":
        return {"bytes": M * K * ((3 * e if case["residual"] else e) + 1) + e * K + 4 * M, "flops": 10 * M * K}
    return {"bytes": M * K * (e + 1) + 4 * M, "flops": 4 * M * K}


def exact(case, seed):
    """In 64 bits. Codes have no value there: a real number next to a border rounds either way."""
    state = prepare(case, seed)
    if case["op"] == "gemm":
        acc = torch.matmul(state["aq"].double(), state["bq"].double().t().contiguous())
        c = torch.einsum("mn,m,n->mn", acc, state["a_scale"].double(), state["b_scale"].double())
        return c if state["bias_values"] is None else c + state["bias_values"].double()
    y = state["x"].double()
    if case["op"] == "quant":
        return None, (torch.linalg.vector_norm(y, ord=math.inf, dim=1) / 127.0).clamp_min(_MIN_SCALE)
    total = y if state["r"] is None else y + state["r"].double()
    h = total.to(state["x"].dtype).double()  # the norm is of the rounded sum: the stream that is kept
    rms = torch.linalg.vector_norm(h, dim=1).square().div(case["K"]).add(_EPS).sqrt()
    y = h * state["w"].double() / rms[:, None]
    s = (torch.linalg.vector_norm(y, ord=math.inf, dim=1) / 127.0).clamp_min(_MIN_SCALE)
    return (None, s) if state["r"] is None else (None, s, total)
