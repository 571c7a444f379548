"""The router's choice and the experts' gated MLP on MXFP4 weights against plain forms in 64 bits."""
import math

import pytest
import torch

from mxfp4_block_scaled_02_amd import ops
from tests import picked

pytestmark = pytest.mark.gpu


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def weight(g, E, N, K):
    codes = torch.randint(0, 256, (E, N, K // 2), generator=g, device="cuda", dtype=torch.uint8)
    low = 124 - round(0.5 * math.log2(K))
    return codes, torch.randint(low, low + 3, (E, N, K // 32), generator=g, device="cuda", dtype=torch.uint8)


def layer(seed, T, H, I, E, k):
    g = gen(seed)
    w13, w2 = weight(g, E, 2 * I, H), weight(g, E, H, I)
    x = torch.randn(T, H, generator=g, device="cuda").bfloat16()
    score, ids = torch.topk(torch.randn(T, E, generator=g, device="cuda"), k, dim=1)
    return x, ids.int(), torch.softmax(score, dim=1), w13, w2


def check(x, ids, weights, w13, w2, **kw):
    I = w2[0].shape[2] * 2
    y = ops.moe_a16w4(x, ids, weights, ops.pack_experts(*w13), ops.pack_experts(*w2), I, **kw)
    ref, bound = picked.experts(x, ids, weights, picked.dequantised(*w13), picked.dequantised(*w2))
    off = (y.double() - ref).abs()
    assert torch.isfinite(y).all()
    assert (off <= bound).all(), (off / bound).max().item()
    return y


@pytest.mark.parametrize("T,H,I,E,k", [
    (1, 32, 32, 1, 1), (1, 512, 256, 8, 2), (2, 512, 256, 8, 2), (1, 96, 2112, 4, 4), (3, 2112, 96, 5, 3), (5, 64, 544, 7, 1),
    (16, 288, 160, 1, 1), (17, 288, 160, 1, 1), (33, 160, 288, 2, 2), (64, 256, 96, 1, 1), (65, 256, 96, 1, 1),
    (130, 128, 64, 3, 2), (37, 2112, 1056, 24, 3), (256, 192, 128, 130, 8), (11, 7168, 32, 33, 4), (512, 64, 64, 1024, 8),
    (4096, 32, 32, 40, 1), (1, 64, 64, 600, 64), (1, 32, 32, 16, 7),
])
def test_experts(T, H, I, E, k):
    check(*layer(T + H + I, T, H, I, E, k))


def test_indices_outside_the_range_are_left_out():
    x, ids, weights, w13, w2 = layer(1, 24, 256, 128, 6, 3)
    ids[0] = -1                                # a token without an expert
    ids[1, 1] = -1
    ids[2, 0], ids[2, 2] = 6, 2 ** 31 - 1      # another rank's experts
    ids[3] = -2 ** 31
    y = check(x, ids, weights, w13, w2)
    assert (y[0] == 0).all() and (y[3] == 0).all()
    ids[:] = -1
    assert (check(x, ids, weights, w13, w2) == 0).all()


def test_the_same_expert_twice_counts_twice():
    x, ids, weights, w13, w2 = layer(2, 9, 128, 96, 4, 2)
    ids[:] = ids[:, :1]
    check(x, ids, weights, w13, w2)
    ids[:] = 3
    check(x, ids, weights, w13, w2)


@pytest.mark.parametrize("T,E", [(9, 3), (70, 3), (70, 40)])
def test_a_row_depends_on_itself_alone(T, E):
    """The other rows may hold anything; the same call gives the same bits."""
    x, ids, weights, w13, w2 = layer(3, T, 544, 160, E, 2)
    p13, p2 = ops.pack_experts(*w13), ops.pack_experts(*w2)
    y = ops.moe_a16w4(x, ids, weights, p13, p2, 160)
    assert torch.equal(ops.moe_a16w4(x, ids, weights, p13, p2, 160), y)
    x[5], x[6, 3], x[7, 9] = math.nan, math.inf, -math.inf
    z = ops.moe_a16w4(x, ids, weights, p13, p2, 160)
    keep = torch.ones(T, dtype=torch.bool, device="cuda")
    keep[5:8] = False
    assert torch.equal(z[keep], y[keep]) and not torch.isfinite(z[5:8]).all(dim=1).any()


def test_strides_and_given_output():
    x, ids, weights, w13, w2 = layer(4, 21, 288, 64, 5, 2)
    wide = torch.full((21, 288 + 24), math.nan, device="cuda").bfloat16()
    wide[:, 8:296] = x
    out = torch.full((21, 300), 7.0, device="cuda").bfloat16()
    y = check(wide[:, 8:296], ids, weights, w13, w2, out=out[:, 4:292])
    assert y.data_ptr() == out[:, 4:].data_ptr()
    assert (out[:, :4] == 7).all() and (out[:, 292:] == 7).all()
    # experts further apart than their packed bytes
    p13, p2 = ops.pack_experts(*w13), ops.pack_experts(*w2)
    q13 = torch.zeros(5, p13.shape[1] + 48, dtype=torch.uint8, device="cuda")
    q13[:, :p13.shape[1]] = p13
    assert torch.equal(ops.moe_a16w4(x, ids, weights, q13, p2, 64), y)


def test_expert_weights_past_32_bit_offsets():
    """The last experts of weights of 4.8 GB."""
    E, H, I = 320, 2048, 4096
    g = gen(5)
    n13, n2 = ops.pack_B_bytes(2 * I, H), ops.pack_B_bytes(H, I)
    w13, w2 = weight(g, 2, 2 * I, H), weight(g, 2, H, I)
    p13 = torch.full((E, n13), 0x77, dtype=torch.uint8, device="cuda")
    p2 = torch.full((E, n2), 0x77, dtype=torch.uint8, device="cuda")
    assert E * n2 > 2 ** 30 and E * n13 > 2 ** 31
    p13[-2:], p2[-2:] = ops.pack_experts(*w13), ops.pack_experts(*w2)
    x = torch.randn(3, H, generator=g, device="cuda").bfloat16()
    ids = torch.tensor([[E - 1, E - 2], [E - 2, -1], [E, E - 1]], dtype=torch.int32, device="cuda")
    weights = torch.rand(3, 2, generator=g, device="cuda")
    y = ops.moe_a16w4(x, ids, weights, p13, p2, I)
    near = torch.where(ids < E, ids - (E - 2), -1)
    ref, bound = picked.experts(x, near, weights, picked.dequantised(*w13), picked.dequantised(*w2))
    assert ((y.double() - ref).abs() <= bound).all()


def test_the_layer_together_captured_and_replayed():
    """Logits to output, in a graph that is replayed with new inputs between eager work on another stream."""
    T, H, I, E, k = 8, 512, 256, 16, 4
    x, _, _, w13, w2 = layer(6, T, H, I, E, k)
    p13, p2 = ops.pack_experts(*w13), ops.pack_experts(*w2)
    wr = torch.randn(E, H, generator=gen(7), device="cuda").bfloat16() / 16

    def run(x, logits):
        weights, ids = ops.moe_route(logits, k, score="sigmoid")
        return ops.moe_a16w4(x, ids, weights, p13, p2, I)

    logits = x.float() @ wr.float().t()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        eager = run(x, logits)
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = run(x, logits)
    for i in range(4):
        x.copy_(torch.randn(T, H, generator=gen(20 + i), device="cuda"))
        logits.copy_(x.float() @ wr.float().t())
        eager = run(x, logits)
        y.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, eager)
        weights, ids = ops.moe_route(logits, k, score="sigmoid")
        check(x, ids, weights, w13, w2)


ROUTES = [(1, 4, 1), (3, 8, 2), (16, 256, 8), (5, 60, 3), (7, 65, 64), (9, 1024, 40), (130, 257, 8), (2, 1, 1), (4, 64, 64)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,k", ROUTES)
def test_route(T, E, k, score, dtype):
    g = gen(T + E)
    logits = (2 * torch.randn(T, E, generator=g, device="cuda")).to(dtype)
    for bias in (None, torch.randn(E, generator=g, device="cuda") * 0.1):
        for renormalize in (True, False):
            w, ids = ops.moe_route(logits, k, bias=bias, score=score, renormalize=renormalize, scale=1.5)
            rw, rids = picked.route(logits.cpu(), k, None if bias is None else bias.cpu(), score, renormalize, 1.5)
            assert torch.equal(ids.cpu(), rids)
            assert ((w.cpu().double() - rw).abs() <= 2.0 ** -24 * (1 + 1e-6) * rw.abs() + 2.0 ** -149).all()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("biased", [False, True])
def test_route_rows_at_the_edge(score, biased):
    inf, low = math.inf, torch.finfo(torch.float32).min
    rows = [[-inf] * 6, [1, -inf, 3, -inf, -inf, 2], [low] * 6, [low, 0, low, low, 1, low], [2, 2, 2, 2, 2, 2],
            [0.0, -0.0, 0.0, -0.0, 0.0, -0.0], [1, math.nan, 2, 3, 4, 5], [1, inf, 2, 3, 4, 5], [-inf, math.nan, -inf, -inf, -inf, -inf],
            [300, -300, 299, 0, -inf, 1], [1e30, 1e30, -1e30, 0, 5, 1e38]]
    logits = torch.tensor(rows, device="cuda")
    bias = torch.tensor([0.25, 0.0, -0.25, 0.0, 0.5, -inf], device="cuda") if biased else None
    for k in (1, 4, 6):
        for renormalize in (True, False):
            w, ids = ops.moe_route(logits, k, bias=bias, score=score, renormalize=renormalize)
            rw, rids = picked.route(logits.cpu(), k, None if bias is None else bias.cpu(), score, renormalize, 1.0)
            assert torch.equal(ids.cpu(), rids)
            assert torch.equal(w.cpu().isnan(), rw.isnan())
            assert ((w.cpu().double() - rw).nan_to_num(0.0).abs() <= 2.0 ** -24 * (1 + 1e-6) * rw.nan_to_num(0.0).abs() + 2.0 ** -149).all()


def test_route_a_bias_that_is_not_finite_shows():
    logits = torch.randn(3, 5, device="cuda")
    for v in (math.nan, math.inf):
        w, ids = ops.moe_route(logits, 2, bias=torch.tensor([0.0, v, 0.0, 0.0, 0.0], device="cuda"))
        assert w.isnan().all() and (ids == torch.tensor([0, 1], device="cuda")).all()


def test_route_strides_and_given_outputs():
    base = torch.randn(9, 50, device="cuda")
    logits = base[:, 3:40]
    out = (torch.empty(9, 4, device="cuda"), torch.empty(9, 4, dtype=torch.int32, device="cuda"))
    w, ids = ops.moe_route(logits, 4, out=out)
    rw, rids = picked.route(logits.cpu(), 4, None, "softmax", True, 1.0)
    assert w is out[0] and ids is out[1] and torch.equal(ids.cpu(), rids)
    assert ((w.cpu().double() - rw).abs() <= 2.0 ** -24 * (1 + 1e-6) * rw).all()


def test_workspace_contents_do_not_matter_and_its_end_is_kept():
    """The C call with a workspace of NaNs, and bytes behind it that stay."""
    for T, H, I, E, k in ((1, 512, 256, 8, 2), (20, 288, 96, 30, 5), (70, 288, 96, 3, 2)):
        x, ids, weights, w13, w2 = layer(11, T, H, I, E, k)
        ids[0, 0] = -1
        p13, p2 = ops.pack_experts(*w13), ops.pack_experts(*w2)
        y = ops.moe_a16w4(x, ids, weights, p13, p2, I)
        n = ops.lib().moe_a16w4_workspace_bytes(T, k, H, I)
        ws = torch.full((n + 256,), 0xFF, dtype=torch.uint8, device="cuda")
        z = torch.full((T + 1, H), 7.0, device="cuda").bfloat16()
        rc = ops.lib().moe_a16w4(x.data_ptr(), H, ids.data_ptr(), weights.data_ptr(), p13.data_ptr(), p13.stride(0),
                                 p2.data_ptr(), p2.stride(0), z.data_ptr(), H, T, k, E, H, I, ws.data_ptr(), n,
                                 torch.cuda.current_stream().cuda_stream)
        assert rc == 0 and torch.equal(z[:T], y) and (z[T] == 7).all() and (ws[n:] == 0xFF).all()


def test_two_captured_graphs_replayed_at_once():
    """Each graph has its own scratch memory: replays on two streams do not meet in it."""
    cases = [layer(20 + i, 70, 2048, 1024, 6, 2) for i in range(2)]
    packed = [(ops.pack_experts(*c[3]), ops.pack_experts(*c[4])) for c in cases]
    want = [ops.moe_a16w4(*c[:3], *p, 1024) for c, p in zip(cases, packed)]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for c, p in zip(cases, packed):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(ops.moe_a16w4(*c[:3], *p, 1024))
        graphs.append(g)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(10):
        for o in outs:
            o.zero_()
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        assert torch.equal(outs[0], want[0]) and torch.equal(outs[1], want[1])


def test_skewed_choice():
    """Most tokens take the same expert: more rows for it than go together, few or none for the others."""
    for T, E in ((64, 64), (200, 16), (300, 20)):
        x, ids, weights, w13, w2 = layer(T, T, 160, 96, E, 4)
        ids[:, 0] = E - 1
        ids[: T // 2, 1] = 2
        ids[ids == 5] = -1
        check(x, ids, weights, w13, w2)


@pytest.mark.parametrize("T,H,I,E,k", [(16, 4096, 128, 9, 4), (16, 4128, 128, 9, 4), (8, 4096, 160, 6, 6), (8, 4128, 160, 6, 6),
                                       (1, 4096, 2048, 12, 8), (1, 4128, 4096, 5, 4), (17, 4128, 64, 9, 3),
                                       (3, 288, 1024, 9, 8), (3, 288, 1056, 9, 8), (1, 64, 24576, 3, 2)])
def test_few_tokens(T, H, I, E, k):
    """On either side of the sizes at which the down product goes another way; experts that a token takes more than once."""
    x, ids, weights, w13, w2 = layer(T + H, T, H, I, E, k)
    check(x, ids, weights, w13, w2)
    ids[-1] = ids[0, 0]
    ids[:, 1] = ids[:, 0]
    ids[T // 2, 0] = -1
    check(x, ids, weights, w13, w2)


@pytest.mark.parametrize("T,H,I,E,k", [(100, 160, 96, 2, 1), (300, 96, 160, 2, 2), (700, 64, 544, 3, 2), (1000, 4096, 96, 4, 4),
                                       (250, 96, 2080, 3, 2), (130, 2048, 2048, 2, 1), (4096, 288, 64, 9, 1)])
def test_many_rows_to_an_expert(T, H, I, E, k):
    """More rows of an expert than go together: several workgroups have them, or one in turns, or one expert has all."""
    x, ids, weights, w13, w2 = layer(T + H, T, H, I, E, k)
    check(x, ids, weights, w13, w2)
    ids[:] = E - 1
    ids[T // 2 :, 0] = -1
    check(x, ids, weights, w13, w2)
    ids[:, 0] = torch.arange(T, device="cuda") % E
    check(x, ids, weights, w13, w2)


def test_a_bad_row_of_logits_shows_in_its_token_alone():
    x, _, _, w13, w2 = layer(40, 12, 256, 128, 10, 3)
    p13, p2 = ops.pack_experts(*w13), ops.pack_experts(*w2)
    logits = torch.randn(12, 10, generator=gen(41), device="cuda")
    want = ops.moe_a16w4(x, *reversed(ops.moe_route(logits, 3)), p13, p2, 128)
    logits[4, 7], logits[9, 0] = math.nan, math.inf
    weights, ids = ops.moe_route(logits, 3)
    y = ops.moe_a16w4(x, ids, weights, p13, p2, 128)
    bad = torch.zeros(12, dtype=torch.bool, device="cuda")
    bad[[4, 9]] = True
    assert y[bad].isnan().all()
    ref, bound = picked.experts(x[~bad], ids[~bad], weights[~bad], picked.dequantised(*w13), picked.dequantised(*w2))
    assert ((y[~bad].double() - ref).abs() <= bound).all() and torch.isfinite(want).all()


def test_the_same_packed_weights_serve_the_grouped_call():
    """Prompts' rows through the grouped product on the experts' packed weights, as the codes dequantise."""
    g = gen(42)
    codes, scales = weight(g, 3, 192, 256)
    p = ops.pack_experts(codes, scales)
    rows = [torch.randint(-4, 5, (m, 256), generator=g, device="cuda").bfloat16() for m in (5, 70, 130)]
    for r in rows:
        r[:, ::32] = 4.0               # every block's scale is 1, so that its values are E2M1 numbers
    w = picked.dequantised(codes, scales)
    for c, r, e in zip(ops.grouped_gemm(rows, list(p), 192), rows, range(3)):
        ref = r.double() @ w[e].t()
        bound = (256 * picked.ADD) * (r.double().abs() @ w[e].abs().t()) + picked.HALF[torch.bfloat16] * ref.abs() * 1.01
        assert ((c.double() - ref).abs() <= bound + 2.0 ** -130).all()


@pytest.mark.parametrize("T,E,k", [(1, 8, 8), (3, 40, 2), (16, 5, 4), (20, 40, 1), (90, 4, 1)])
def test_no_token_has_an_expert(T, E, k):
    x, ids, weights, w13, w2 = layer(T, T, 288, 96, E, k)
    ids[:] = torch.tensor([-1, E, 2 ** 31 - 1, -2 ** 31], device="cuda").repeat(T * k)[: T * k].view(T, k).int()
    out = torch.full((T, 288), math.nan, device="cuda").bfloat16()
    assert (check(x, ids, weights, w13, w2, out=out) == 0).all()


def test_calls_on_two_streams_at_once():
    cases = [layer(50 + i, T, 1024, 512, 12, 3) for i, T in enumerate((9, 100))]
    packed = [(ops.pack_experts(*c[3]), ops.pack_experts(*c[4])) for c in cases]
    want = [ops.moe_a16w4(*c[:3], *p, 512) for c, p in zip(cases, packed)]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream(), torch.cuda.Stream()], [[], []]
    for _ in range(20):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(ops.moe_a16w4(*cases[i][:3], *packed[i], 512))
    torch.cuda.synchronize()
    for g, w in zip(got, want):
        assert all(torch.equal(y, w) for y in g)
