"""What the experts' call promises of its numbers: h within 2^-17, every scale byte, offsets past 32 bits; on every way that
a call can take (by tokens, few and many rows to an expert)."""
import math

import pytest
import torch

from mxfp4_block_scaled_02_amd import ops
from tests import picked, picked_close
from tests.test_gpu_lora_paths import grids
from tests.test_gpu_moe import gen, layer, weight

pytestmark = pytest.mark.gpu

# T, H, I, E, k: the down product by tokens with 16 and 32 columns to a workgroup; few rows to an expert; many in groups of 32
# and of 64 rows (50 an expert on average).
WAYS = [(5, 256, 96, 6, 2), (5, 4128, 96, 6, 2), (6, 256, 96, 6, 2), (20, 256, 96, 30, 5), (90, 256, 96, 4, 2), (800, 928, 480, 64, 4)]
CODE = {v: i for i, v in enumerate(picked.E2M1)}


def run(x, ids, weights, w13, w2):
    return ops.moe_a16w4(x, ids, weights, ops.pack_experts(*w13), ops.pack_experts(*w2), w2[0].shape[2] * 2)


def close(y, ref, bound):
    off = (y.double() - ref).abs()
    assert torch.isfinite(y).all()
    assert (off <= bound).all(), (off / bound).max().item()


def pair_up(values):
    """E2M1 values [..., K] -> codes [..., K/2]."""
    table = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=values.device)
    code = torch.searchsorted(table, values.abs().contiguous()) + 8 * (values < 0)
    assert (table[code % 8] == values.abs()).all()
    return (code[..., ::2] | code[..., 1::2] << 4).to(torch.uint8)


@pytest.mark.parametrize("T,H,I,E,k", WAYS + [(1, 32, 32, 1, 1), (37, 2112, 1056, 24, 3), (300, 1024, 64, 8, 1)])
def test_random_layers_within_the_contract(T, H, I, E, k):
    x, ids, weights, w13, w2 = layer(T + H + 1, T, H, I, E, k)
    close(run(x, ids, weights, w13, w2),
          *picked_close.experts(x, ids, weights, picked.dequantised(*w13), picked.dequantised(*w2)))


@pytest.mark.parametrize("T,H,I,E,k", WAYS)
def test_h_keeps_its_second_part(T, H, I, E, k):
    """h of 1, 2 and 3 times the same value, which cancel in the down product: what is left is what h was rounded by."""
    g = gen(T + H + I)
    m = I // 3

    def some(choice, *shape, share):
        v = torch.tensor(choice, device="cuda")[torch.randint(0, len(choice), shape, generator=g, device="cuda")]
        return torch.where(torch.rand(*shape, generator=g, device="cuda") < share, v, 0.0)

    gate = some([-2.0, -1.5, 0.5, 1.0, 3.0], E, m, H, share=4 / H)
    gate[:, torch.arange(m), torch.arange(m) % H] = 1.5
    up = some([-2.0, -1.0, 0.5, 1.0, 2.0], E, m, H, share=2 / H)
    up[:, torch.arange(m), (torch.arange(m) + 7) % H] = 1.0
    w13 = torch.cat([gate] * 3 + [up, 2 * up, 3 * up], dim=1)
    down = some([-3.0, -1.0, 0.5, 2.0], E, H, m, share=0.3)
    w2 = torch.cat([down, down, -down], dim=2)
    scale13 = torch.full((E, 2 * I, H // 32), 127, dtype=torch.uint8, device="cuda")
    scale2 = torch.full((E, H, I // 32), 126, dtype=torch.uint8, device="cuda")
    x = torch.randn(T, H, generator=g, device="cuda").bfloat16()
    ids = torch.rand(T, E, generator=g, device="cuda").argsort(dim=1)[:, :k].int().contiguous()
    weights = torch.rand(T, k, generator=g, device="cuda") + 0.5
    w13, w2 = (pair_up(w13), scale13), (pair_up(w2), scale2)
    d13, d2 = picked.dequantised(*w13), picked.dequantised(*w2)
    ref, bound = picked_close.experts(x, ids, weights, d13, d2)
    one, _ = picked_close.experts(x, ids, weights, d13, d2, parts=1)
    assert ((one - ref).abs() > 2 * bound).any(dim=1).float().mean() > 0.9  # one part would show in most tokens
    close(run(x, ids, weights, w13, w2), ref, bound)


def one_each(E, T, way):
    """Tokens with one expert each, all of them taken: calls of (first token, tokens)."""
    step = 10 if way == "tokens" else T
    return [(a, min(step, T - a)) for a in range(0, T, step)]


@pytest.mark.parametrize("way", ["tokens", "few", "many"])
def test_gate_and_up_with_every_scale_byte(way):
    """Expert e has scale bytes e throughout, its tokens activations of about 2^(127 - e)."""
    E, H, I = 253, 64, 32
    T = 12 * E if way == "many" else E
    g = gen(70)
    w13, w2 = weight(g, E, 2 * I, H), weight(g, E, H, I)
    w13[1][:] = torch.arange(E, device="cuda")[:, None, None]
    ids = (torch.arange(T, device="cuda") % E)[:, None].int()
    m = (1 + 0.75 * torch.rand(T, H, generator=g, device="cuda")) * torch.where(
        torch.rand(T, H, generator=g, device="cuda") < 0.5, -1.0, 1.0)
    x = (m.bfloat16().double() * torch.exp2(127.0 - ids.double())).bfloat16()
    weights = torch.rand(T, 1, generator=g, device="cuda") + 0.5
    ref, bound = picked_close.experts(x, ids, weights, picked.dequantised(*w13), picked.dequantised(*w2))
    packed = ops.pack_experts(*w13), ops.pack_experts(*w2)
    y = torch.cat([ops.moe_a16w4(x[a:a + n], ids[a:a + n], weights[a:a + n], *packed, I) for a, n in one_each(E, T, way)])
    off = (y.double() - ref).abs()
    wrong = torch.unique(ids[(~(off <= bound)).any(dim=1)]).tolist()
    assert not wrong, wrong


@pytest.mark.parametrize("way", ["tokens", "few", "many"])
def test_down_with_scale_bytes(way):
    """Expert e has down weights of scale byte e + 8, and an h of about 2^(119 - e) that its up rows' scales make."""
    E, H, I = 237, 64, 96
    T = 12 * E if way == "many" else E
    g = gen(71)
    w13, w2 = weight(g, E, 2 * I, H), weight(g, E, H, I)
    byte = torch.arange(E, device="cuda")[:, None, None] + 8
    w13[1][:, :I], w13[1][:, I:], w2[1][:] = 130, 254 - byte, byte
    ids = (torch.arange(T, device="cuda") % E)[:, None].int()
    x = (torch.randn(T, H, generator=g, device="cuda") * 2.0 ** -8).bfloat16()
    weights = torch.rand(T, 1, generator=g, device="cuda") + 0.5
    ref, bound = picked_close.experts(x, ids, weights, picked.dequantised(*w13), picked.dequantised(*w2))
    packed = ops.pack_experts(*w13), ops.pack_experts(*w2)
    y = torch.cat([ops.moe_a16w4(x[a:a + n], ids[a:a + n], weights[a:a + n], *packed, I) for a, n in one_each(E, T, way)])
    off = (y.double() - ref).abs()
    wrong = torch.unique(ids[(~(off <= bound)).any(dim=1)] + 8).tolist()
    assert not wrong, wrong


def test_weights_past_32_bit_offsets_on_every_way():
    """The last experts of weights of 8.8 and 4.4 GB."""
    E, H, I = 304, 4096, 6688
    g = gen(72)
    w13, w2 = weight(g, 2, 2 * I, H), weight(g, 2, H, I)
    p13 = torch.full((E, ops.pack_B_bytes(2 * I, H)), 0x77, dtype=torch.uint8, device="cuda")
    p2 = torch.full((E, ops.pack_B_bytes(H, I)), 0x77, dtype=torch.uint8, device="cuda")
    p13[-2:], p2[-2:] = ops.pack_experts(*w13), ops.pack_experts(*w2)
    assert p13[-2:].storage_offset() > 2 ** 33 and p2[-2:].storage_offset() > 2 ** 32
    d13, d2 = picked.dequantised(*w13), picked.dequantised(*w2)
    for T, k, some in ((1, 2, 1), (20, 2, 20), (3100, 1, 100)):  # by tokens; few; many rows to an expert
        x = torch.randn(T, H, generator=g, device="cuda").bfloat16()
        ids = torch.full((T, k), -1, dtype=torch.int32, device="cuda")
        ids[:some] = E - 1 - torch.arange(some * k, device="cuda").view(some, k).int() % 2
        weights = torch.rand(T, k, generator=g, device="cuda")
        y = ops.moe_a16w4(x, ids, weights, p13, p2, I)
        near = torch.where(ids >= 0, ids - (E - 2), -1)[:some]
        close(y[:some], *picked_close.experts(x[:some], near, weights[:some], d13, d2))
        assert (y[some:] == 0).all()


@pytest.mark.parametrize("T,H,I,E,k", [(16, 256, 96, 6, 2), (10, 256, 96, 6, 1), (40, 256, 96, 30, 3), (40, 256, 96, 3, 2)])
def test_rows_past_32_bit_offsets(T, H, I, E, k):
    """x and y with rows so far apart that the last ones lie past 2^32 bytes."""
    x, ids, weights, w13, w2 = layer(73 + E, T, H, I, E, k)
    ld = 2 ** 33 // T // 16 * 16 // 2  # elements; T rows take 8 GB
    far, out = (torch.zeros(T * ld, dtype=torch.bfloat16, device="cuda").as_strided((T, H), (ld, 1)) for _ in range(2))
    far.copy_(x)
    assert (T - 1) * ld * 2 > 2 ** 32
    p13, p2 = ops.pack_experts(*w13), ops.pack_experts(*w2)
    want = ops.moe_a16w4(x, ids, weights, p13, p2, I)
    y = ops.moe_a16w4(far, ids, weights, p13, p2, I, out=out)
    assert y is out and torch.equal(y, want)
    close(want, *picked_close.experts(x, ids, weights, picked.dequantised(*w13), picked.dequantised(*w2)))


def test_logits_past_32_bit_offsets():
    for dtype in (torch.bfloat16, torch.float32):
        T, E = 40, 130
        ld = 2 ** 33 // T // torch.finfo(dtype).bits * 8
        logits = torch.randn(T, E, generator=gen(74), device="cuda").to(dtype)
        far = torch.zeros(T * ld, dtype=dtype, device="cuda").as_strided((T, E), (ld, 1))
        far.copy_(logits)
        for a, b in zip(ops.moe_route(far, 8), ops.moe_route(logits, 8)):
            assert torch.equal(a, b)
        del far


def test_one_part_of_h_differs_where_the_contract_says():
    """The form with one part is the other one's with h rounded to bf16: by hand."""
    w13 = torch.tensor([[[2.0], [3.0]]], dtype=torch.float64)
    w2 = torch.tensor([[[0.5]]], dtype=torch.float64)
    x, ids, w = torch.tensor([[1.0]]).bfloat16(), torch.tensor([[0]]), torch.tensor([[1.0]])
    h = 2 / (1 + math.exp(-2)) * 3
    y, bound = picked_close.experts(x, ids, w, w13, w2)
    one, _ = picked_close.experts(x, ids, w, w13, w2, parts=1)
    assert abs(y.item() - h / 2) < 1e-12 and one.item() == torch.tensor(h).bfloat16().double().item() / 2
    assert 2.0 ** -8 * h / 2 < bound.item() < 1.02 * 2.0 ** -8 * h / 2


@pytest.mark.parametrize("T,H,I,E,k,launches", [
    (1, 256, 96, 6, 2, 2), (5, 256, 96, 6, 2, 2), (10, 4128, 96, 12, 1, 2), (1, 64, 24576, 3, 1, 2), (1, 64, 24608, 3, 1, 3),
    (1, 256, 96, 20, 10, 2), (1, 256, 96, 20, 11, 3), (11, 256, 96, 12, 1, 3), (4, 4128, 96, 12, 4, 3), (2, 160, 2432, 9, 5, 2),
    (2, 160, 2464, 9, 5, 3),
])
def test_either_side_of_the_way_by_tokens(T, H, I, E, k, launches):
    """Up to 10 pairs, and as much of h as there is room for, the down product adds up a token's experts itself; experts that a
    token takes more than once, and a token without any."""
    x, ids, weights, w13, w2 = layer(T + H + I, T, H, I, E, k)
    d13, d2 = picked.dequantised(*w13), picked.dequantised(*w2)
    packed = ops.pack_experts(*w13), ops.pack_experts(*w2)
    for _ in range(3):
        close(ops.moe_a16w4(x, ids, weights, *packed, I), *picked_close.experts(x, ids, weights, d13, d2))
        ids[T // 2, -1], ids[-1] = -1, ids[0, 0].clone()
        ids[0] = ids[0, 0].clone()
    graph = torch.cuda.CUDAGraph(keep_graph=True)
    with torch.cuda.graph(graph):
        ops.moe_a16w4(x, ids, weights, *packed, I)
    assert len(grids(graph)) == launches


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("value", [math.nan, math.inf])
def test_a_bias_of_an_expert_out_of_use_does_not_show(score, value):
    """The rank of a logit of -inf is -inf, whatever the expert's bias; where its logit is finite the row shows it."""
    logits = torch.randn(9, 70, generator=gen(75), device="cuda")
    logits[:, [3, 66]] = -math.inf
    logits[4, 3] = 0.5
    bias = 0.1 * torch.randn(70, generator=gen(76), device="cuda")
    bias[3], bias[66] = value, -value
    w, ids = ops.moe_route(logits, 8, bias=bias, score=score)
    rw, rids = picked.route(logits.cpu(), 8, bias.cpu(), score, True, 1.0)
    assert torch.equal(ids.cpu(), rids) and torch.equal(w.cpu().isnan(), rw.isnan())
    assert rw.isnan().any(dim=1).tolist() == [r == 4 for r in range(9)]
    assert ((w.cpu().double() - rw).nan_to_num(0.0).abs() <= 2.0 ** -24 * (1 + 1e-6) * rw.nan_to_num(0.0).abs()).all()
