"""Low-rank adapters of many requests against a plain form in 64 bits."""
import math

import pytest
import torch

from mxfp4_block_scaled_02_amd import ops
from tests import picked

pytestmark = pytest.mark.gpu


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def case(seed, T, K, N, R, n, dtype, out):
    g = gen(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    return dict(y=normal(T, N).to(out), x=normal(T, K).to(dtype), a=(normal(n, R, K) / math.sqrt(K)).to(dtype),
                b=(normal(n, N, R) / math.sqrt(R)).to(dtype),
                index=torch.randint(-1, n, (T,), generator=g, device="cuda").int(),
                scale=torch.rand(n, generator=g, device="cuda") + 0.5)


def check(c):
    ref, bound = picked.adapters(**c)
    before = c["y"].clone()
    y = ops.lora_add(c["y"], c["x"], c["a"], c["b"], c["index"], scale=c["scale"])
    assert y is c["y"]
    off = (y.double() - ref).abs()
    assert (off <= bound).all(), (off / bound).max().item()
    none = (c["index"] < 0) | (c["index"] >= c["a"].shape[0])
    assert torch.equal(y[none], before[none])
    return y


TYPES = [(torch.bfloat16, torch.bfloat16), (torch.bfloat16, torch.float32), (torch.float16, torch.float16),
         (torch.float16, torch.float32)]


@pytest.mark.parametrize("dtype,out", TYPES)
@pytest.mark.parametrize("T,K,N,R,n", [
    (1, 8, 1, 8, 1), (1, 512, 256, 16, 4), (1, 7168, 2112, 16, 8), (3, 40, 17, 8, 2), (16, 128, 64, 24, 3),
    (17, 136, 65, 32, 40), (64, 2048, 300, 40, 24), (100, 264, 1023, 64, 7), (33, 1000, 257, 72, 5), (50, 96, 511, 128, 3),
    (777, 520, 333, 24, 5), (2049, 64, 48, 104, 9), (65, 72, 40, 8, 3),
    (256, 96, 70, 16, 60), (300, 64, 33, 8, 300), (2100, 136, 130, 16, 2),
])
def test_adapters(T, K, N, R, n, dtype, out):
    check(case(T + K + N, T, K, N, R, n, dtype, out))


@pytest.mark.parametrize("dtype,out", TYPES)
def test_without_scales_and_without_adapters(dtype, out):
    c = case(1, 40, 256, 130, 16, 4, dtype, out)
    c["scale"] = None
    check(c)
    c = case(2, 40, 256, 130, 16, 4, dtype, out)
    c["index"][:16] = -1               # a whole tile without an adapter
    c["index"][20], c["index"][21], c["index"][22] = 4, 2 ** 31 - 1, -2 ** 31
    check(c)
    c["index"][:] = -1
    before = c["y"].clone()
    ops.lora_add(**{k: v for k, v in c.items()})
    assert torch.equal(c["y"], before)


@pytest.mark.parametrize("dtype,out", TYPES)
def test_row_strides_and_odd_addresses(dtype, out):
    c = case(3, 21, 72, 75, 16, 3, dtype, out)
    wide = torch.full((21, 88), math.nan, device="cuda").to(dtype)
    wide[:, 8:80] = c["x"]
    y = torch.full((21, 79), 7.0, device="cuda").to(out)
    y[:, 3:78] = c["y"]
    c["x"], c["y"] = wide[:, 8:80], y[:, 3:78]
    check(c)
    assert (y[:, :3] == 7).all() and (y[:, 78:] == 7).all()


@pytest.mark.parametrize("dtype,out", TYPES)
def test_a_row_depends_on_itself_and_its_adapter_alone(dtype, out):
    c = case(4, 50, 264, 200, 24, 4, dtype, out)
    y0 = c["y"].clone()
    y = ops.lora_add(**c)
    d = dict(c, y=y0.clone())
    d["x"] = c["x"].clone()
    d["x"][7, 3], d["x"][8] = math.inf, math.nan
    d["a"] = c["a"].clone()
    d["a"][2, 0, 5] = math.nan         # an adapter that is not finite
    ops.lora_add(**d)
    hit = (c["index"] == 2)
    hit[7:9] = True
    assert torch.equal(d["y"][~hit], y[~hit])
    bad = hit & (c["index"] >= 0)
    assert not torch.isfinite(d["y"][bad]).all(dim=1).any()


def test_fp16_products_past_the_type_and_far_below_it():
    """x . A^T of 1e6 and of 1e-7: neither is an fp16 number (or one of few bits); their products with B are."""
    for up, down in ((64.0, 2.0 ** -14), (2.0 ** -12, 8.0)):
        c = case(5, 20, 4096, 96, 16, 2, torch.float16, torch.float16)
        c["x"] = (c["x"].float().abs() * up).half()
        c["a"] = (c["a"].float().abs() * (16.0 if up > 1 else 2.0 ** -6)).half()
        c["b"] = (c["b"].float() * down).half()
        check(c)


def test_rows_past_32_bit_offsets():
    """y and x with rows so far apart that the last ones lie past 2^32 bytes."""
    c = case(6, 40, 64, 48, 16, 3, torch.bfloat16, torch.bfloat16)
    ld = (1 << 31) // 32  # elements: row 32 begins at 2^32 bytes
    y = torch.zeros(40 * ld, dtype=torch.bfloat16, device="cuda").as_strided((40, 48), (ld, 1))
    x = torch.zeros(40 * ld, dtype=torch.bfloat16, device="cuda").as_strided((40, 64), (ld, 1))
    y.copy_(c["y"])
    x.copy_(c["x"])
    c["y"], c["x"] = y, x
    check(c)


def test_beside_a_quantised_projection_captured_and_replayed():
    """The MXFP4 product and the adapters on it, in a graph that is replayed with new inputs."""
    T, K, N, R, n = 24, 512, 320, 16, 5
    c = case(7, T, K, N, R, n, torch.bfloat16, torch.bfloat16)
    bq, bs = ops.quant((torch.randn(N, K, generator=gen(8), device="cuda") / 16).bfloat16())
    bp = ops.pack_B(bq, bs)

    def run():
        return ops.lora_add(ops.gemm(c["x"], bp, N), c["x"], c["a"], c["b"], c["index"], scale=c["scale"])

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        run()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = run()
    for i in range(4):
        c["x"].copy_(torch.randn(T, K, generator=gen(30 + i), device="cuda"))
        c["index"].copy_(torch.randint(-1, n, (T,), generator=gen(40 + i), device="cuda"))
        eager = run()
        y.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, eager)
        ref, bound = picked.adapters(ops.gemm(c["x"], bp, N), c["x"], c["a"], c["b"], c["index"], c["scale"])
        assert ((y.double() - ref).abs() <= bound).all()


def test_workspace_contents_do_not_matter_and_its_end_is_kept():
    """The C call with a workspace of NaNs, and bytes behind it that stay."""
    for T, n in ((3, 2), (64, 5), (65, 5), (300, 400), (2500, 7), (5000, 3)):
        c = case(T, T, 520, 130, 24, n, torch.float16, torch.float16)
        y0 = c["y"].clone()
        y = ops.lora_add(**c)
        size = ops.lib().lora_add_workspace_bytes(T, 520, 24, n)
        ws = torch.full((size + 256,), 0xFF, dtype=torch.uint8, device="cuda")
        rc = ops.lib().lora_add(y0.data_ptr(), 130, 1, c["x"].data_ptr(), 520, 1, c["a"].data_ptr(), c["b"].data_ptr(),
                                c["index"].data_ptr(), c["scale"].data_ptr(), T, 130, 520, 24, n, ws.data_ptr(), size,
                                torch.cuda.current_stream().cuda_stream)
        assert rc == 0 and torch.equal(y0, y) and (ws[size:] == 0xFF).all()


@pytest.mark.parametrize("T", [4095, 4096, 4097, 9000])
def test_more_rows_than_a_block(T):
    check(case(T, T, 40, 33, 8, 6, torch.bfloat16, torch.float32))
    c = case(T, T, 40, 33, 8, 6, torch.bfloat16, torch.bfloat16)
    c["index"][:] = 4                  # one adapter for all
    check(c)
    c["index"][:] = torch.arange(T, device="cuda") * 7 // T - 1   # spans, the first without one
    check(c)


def test_as_many_adapters_as_there_may_be():
    c = case(9, 5000, 16, 20, 8, 4096, torch.bfloat16, torch.bfloat16)
    check(c)
    c = case(10, 60, 16, 20, 8, 4096, torch.bfloat16, torch.bfloat16)
    check(c)


def test_two_captured_graphs_replayed_at_once():
    """Each graph has its own scratch memory: replays on two streams do not meet in it."""
    cases = [case(30 + i, 600, 2048, 1024, 32, 6, torch.bfloat16, torch.bfloat16) for i in range(2)]
    start = [c["y"].clone() for c in cases]
    want = [ops.lora_add(**dict(c, y=y.clone())) for c, y in zip(cases, start)]
    torch.cuda.synchronize()
    graphs = []
    for c in cases:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            ops.lora_add(**c)
        graphs.append(g)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(10):
        for c, y in zip(cases, start):
            c["y"].copy_(y)
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        assert torch.equal(cases[0]["y"], want[0]) and torch.equal(cases[1]["y"], want[1])


@pytest.mark.parametrize("T,n", [(40, 3), (400, 3), (400, 90), (5000, 40)])
def test_calls_on_two_streams_at_once(T, n):
    cases = [case(50 + i, T, 520, 264, 16, n, torch.bfloat16, torch.float32) for i in range(2)]
    want = [ops.lora_add(**dict(c, y=c["y"].clone())) for c in cases]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream(), torch.cuda.Stream()], [[], []]
    for _ in range(10):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(ops.lora_add(**dict(cases[i], y=cases[i]["y"].clone())))
    torch.cuda.synchronize()
    for g, w in zip(got, want):
        assert all(torch.equal(y, w) for y in g)


@pytest.mark.parametrize("N,n", [(255, 23), (256, 23), (24 * 256, 15), (25 * 256, 16)])
def test_either_side_of_the_way_a_unit_is_taken(N, n):
    """Whole units of 64 rows or a tile at a time; spans and rows in any order."""
    for dtype, out in TYPES:
        c = case(N + n, 64, 72, N, 24, n, dtype, out)
        check(c)
        c["index"][:] = n - 1
        check(c)
        c = case(N, 200, 72, N, 24, n, dtype, out)
        c["index"][:] = torch.arange(200, device="cuda") // 90
        check(c)
