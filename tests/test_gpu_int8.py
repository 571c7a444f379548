"""Parity of the 8-bit integer path with its oracle (``oracle.int8``) on an MI355X.

Codes, scales and the residual stream are fixed bit for bit by the definition
(every fp32 step rounds by itself; the float64 sum of squares may differ from the
exact sum in its last bits, which moves a row's inv only across an fp32 rounding
boundary: about 1e-7 of the rows). The product is fixed bit for bit too: the
integer sums are exact, the scaling steps round one by one.
"""
import numpy as np
import pytest
import torch

from mxfp4_block_scaled_02_amd import ops
from oracle import int8 as o8
from tests.test_int8_abi import PATH_SHAPES

pytestmark = pytest.mark.gpu

T = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp16": 2, "fp32": 4}
MIN_SCALE = np.float32(2.0 ** -126)


def say(*a):
    print(*a, flush=True)


def values(rng, M, K, dtype, spread=3.0):
    """Rows of different magnitude with a few outliers, as float32 holding values of `dtype`."""
    v = rng.standard_normal((M, K)) * 2.0 ** rng.uniform(-spread, spread, (M, 1))
    v[:, ::max(1, K // 5)] *= 12.0
    return o8.round_to(v, dtype)


def dev(v, dtype, pad=0):
    """On the GPU, as the first columns of rows padded by `pad` elements that must not matter."""
    t = torch.full((v.shape[0], v.shape[1] + pad), 77.0, dtype=T[dtype], device="cuda")
    t[:, :v.shape[1]] = torch.from_numpy(np.ascontiguousarray(v)).to("cuda").to(T[dtype])
    return t[:, :v.shape[1]]


def host(t):
    return t.float().cpu().numpy()


def same(got, want, what):
    assert got.shape == want.shape, what
    ok = (got == want) | (np.isnan(got) & np.isnan(want)) if got.dtype.kind == "f" else got == want
    assert ok.all(), f"{what}: {int((~ok).sum())} of {ok.size} differ, first at {np.argwhere(~ok)[:3].tolist()}"


def codes_buffers(M, K, pad):
    """Output buffers inside larger ones that are filled with marks."""
    q = torch.full((M + 2, K + pad), 99, dtype=torch.int8, device="cuda")
    s = torch.full((M + 2,), 99.0, device="cuda")
    return q, s


# Every row kernel: pieces of 16 bytes up to 64, 128, 256, 512, 1024, 2048, 4096 and past, both sides of each limit.
ROWS = [(1, 16), (3, 48), (6, 256), (5, 512), (4, 528), (2, 1024), (7, 1040), (2, 2048), (3, 2064), (2, 4096), (3, 4112),
        (9, 7168), (2, 8192), (3, 8208), (1, 16384), (2, 16400), (1, 32768), (2, 32784), (1, 100000)]


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("M,K", ROWS)
def test_quant(M, K, dtype):
    say(f"[int8_quant] M{M} K{K} {dtype}")
    v = values(np.random.default_rng(M * K), M, K, dtype)
    pad = 32
    q, s = codes_buffers(M, K, pad)
    ops.int8_quant(dev(v, dtype, pad), out=(q[:M, :K], s[:M]))
    qr, sr = o8.row_codes(v)
    same(s[:M].cpu().numpy(), sr, "scales")
    same(q[:M, :K].cpu().numpy(), qr, "codes")
    assert (q[M:] == 99).all() and (q[:, K:] == 99).all() and (s[M:] == 99).all(), "written outside the output"
    q2, s2 = ops.int8_quant(dev(v, dtype))
    assert torch.equal(q2, q[:M, :K]) and torch.equal(s2, s[:M])


@pytest.mark.parametrize("M", [1000, 5000])
def test_quant_many_rows(M):
    v = values(np.random.default_rng(M), M, 80, "bf16")
    q, s = ops.int8_quant(dev(v, "bf16"))
    qr, sr = o8.row_codes(v)
    same(s.cpu().numpy(), sr, "scales")
    same(q.cpu().numpy(), qr, "codes")


@pytest.mark.parametrize("M,K", [((1 << 20) + 3, 528), ((1 << 22) + 5, 16)])
def test_quant_more_rows_than_one_row_of_the_grid(M, K):
    """The rows around the limits (2^20 workgroups of one row, or of four) against the oracle, the others against
    themselves: the input repeats every 1021 rows."""
    v = values(np.random.default_rng(M), 1021, K, "bf16")
    x = dev(v, "bf16").repeat(M // 1021 + 1, 1)[:M]
    q, s = ops.int8_quant(x)
    qr, sr = o8.row_codes(v)
    rows = [0, 1, 1020, (1 << 20) - 1, 1 << 20, (1 << 20) + 1, M - 2, M - 1]
    at = np.array(rows) % 1021
    same(s[rows].cpu().numpy(), sr[at], "scales")
    same(q[rows].cpu().numpy(), qr[at], "codes")
    n = M // 1021 * 1021
    assert (q[:n].view(-1, 1021, K) == q[:1021]).all() and (s[:n].view(-1, 1021) == s[:1021]).all()


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("K", [64, 2064, 33024])
def test_quant_rows_at_the_edges(K, dtype):
    """Zeros, the type's smallest and largest values, Inf and NaN, each in a row of its own."""
    rng = np.random.default_rng(3)
    top = float(torch.finfo(T[dtype]).max)
    tiny = {"bf16": 2.0 ** -133, "fp16": 2.0 ** -24, "fp32": 2.0 ** -149}[dtype]
    v = values(rng, 10, K, dtype)
    v[1] = 0.0
    v[2] = -0.0
    v[3] = 0.0
    v[3, K - 1] = tiny
    v[4] = np.where(rng.random(K) < 0.5, top, -top)
    v[5, 7] = np.inf
    v[6, K - 1] = np.nan
    v[7, 0], v[7, 1] = -np.inf, np.nan
    v[8] = o8.round_to(rng.standard_normal(K) * 2.0 ** -120, dtype)
    q, s = ops.int8_quant(dev(v, dtype))
    qr, sr = o8.row_codes(v)
    same(s.cpu().numpy(), sr, "scales")
    same(q.cpu().numpy(), qr, "codes")
    assert sr[1] == MIN_SCALE and np.isnan(sr[5:8]).all()


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("M,K", ROWS)
def test_rmsnorm_quant(M, K, residual, dtype):
    say(f"[int8_rmsnorm_quant] M{M} K{K} {dtype} residual {residual}")
    rng = np.random.default_rng(M + K)
    x, w = values(rng, M, K, dtype), o8.round_to(1 + 0.2 * rng.standard_normal(K), dtype)
    r = values(rng, M, K, dtype) if residual else None
    y, h = o8.rmsnorm(x, w, 1e-6, dtype, residual=r)
    qr, sr = o8.row_codes(y)
    pad = 16
    q, s = codes_buffers(M, K, pad)
    wd = dev(w[None], dtype)[0]
    if not residual:
        ops.int8_rmsnorm_quant(dev(x, dtype, pad), wd, 1e-6, out=(q[:M, :K], s[:M]))
    else:
        hb = torch.full((M + 1, K + pad), 55.0, dtype=T[dtype], device="cuda")
        ops.int8_rmsnorm_quant(dev(x, dtype, pad), wd, 1e-6, residual=dev(r, dtype, 2 * pad),
                               out=(q[:M, :K], s[:M], hb[:M, :K]))
        same(host(hb[:M, :K]), h, "residual stream")
        assert (hb[M:] == 55).all() and (hb[:, K:] == 55).all(), "written outside h"
    same(s[:M].cpu().numpy(), sr, "scales")
    same(q[:M, :K].cpu().numpy(), qr, "codes")
    assert (q[M:] == 99).all() and (q[:, K:] == 99).all() and (s[M:] == 99).all(), "written outside the output"


@pytest.mark.parametrize("into", ["x", "residual"])
@pytest.mark.parametrize("M,K", [(5, 512), (6, 7168), (3, 33024)])
def test_rmsnorm_quant_updates_the_stream_in_place(M, K, into):
    rng = np.random.default_rng(K)
    x, r = values(rng, M, K, "bf16"), values(rng, M, K, "bf16")
    w = o8.round_to(1 + 0.2 * rng.standard_normal(K), "bf16")
    xd, rd, wd = dev(x, "bf16"), dev(r, "bf16"), dev(w[None], "bf16")[0]
    q, s = torch.empty((M, K), dtype=torch.int8, device="cuda"), torch.empty(M, device="cuda")
    h = xd if into == "x" else rd
    q, s, h = ops.int8_rmsnorm_quant(xd, wd, 1e-5, residual=rd, out=(q, s, h))
    y, hr = o8.rmsnorm(x, w, 1e-5, "bf16", residual=r)
    qr, sr = o8.row_codes(y)
    same(host(h), hr, "h")
    same(s.cpu().numpy(), sr, "scales")
    same(q.cpu().numpy(), qr, "codes")


@pytest.mark.parametrize("K", [64, 7168, 33024])
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
def test_rmsnorm_quant_rows_at_the_edges(K, dtype):
    rng = np.random.default_rng(4)
    x, r = values(rng, 8, K, dtype), values(rng, 8, K, dtype)
    w = o8.round_to(1 + 0.2 * rng.standard_normal(K), dtype)
    x[1], r[1] = 0.0, 0.0
    x[2], r[2] = 0.0, 0.0
    x[2, 3] = {"bf16": 2.0 ** -133, "fp16": 2.0 ** -24, "fp32": 2.0 ** -149}[dtype]
    x[3], r[3] = 5.0, -5.0                       # the sum cancels
    x[4, K - 1] = np.inf
    r[5, 0] = np.nan
    x[6, 2] = r[6, 2] = float(torch.finfo(T[dtype]).max)  # the sum overflows the type
    q, s, h = ops.int8_rmsnorm_quant(dev(x, dtype), dev(w[None], dtype)[0], 1e-6, residual=dev(r, dtype))
    with np.errstate(all="ignore"):
        y, hr = o8.rmsnorm(x, w, 1e-6, dtype, residual=r)
    qr, sr = o8.row_codes(y)
    same(host(h), hr, "h")
    same(s.cpu().numpy(), sr, "scales")
    same(q.cpu().numpy(), qr, "codes")
    assert np.isnan(sr[4:7]).all() and (qr[4:7] == 0).all() and (qr[1] == 0).all()


def operands(rng, M, N, K, full=False):
    lo, hi = (-128, 128) if full else (-127, 128)
    aq, bq = (rng.integers(lo, hi, (n, K)).astype(np.int8) for n in (M, N))
    return aq, (rng.random(M) * 0.04 + 0.01).astype(np.float32), bq, (rng.random(N) * 8e-4 + 2e-4).astype(np.float32)


def dev8(v, pad=0, rows=0):
    t = torch.full((v.shape[0] + rows, v.shape[1] + pad), 101, dtype=torch.int8, device="cuda")
    t[:v.shape[0], :v.shape[1]] = torch.from_numpy(v).cuda()
    return t[:v.shape[0], :v.shape[1]]


def check_gemm(rng, M, N, K, dtype="bf16", bias=False, pads=(0, 0, 0), full=False):
    say(f"[gemm_a8w8] M{M} N{N} K{K} {dtype} bias {bias} pads {pads}")
    aq, a_s, bq, b_s = operands(rng, M, N, K, full)
    bv = o8.round_to(rng.standard_normal(N), dtype) if bias else None
    C = torch.full((M + 1, N + pads[2]), 33.0, dtype=T[dtype], device="cuda")
    ops.gemm_a8w8(dev8(aq, pads[0]), torch.from_numpy(a_s).cuda(), dev8(bq, pads[1]), torch.from_numpy(b_s).cuda(),
                  bias=None if bv is None else torch.from_numpy(bv).cuda().to(T[dtype]), out=C[:M, :N])
    got = host(C[:M, :N])
    same(got, o8.round_to(o8.gemm(aq, a_s, bq, b_s, bv), dtype), "C")
    assert (C[M:] == 33).all() and (C[:, N:] == 33).all(), "written outside C"
    # and against 64 bits: half a step of the type, the conversion of acc, two products and the sum in fp32
    want = o8.gemm_f64(aq, a_s, bq, b_s, bv)
    size = np.abs(want) + (0 if bv is None else 2 * np.abs(bv)[None, :])
    eps = torch.finfo(T[dtype]).eps / 2
    tiny = float(torch.finfo(T[dtype]).smallest_normal) * eps * 2
    assert (np.abs(got - want) <= np.abs(want) * eps + size * (1 + eps) * 4 * 2.0 ** -24 + tiny).all()


# Small products with extents around the tiles', K inside a step and over many; they take the skinny kernels and the
# ring tiles to 64 x 64 (PATH_SHAPES reaches every kernel, test_gpu_int8_kernels.py with every type).
SHAPES = [(1, 1, 16), (1, 16, 64), (4, 256, 512), (3, 17, 48), (16, 33, 128), (17, 15, 144), (16, 264, 7168),
          (1, 100, 8192), (32, 130, 2064), (33, 70, 1040), (48, 257, 528), (64, 64, 256), (65, 129, 272), (100, 31, 4096),
          (127, 255, 400), (128, 256, 1024), (129, 257, 1040), (200, 512, 2048), (255, 300, 96), (256, 256, 128),
          (257, 511, 1936), (300, 1000, 640), (511, 513, 272), (513, 1025, 336), (600, 90, 208)]


@pytest.mark.parametrize("path,M,N,K", PATH_SHAPES)
def test_gemm_paths(path, M, N, K):
    check_gemm(np.random.default_rng(M + N + K), M, N, K, "fp32", True, (16, 32, 0))
    check_gemm(np.random.default_rng(M + N + K + 1), M, N, K, "bf16", False, (0, 0, 6), full=True)


@pytest.mark.parametrize("M,N,K", SHAPES)
def test_gemm(M, N, K):
    rng = np.random.default_rng(M * 7 + N * 3 + K)
    for dtype, bias, pads in [("bf16", False, (0, 0, 0)), ("fp16", True, (16, 48, 3)), ("fp32", True, (32, 16, 1))]:
        check_gemm(rng, M, N, K, dtype, bias, pads)


@pytest.mark.parametrize("M,N,K", [(2, 3, 131056), (70, 40, 131056), (300, 270, 16400)])
def test_gemm_long_sums(M, N, K):
    """All codes -128: the largest sums that the longest K gives, 128 * 128 * K < 2^31; then random ones of all 256."""
    aq, a_s, bq, b_s = operands(np.random.default_rng(0), M, N, K)
    aq[:], bq[:] = -128, -128
    c = ops.gemm_a8w8(dev8(aq), torch.from_numpy(a_s).cuda(), dev8(bq), torch.from_numpy(b_s).cuda(),
                      out_dtype=torch.float32)
    same(host(c), o8.gemm(aq, a_s, bq, b_s), "C")
    check_gemm(np.random.default_rng(1), M, N, K, "fp32", full=True)


@pytest.mark.parametrize("M,N,K", [(2100, 1030, 512), (4096, 4096, 256), (1024, 4160, 1040), (5000, 300, 144),
                                   (20, 20000, 160), (130, 9000, 272)])
def test_gemm_many_tiles(M, N, K):
    check_gemm(np.random.default_rng(9), M, N, K)


def test_gemm_rows_do_not_depend_on_the_other_rows():
    """One token's result is the same alone, in a decode batch, and in a prompt."""
    rng = np.random.default_rng(12)
    aq, a_s, bq, b_s = operands(rng, 700, 520, 2064)
    a, s, b, t = dev8(aq), torch.from_numpy(a_s).cuda(), dev8(bq), torch.from_numpy(b_s).cuda()
    whole = ops.gemm_a8w8(a, s, b, t)
    for n in (1, 8, 16, 17, 40, 64, 65, 128, 200, 256, 400):
        assert torch.equal(ops.gemm_a8w8(a[:n], s[:n], b, t), whole[:n]), n


@pytest.mark.parametrize("M", [3, 40, 300])
def test_gemm_scales_that_are_not_finite_reach_their_rows_only(M):
    rng = np.random.default_rng(13)
    aq, a_s, bq, b_s = operands(rng, M, 80, 256)
    a_s[1] = np.nan
    b_s[5] = np.inf
    aq[2] = 0  # 0 * Inf
    c = host(ops.gemm_a8w8(dev8(aq), torch.from_numpy(a_s).cuda(), dev8(bq), torch.from_numpy(b_s).cuda()))
    same(c, o8_bf16(o8.gemm(aq, a_s, bq, b_s)), "C")
    assert np.isnan(c[1]).all() and np.isnan(c[2, 5]) and np.isfinite(np.delete(np.delete(c, 1, 0), 5, 1)).all()


def o8_bf16(v):
    ok = np.isfinite(v)
    return np.where(ok, o8.round_to(np.where(ok, v, 0), "bf16"), v).astype(np.float32)


def test_gemm_overflow_of_fp16_is_infinite():
    aq, bq = np.full((5, 64), 127, np.int8), np.full((20, 64), 127, np.int8)
    bq[3] = -127
    c = host(ops.gemm_a8w8(dev8(aq), torch.ones(5, device="cuda"), dev8(bq), torch.ones(20, device="cuda"),
                           out_dtype=torch.float16))
    assert (c[:, 3] == -np.inf).all() and (np.delete(c, 3, 1) == np.inf).all()


class Block:
    """Norm -> product -> quantisation -> product on a residual stream, as a layer runs them."""

    def __init__(self, M, K, F, seed=20):
        self.rng = np.random.default_rng(seed)
        self.M, self.K, self.F = M, K, F
        self.w = o8.round_to(1 + 0.2 * self.rng.standard_normal(K), "bf16")
        self.wd = dev(self.w[None], "bf16")[0]
        w1, w2 = self.rng.standard_normal((F, K)) * 0.05, self.rng.standard_normal((K, F)) * 0.05
        self.b1, self.s1 = ops.int8_quant(dev(w1, "bf16"))
        self.b2, self.s2 = ops.int8_quant(dev(w2, "bf16"))

    def inputs(self):
        return values(self.rng, self.M, self.K, "bf16"), values(self.rng, self.M, self.K, "bf16")

    def run(self, x, r):
        q, s, h = ops.int8_rmsnorm_quant(x, self.wd, 1e-6, residual=r)
        u = ops.gemm_a8w8(q, s, self.b1, self.s1)
        q2, s2 = ops.int8_quant(u)
        return h, ops.gemm_a8w8(q2, s2, self.b2, self.s2)

    def ref(self, x, r):
        y, h = o8.rmsnorm(x, self.w, 1e-6, "bf16", residual=r)
        q, s = o8.row_codes(y)
        n = lambda t: t.cpu().numpy()  # noqa: E731
        u = o8.round_to(o8.gemm(q, s, n(self.b1), n(self.s1)), "bf16")
        q2, s2 = o8.row_codes(u)
        return h, o8.round_to(o8.gemm(q2, s2, n(self.b2), n(self.s2)), "bf16")


@pytest.mark.parametrize("M", [1, 16, 70, 300])
def test_block(M):
    b = Block(M, 1040, 528)
    x, r = b.inputs()
    h, c = b.run(dev(x, "bf16"), dev(r, "bf16"))
    hr, cr = b.ref(x, r)
    same(host(h), hr, "residual stream")
    same(host(c), cr, "output")


@pytest.mark.parametrize("M", [4, 300])
def test_block_captured_and_replayed(M):
    """Replays on new data in the same buffers, eager work and another graph of the same block in between."""
    b = Block(M, 528, 1040)
    x, r = (dev(v, "bf16") for v in b.inputs())
    graphs = []
    for _ in range(2):
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            out = b.run(x, r)
        graphs.append((g, out))
    torch.cuda.synchronize()
    for i in range(4):
        say(f"replay {i}")
        nx, nr = b.inputs()
        x.copy_(torch.from_numpy(nx))
        r.copy_(torch.from_numpy(nr))
        eager = b.run(x, r)
        torch.cuda.synchronize()
        for g, out in graphs:
            g.replay()
        torch.cuda.synchronize()
        hr, cr = b.ref(nx, nr)
        for got in [eager] + [o for _, o in graphs]:
            same(host(got[0]), hr, "residual stream")
            same(host(got[1]), cr, "output")


def test_block_on_two_streams_at_once():
    b = Block(64, 1040, 528)
    ins = [b.inputs() for _ in range(6)]
    devs = [(dev(x, "bf16"), dev(r, "bf16")) for x, r in ins]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    outs = []
    for i, (x, r) in enumerate(devs):
        with torch.cuda.stream(streams[i % 2]):
            outs.append(b.run(x, r))
    torch.cuda.synchronize()
    for (x, r), (h, c) in zip(ins, outs):
        hr, cr = b.ref(x, r)
        same(host(h), hr, "residual stream")
        same(host(c), cr, "output")


def test_runs_repeat_bit_for_bit():
    b = Block(40, 2064, 528)
    x, r = (dev(v, "bf16") for v in b.inputs())
    first = b.run(x, r)
    for _ in range(5):
        again = b.run(x, r)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


def test_binding_refusals_on_the_device():
    x = torch.zeros((4, 64), dtype=torch.bfloat16, device="cuda")
    q, s = ops.int8_quant(x)
    w = torch.ones(64, dtype=torch.bfloat16, device="cuda")
    for bad in (x[:, ::2], x.double(), x[0], x.t()):
        with pytest.raises((ValueError, ops.Mxfp4Error)):
            ops.int8_quant(bad)
    with pytest.raises(ops.Mxfp4Error, match="SHAPE"):
        ops.int8_quant(x[:0])
    with pytest.raises(ops.Mxfp4Error, match="SHAPE"):
        ops.int8_quant(x[:, :24])
    with pytest.raises(ops.Mxfp4Error, match="ALIGN"):
        ops.int8_quant(x[:, 4:20])
    with pytest.raises(ValueError, match="q must be"):
        ops.int8_quant(x, out=(q[:3], s))
    with pytest.raises(ValueError, match="s must be"):
        ops.int8_quant(x, out=(q, s.double()))
    with pytest.raises(ValueError, match="w must be"):
        ops.int8_rmsnorm_quant(x, w.float(), 1e-6)
    with pytest.raises(ValueError, match="residual must be"):
        ops.int8_rmsnorm_quant(x, w, 1e-6, residual=x.half())
    with pytest.raises(ops.Mxfp4Error, match="ARG"):
        ops.int8_rmsnorm_quant(x, w, 0.0)
    with pytest.raises(ValueError, match="a_scale"):
        ops.gemm_a8w8(q, s[:3], q, s)
    with pytest.raises(ValueError, match="bq must be"):
        ops.gemm_a8w8(q, s, q[:, :32], s)
    with pytest.raises(ValueError, match="aq must be"):
        ops.gemm_a8w8(x, s, q, s)
    with pytest.raises(ValueError, match="bias must be"):
        ops.gemm_a8w8(q, s, q, s, bias=torch.zeros(4, device="cuda"))
    with pytest.raises(ValueError, match="out_dtype"):
        ops.gemm_a8w8(q, s, q, s, out_dtype=torch.int32)
    with pytest.raises(ValueError, match="out must be"):
        ops.gemm_a8w8(q, s, q, s, out=x[:, :3])
    with pytest.raises(ValueError, match="on device 0"):
        ops.gemm_a8w8(q, s, q.cpu(), s)
