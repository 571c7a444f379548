"""The 8-bit integer path at its documented limits on an MI355X: strides, row counts, columns and lengths up to the
largest that the calls accept, with offsets past 32 bits; weights, epsilons and rows at the ends of their types; sums
written over one of their terms; calls from two threads. All bit for bit.
"""
import threading

import numpy as np
import pytest
import torch

from mxfp4_block_scaled_02_amd import ops
from oracle import int8 as o8
from tests.test_gpu_int8 import Block, T, dev, host, same, say, values
from tests.test_gpu_int8_kernels import biases, check, marked, marks_left, operands, sums

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _free_large_buffers():
    yield
    torch.cuda.synchronize()
    torch.cuda.empty_cache()


@pytest.mark.parametrize("path,M,N,K", [
    ("skinny_16x16", 17, 33, 144), ("skinny_32x16", 17, 2050, 528), ("skinny_32x32", 33, 2050, 1040),
    ("ring_32x32", 33, 257, 16), ("ring_64x32", 257, 1030, 16), ("ring_64x64", 257, 2050, 16),
    ("ring_128x64", 515, 2050, 16), ("ring_128x128", 1030, 2050, 16), ("ring_128x256", 1030, 4100, 16),
    ("large_256x256", 2067, 3985, 272)])
def test_operands_of_the_largest_stride(path, M, N, K):
    """Rows of 2^22 bytes: a tile's offsets come to 2^30, the later tiles' to gigabytes."""
    say(f"[gemm_a8w8] stride 2^22 {path} M{M} N{N} K{K}")
    assert ops.a8w8_path(M, N, K) == path
    aq, a_s, bq, b_s = operands(M, N, K, 3, 1 << 22, 1 << 22)
    C = torch.empty((M, N), dtype=torch.bfloat16, device="cuda")
    ops.gemm_a8w8(aq, a_s, bq, b_s, out=C)
    check(C, sums(aq, bq), a_s, b_s, None, "bf16", path)


@pytest.mark.parametrize("path,M,N,K,dtype,ldc", [
    ("skinny_16x16", 17, 33, 144, "bf16", (1 << 28) + 1), ("skinny_32x32", 33, 2050, 1040, "fp32", (1 << 27) + 3),
    ("skinny_16x16", 3, 33, 144, "fp16", (1 << 32) + 1), ("ring_32x32", 33, 257, 16, "fp16", (1 << 27) + 1),
    ("ring_128x128", 1030, 2050, 16, "bf16", (1 << 22) + 1), ("large_256x256", 2067, 3985, 272, "fp32", (1 << 21) + 1),
    ("large_256x256", 2067, 3985, 272, "bf16", (1 << 21) + 2)])
def test_rows_of_c_past_32_bits(path, M, N, K, dtype, ldc):
    """The last rows of C start past 2^32 elements."""
    say(f"[gemm_a8w8] ldc {ldc} {path} M{M} N{N} K{K} {dtype}")
    assert ops.a8w8_path(M, N, K) == path and (M - 1) * ldc >= 1 << 32
    aq, a_s, bq, b_s = operands(M, N, K, 4)
    bias = biases(N, dtype, 6)
    buf, C = marked(M, N, dtype, ldc, 5)
    ops.gemm_a8w8(aq, a_s, bq, b_s, bias=bias, out=C)
    check(C.contiguous(), sums(aq, bq), a_s, b_s, bias, dtype, path)
    marks_left(buf, M, N, 5)


@pytest.mark.parametrize("M,N", [(1 << 24, 17), (3, 1 << 24), (40, 1 << 24), (1 << 24, 300)])
def test_most_rows_and_columns(M, N):
    """2^24 rows or columns; the operands repeat every 1021, so that a small product holds every value of C."""
    K, period = 16, 1021
    say(f"[gemm_a8w8] M{M} N{N} K{K} {ops.a8w8_path(M, N, K)}")
    m, n = min(M, period), min(N, period)
    aq, a_s, bq, b_s = operands(m, n, K, 7)
    small = ops.gemm_a8w8(aq, a_s, bq, b_s)
    check(small, sums(aq, bq), a_s, b_s, None, "bf16", "small")

    def repeated(t, count):
        return t.repeat(-(-count // t.shape[0]), *[1] * (t.dim() - 1))[:count]

    C = ops.gemm_a8w8(repeated(aq, M), repeated(a_s, M), repeated(bq, N), repeated(b_s, N))
    if M > N:
        for r in range(0, M // m, 512):  # whole periods of rows, many at a time
            k = min(512, M // m - r)
            assert bool((C[r * m:(r + k) * m].view(k, m, N) == small).all()), r
        assert torch.equal(C[M // m * m:], small[:M % m])
    else:
        k = N // n
        assert bool((C[:, :k * n].view(M, k, n) == small[:, None]).all())
        assert torch.equal(C[:, k * n:], small[:, :N % n])


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("K", [16, 1040, 7168, 33024])
def test_row_calls_with_rows_a_gigabyte_apart(K, dtype):
    """Six rows over more than 2^32 bytes in every argument."""
    say(f"[row calls] K{K} {dtype}")
    rng, M, size = np.random.default_rng(K), 6, torch.finfo(T[dtype]).bits // 8

    def far(v, t, ld):
        buf = torch.empty((M, ld), dtype=t, device="cuda")
        buf[:, :K] = v
        return buf[:, :K]

    x, r = values(rng, M, K, dtype), values(rng, M, K, dtype)
    w = o8.round_to(1 + 0.2 * rng.standard_normal(K), dtype)
    ld = (1 << 30) // size + 16
    xd, rd, wd = far(dev(x, dtype), T[dtype], ld), far(dev(r, dtype), T[dtype], ld + 16), dev(w[None], dtype)[0]
    q = far(0, torch.int8, (1 << 30) + 32)
    s = torch.empty(M, device="cuda")
    ops.int8_quant(xd, out=(q, s))
    qr, sr = o8.row_codes(x)
    same(s.cpu().numpy(), sr, "scales")
    same(q.cpu().numpy(), qr, "codes")
    h = far(0, T[dtype], ld + 32)
    ops.int8_rmsnorm_quant(xd, wd, 1e-6, residual=rd, out=(q, s, h))
    y, hr = o8.rmsnorm(x, w, 1e-6, dtype, residual=r)
    qr, sr = o8.row_codes(y)
    same(host(h), hr, "h")
    same(s.cpu().numpy(), sr, "scales")
    same(q.cpu().numpy(), qr, "codes")


def test_quant_of_more_than_2_to_the_32_bytes():
    M, K, period = 320003, 7168, 1021
    v = values(np.random.default_rng(1), period, K, "bf16")
    x = dev(v, "bf16").repeat(M // period + 1, 1)[:M]
    q, s = ops.int8_quant(x)
    qr, sr = o8.row_codes(v)
    same(q[:period].cpu().numpy(), qr, "codes")
    same(s[:period].cpu().numpy(), sr, "scales")
    n = M // period * period
    assert (q[:n].view(-1, period, K) == q[:period]).all() and (s[:n].view(-1, period) == s[:period]).all()
    assert torch.equal(q[n:], q[:M - n]) and torch.equal(s[n:], s[:M - n])


@pytest.mark.parametrize("M,dtype", [(1, "fp32"), (2, "bf16")])
def test_longest_rows(M, dtype):
    """K = 2^28. The values are quarters, so the sum of squares is exact in float64 in any order."""
    K = 1 << 28
    say(f"[row calls] M{M} K2^28 {dtype}")
    g = torch.Generator(device="cuda").manual_seed(8)

    def quarters(lo, hi, *shape):
        return (torch.randint(lo, hi, shape, generator=g, device="cuda", dtype=torch.int8).to(T[dtype]) * 0.25)

    def codes_of(y):  # one row of fp32 values
        s = max(np.float32(y.abs().max().item()) * np.float32(1 / np.float32(127)), np.float32(2.0 ** -126))
        return torch.round(y * float(np.float32(1) / s)).to(torch.int8), float(s)

    x, r, w = quarters(-12, 13, M, K), quarters(-12, 13, M, K), quarters(2, 7, K)
    q, s = ops.int8_quant(x)
    for i in range(M):
        qr, sr = codes_of(x[i].float())
        assert s[i].item() == sr and torch.equal(q[i], qr)
    q, s, h = ops.int8_rmsnorm_quant(x, w, 1e-6, residual=r)
    assert torch.equal(h, x + r)  # at most 24 quarters: exact in both types
    for i in range(M):
        ss = float(h[i].double().square().sum().item())
        inv = np.float32(1.0 / np.sqrt(ss / K + np.float64(np.float32(1e-6))))
        qr, sr = codes_of((h[i].float() * float(inv)) * w.float())
        assert s[i].item() == sr and torch.equal(q[i], qr)


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("eps", [2.0 ** -149, 1e-12, 1.0, 3.4028234663852886e38])
@pytest.mark.parametrize("K", [64, 2064, 33024])
def test_norm_of_rows_and_epsilons_at_the_ends_of_their_types(K, eps, dtype):
    """Rows of the type's largest values (their norm's factor is an fp32 subnormal for bf16 and fp32), of its smallest
    value and of zeros, under the smallest and largest epsilon."""
    rng = np.random.default_rng(K)
    top = float(torch.finfo(T[dtype]).max)
    tiny = {"bf16": 2.0 ** -133, "fp16": 2.0 ** -24, "fp32": 2.0 ** -149}[dtype]
    x = values(rng, 7, K, dtype)
    x[1] = np.where(rng.random(K) < 0.5, top, -top)
    x[2] = 0.0
    x[2, K - 1] = top
    x[3] = tiny
    x[4] = 0.0
    x[5, 5] = -np.inf
    w = o8.round_to(1 + 0.2 * rng.standard_normal(K), dtype)
    q, s = ops.int8_rmsnorm_quant(dev(x, dtype), dev(w[None], dtype)[0], eps)
    with np.errstate(all="ignore"):
        y, _ = o8.rmsnorm(x, w, eps, dtype)
    qr, sr = o8.row_codes(y)
    same(s.cpu().numpy(), sr, "scales")
    same(q.cpu().numpy(), qr, "codes")
    assert np.isnan(sr[5]) and np.isfinite(np.delete(sr, 5)).all()


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("K", [64, 2064, 33024])
@pytest.mark.parametrize("weight", ["zero", "nan", "inf", "largest"])
def test_norm_with_weights_at_the_ends_of_their_type(weight, K, dtype):
    rng = np.random.default_rng(K + 1)
    x = values(rng, 4, K, dtype)
    x[1] = 0.0
    x[2, 3] = np.inf
    w = o8.round_to(1 + 0.2 * rng.standard_normal(K), dtype)
    if weight == "zero":
        w[:] = 0.0
    elif weight == "largest":
        w[:] = float(torch.finfo(T[dtype]).max)
    else:
        w[K - 2] = np.nan if weight == "nan" else np.inf
    q, s = ops.int8_rmsnorm_quant(dev(x, dtype), dev(w[None], dtype)[0], 1e-5)
    with np.errstate(all="ignore"):
        y, _ = o8.rmsnorm(x, w, 1e-5, dtype)
    qr, sr = o8.row_codes(y)
    same(s.cpu().numpy(), sr, "scales")
    same(q.cpu().numpy(), qr, "codes")


@pytest.mark.parametrize("into", ["x", "residual"])
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("K", [256, 1040, 4112, 16384, 33024])
def test_stream_updated_in_place_in_every_type(K, dtype, into):
    """Padded rows, the sum written over one of its terms."""
    rng, M = np.random.default_rng(K), 5
    x, r = values(rng, M, K, dtype), values(rng, M, K, dtype)
    w = o8.round_to(1 + 0.2 * rng.standard_normal(K), dtype)
    xd, rd = dev(x, dtype, 16), dev(r, dtype, 32)
    q, s = torch.empty((M, K), dtype=torch.int8, device="cuda"), torch.empty(M, device="cuda")
    ops.int8_rmsnorm_quant(xd, dev(w[None], dtype)[0], 1e-5, residual=rd, out=(q, s, xd if into == "x" else rd))
    y, hr = o8.rmsnorm(x, w, 1e-5, dtype, residual=r)
    qr, sr = o8.row_codes(y)
    same(host(xd if into == "x" else rd), hr, "h")
    same(host(rd if into == "x" else xd), r if into == "x" else x, "the other term")
    same(s.cpu().numpy(), sr, "scales")
    same(q.cpu().numpy(), qr, "codes")


def test_block_from_two_threads_at_once():
    b = Block(64, 1040, 528)
    ins = [b.inputs() for _ in range(2)]
    devs = [(dev(x, "bf16"), dev(r, "bf16")) for x, r in ins]
    torch.cuda.synchronize()
    outs = [None, None]

    def work(i):
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(20):
                outs[i] = b.run(*devs[i])
            torch.cuda.current_stream().synchronize()

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    for (x, r), (h, c) in zip(ins, outs):
        hr, cr = b.ref(x, r)
        same(host(h), hr, "residual stream")
        same(host(c), cr, "output")
