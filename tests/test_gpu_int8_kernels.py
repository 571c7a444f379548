"""gemm_a8w8 on an MI355X, every kernel with every type of C, with and without a bias, at lengths from one step of K.

The expected value is the definition in torch on the device: the integer sums as a float64 product (whole numbers below
2^53, exact), then one fp32 operation for each step that rounds to fp32, and one conversion. Equality is bit for bit;
against 64 bits the bound counts the conversion of the sum, two products and the bias's addition in fp32 and half a
step of the type of C.
"""
import pytest
import torch

from mxfp4_block_scaled_02_amd import ops
from tests.test_gpu_int8 import T, say
from tests.test_int8_abi import PATH_SHAPES
from tests.test_int8_short_k import SHORT_K

pytestmark = pytest.mark.gpu


def operands(M, N, K, seed, lda=None, ldb=None):
    """Codes of all 256 values, in the last columns of rows of lda and ldb bytes: the last row ends the buffer."""
    g = torch.Generator(device="cuda").manual_seed(seed)

    def codes(rows, ld):
        t = torch.full((rows, ld), 101, dtype=torch.int8, device="cuda")
        t[:, ld - K:] = torch.randint(-128, 128, (rows, K), generator=g, device="cuda", dtype=torch.int8)
        return t[:, ld - K:]

    return (codes(M, lda or K), torch.rand(M, generator=g, device="cuda") * 0.04 + 0.01,
            codes(N, ldb or K), torch.rand(N, generator=g, device="cuda") * 8e-4 + 2e-4)


def biases(N, dtype, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (3 * torch.randn(N, generator=g, device="cuda")).to(T[dtype])


def sums(aq, bq):
    return aq.double() @ bq.double().t()


def check(got, acc, a_s, b_s, bias, dtype, what):
    want = acc.float() * a_s[:, None] * b_s[None, :]
    exact = acc * a_s.double()[:, None] * b_s.double()[None, :]
    size = exact.abs()
    if bias is not None:
        want = want + bias.float()
        exact = exact + bias.double()
        size = exact.abs() + 2 * bias.double().abs()
    assert torch.equal(got, want.to(T[dtype])), what
    eps = torch.finfo(T[dtype]).eps / 2
    tiny = float(torch.finfo(T[dtype]).smallest_normal) * eps * 2
    bound = exact.abs() * eps + size * ((1 + eps) * 4 * 2.0 ** -24) + tiny
    assert bool(((got.double() - exact).abs() <= bound).all()), what


def marked(M, N, dtype, ld, at):
    """A buffer of marks with one row more than C, and C inside it from column `at` on."""
    buf = torch.full((M + 1, ld), 33.0, dtype=T[dtype], device="cuda")
    return buf, buf[:M, at:at + N]


def marks_left(buf, M, N, at):
    assert bool((buf[M:] == 33).all())
    step = max(1, (1 << 28) // buf.shape[1])
    for m in range(0, M, step):  # in parts: a mask of the whole would be as large as C
        rows = buf[m:min(M, m + step)]
        assert bool((rows[:, :at] == 33).all()) and bool((rows[:, at + N:] == 33).all()), "written outside C"


@pytest.mark.parametrize("path,M,N,K", PATH_SHAPES + SHORT_K)
def test_every_kernel_with_every_type_and_bias(path, M, N, K):
    """C starts at an odd element of rows of another length; A and B are padded."""
    say(f"[gemm_a8w8] {path} M{M} N{N} K{K}")
    assert ops.a8w8_path(M, N, K) == path
    aq, a_s, bq, b_s = operands(M, N, K, M + N + K, K + 16, K + 48)
    acc = sums(aq, bq)
    for dtype in T:
        for bias in (None, biases(N, dtype, N)):
            buf, C = marked(M, N, dtype, N + 9, 3)
            ops.gemm_a8w8(aq, a_s, bq, b_s, bias=bias, out=C)
            check(C, acc, a_s, b_s, bias, dtype, f"{path} {dtype} bias {bias is not None}")
            marks_left(buf, M, N, 3)


@pytest.mark.parametrize("N,K,rows,paths", [
    (3001, 528, (1, 32, 33, 100, 300, 640, 1000, 2000, 2700),
     ["skinny_16x16", "skinny_32x16", "ring_32x32", "ring_64x32", "ring_64x64", "ring_128x64", "ring_128x128",
      "ring_128x256", "large_256x256"]),
    (2051, 1040, (16, 17, 90, 150, 250, 500, 1000, 1930, 3900),
     ["skinny_16x16", "skinny_32x16", "skinny_32x32", "ring_64x32", "ring_64x64", "ring_128x64", "ring_128x128",
      "ring_128x256", "large_256x256"])])
def test_rows_are_the_same_on_every_kernel(N, K, rows, paths):
    """A token's row of C alone, in batches of every size and in a prompt: one result on all ten kernels."""
    assert [ops.a8w8_path(m, N, K) for m in rows] == paths
    aq, a_s, bq, b_s = operands(rows[-1], N, K, K)
    for dtype in ("bf16", "fp32"):
        bias = biases(N, dtype, 5)
        whole = ops.gemm_a8w8(aq, a_s, bq, b_s, bias=bias, out_dtype=T[dtype])
        for m in rows[:-1]:
            assert torch.equal(ops.gemm_a8w8(aq[:m], a_s[:m], bq, b_s, bias=bias, out_dtype=T[dtype]), whole[:m]), m
