"""The 8-bit integer entry points without a GPU: every refusal of the C ABI comes
before any HIP call, and the Python binding refuses what it cannot marshal."""
import pytest
import torch

from mxfp4_block_scaled_02_amd import ops

P = 1 << 20  # a fake, aligned "device pointer": validation never dereferences it
Q = dict(x=P, ldx=64, dtype=0, q=P, ldq=64, s=P, M=4, K=64)


@pytest.mark.parametrize("change,status", [
    (dict(x=None), 1), (dict(q=None), 1), (dict(s=None), 1),
    (dict(dtype=3), 8), (dict(dtype=-1), 8),
    (dict(M=0), 2), (dict(M=-1), 2), (dict(M=(1 << 30) + 1), 2), (dict(K=0), 2), (dict(K=8), 2), (dict(K=72), 2),
    (dict(K=(1 << 28) + 16, ldx=1 << 29, ldq=1 << 29), 2), (dict(ldx=48), 2), (dict(ldq=48), 2), (dict(ldx=0), 2),
    (dict(ldx=1 << 60), 2), (dict(ldq=1 << 62), 2), (dict(ldx=-64), 2),
    (dict(x=P + 8), 3), (dict(q=P + 8), 3), (dict(s=P + 2), 3), (dict(ldx=68), 3), (dict(ldq=72), 3),
    (dict(ldx=66, dtype=2), 3),
])
def test_int8_quant_refusals(change, status):
    a = dict(Q, **change)
    assert ops.lib().int8_quant(a["x"], a["ldx"], a["dtype"], a["q"], a["ldq"], a["s"], a["M"], a["K"], None) == status


R = dict(x=P, ldx=64, residual=P, ldr=64, w=P, eps=1e-6, dtype=0, h=P, ldh=64, q=P, ldq=64, s=P, M=4, K=64)


@pytest.mark.parametrize("change,status", [
    (dict(x=None), 1), (dict(w=None), 1), (dict(q=None), 1), (dict(s=None), 1), (dict(h=None), 1),
    (dict(residual=None), 1),  # h without a residual
    (dict(dtype=7), 8), (dict(eps=0.0), 8), (dict(eps=-1e-6), 8), (dict(eps=float("nan")), 8),
    (dict(eps=float("inf")), 8),
    (dict(M=0), 2), (dict(K=0), 2), (dict(K=40), 2), (dict(ldx=48), 2), (dict(ldr=48), 2), (dict(ldh=48), 2),
    (dict(ldq=48), 2), (dict(ldr=1 << 60), 2), (dict(ldh=1 << 60), 2),
    (dict(x=P + 8), 3), (dict(w=P + 2), 3), (dict(residual=P + 4), 3), (dict(h=P + 4), 3), (dict(ldr=68), 3),
    (dict(ldh=68), 3), (dict(q=P + 4), 3), (dict(s=P + 1), 3),
])
def test_int8_rmsnorm_quant_refusals(change, status):
    a = dict(R, **change)
    got = ops.lib().int8_rmsnorm_quant(a["x"], a["ldx"], a["residual"], a["ldr"], a["w"], a["eps"], a["dtype"], a["h"],
                                       a["ldh"], a["q"], a["ldq"], a["s"], a["M"], a["K"], None)
    assert got == status


G = dict(A=P, lda=64, a_s=P, B=P, ldb=64, b_s=P, bias=None, C=P, ldc=32, ctype=0, M=4, N=32, K=64)


@pytest.mark.parametrize("change,status", [
    (dict(A=None), 1), (dict(a_s=None), 1), (dict(B=None), 1), (dict(b_s=None), 1), (dict(C=None), 1),
    (dict(ctype=3), 8), (dict(ctype=-1), 8),
    (dict(M=0), 2), (dict(N=0), 2), (dict(K=0), 2), (dict(K=24), 2), (dict(K=131072, lda=131072, ldb=131072), 2),
    (dict(M=(1 << 24) + 1), 2), (dict(N=(1 << 24) + 1, ldc=1 << 25), 2),
    (dict(M=1 << 24, N=1 << 24, ldc=1 << 24), 2),
    (dict(lda=48), 2), (dict(ldb=48), 2), (dict(ldc=31), 2), (dict(lda=(1 << 22) + 16), 2),
    (dict(ldb=(1 << 22) + 16), 2), (dict(ldc=(1 << 36) + 1), 2), (dict(lda=-64), 2),
    (dict(A=P + 8), 3), (dict(B=P + 4), 3), (dict(lda=72), 3), (dict(ldb=72), 3), (dict(a_s=P + 2), 3),
    (dict(b_s=P + 1), 3), (dict(C=P + 1), 3), (dict(C=P + 2, ctype=2), 3), (dict(bias=P + 1), 3),
    (dict(bias=P + 2, ctype=2), 3),
])
def test_gemm_a8w8_refusals(change, status):
    a = dict(G, **change)
    got = ops.lib().gemm_a8w8(a["A"], a["lda"], a["a_s"], a["B"], a["ldb"], a["b_s"], a["bias"], a["C"], a["ldc"],
                              a["ctype"], a["M"], a["N"], a["K"], None)
    assert got == status


def test_binding_refuses_host_tensors():
    x = torch.zeros(2, 32, dtype=torch.bfloat16)
    q, s = torch.zeros(2, 32, dtype=torch.int8), torch.zeros(2)
    with pytest.raises(ValueError, match="CUDA"):
        ops.int8_quant(x)
    with pytest.raises(ValueError, match="CUDA"):
        ops.int8_rmsnorm_quant(x, x[0], 1e-6)
    with pytest.raises(ValueError, match="CUDA"):
        ops.gemm_a8w8(q, s, q, s)


@pytest.mark.parametrize("tensor,dtype,shape,device,what", [
    (torch.zeros(2, 32, dtype=torch.int8), torch.uint8, (2, 32), -1, "must be torch.uint8"),
    (torch.zeros(2, 32, dtype=torch.int8), torch.int8, (2, 16), -1, "must be"),
    (torch.zeros(32, dtype=torch.int8), torch.int8, (1, 32), -1, "must be"),
    (torch.zeros(32, 2, dtype=torch.int8).t(), torch.int8, (2, 32), -1, "unit column stride"),
    (torch.zeros(2, 32, dtype=torch.int8), torch.int8, (2, 32), 0, "on device 0"),
])
def test_binding_matrix_check(tensor, dtype, shape, device, what):
    with pytest.raises(ValueError, match=what):
        ops._matrix(tensor, "t", dtype, *shape, device)


def test_binding_stride_of_a_single_row_is_its_length():
    one = torch.zeros(8, 64, dtype=torch.int8)[3:4]
    assert ops._matrix(one, "t", torch.int8, 1, 64, -1) == 64
    odd = torch.zeros(64, dtype=torch.int8).as_strided((1, 64), (1, 1))
    assert ops._matrix(odd, "t", torch.int8, 1, 64, -1) == 64


def test_binding_vector_check():
    with pytest.raises(ValueError, match="contiguous"):
        ops._vector(torch.zeros(8)[::2], "t", torch.float32, 4, -1)
    with pytest.raises(ValueError, match="length 5"):
        ops._vector(torch.zeros(4), "t", torch.float32, 5, -1)
    with pytest.raises(ValueError, match="float32"):
        ops._vector(torch.zeros(4, dtype=torch.float64), "t", torch.float32, 4, -1)


@pytest.mark.parametrize("M,N,K", [(0, 16, 64), (16, 0, 64), (16, 16, 0), (16, 16, 24), (16, 16, 131072),
                                   ((1 << 24) + 1, 16, 64), (1 << 24, 1 << 24, 64)])
def test_path_of_a_rejected_shape(M, N, K):
    assert ops.lib().gemm_a8w8_path(M, N, K) == 0
    with pytest.raises(ValueError, match="rejects"):
        ops.a8w8_path(M, N, K)


# Each path with row, column and K tails: K of fewer steps than the ring's stages and of many, tails of 16 to 112.
PATH_SHAPES = [("skinny_16x16", 17, 33, 144), ("skinny_16x16", 15, 1001, 7184), ("skinny_32x16", 17, 2050, 528),
               ("skinny_32x16", 31, 3000, 7120), ("skinny_32x32", 33, 2050, 1040), ("skinny_32x32", 17, 4100, 2096),
               ("ring_32x32", 17, 33, 16), ("ring_32x32", 33, 257, 16), ("ring_32x32", 33, 2051, 784),
               ("ring_64x32", 257, 1030, 16), ("ring_64x32", 97, 2113, 1040), ("ring_64x64", 257, 2050, 16),
               ("ring_64x64", 65, 4099, 2064), ("ring_128x64", 515, 2050, 16), ("ring_128x64", 257, 4100, 144),
               ("ring_128x64", 390, 3001, 1040), ("ring_128x128", 1030, 2050, 16), ("ring_128x128", 515, 4100, 144),
               ("ring_128x128", 1030, 2051, 1040), ("ring_128x256", 1030, 4100, 16), ("ring_128x256", 1300, 4100, 528),
               ("large_256x256", 2067, 3985, 272), ("large_256x256", 2586, 3141, 1040)]


@pytest.mark.parametrize("path,M,N,K", PATH_SHAPES)
def test_path_shapes(path, M, N, K):
    assert ops.a8w8_path(M, N, K) == path


def test_paths_follow_the_measured_order():
    """Few tokens take the small tiles, prefills the large ones, and every path is some shape's."""
    assert ops.a8w8_path(1, 4096, 7168) == "skinny_16x16"
    assert ops.a8w8_path(16, 2112, 7168) == "skinny_16x16"
    assert ops.a8w8_path(4096, 4096, 7168) == "large_256x256"
    assert ops.a8w8_path(1024, 4096, 7168) == "ring_128x128"
    seen = {ops.a8w8_path(M, N, K) for M in (1, 16, 32, 64, 128, 256, 512, 1024, 2048, 4096)
            for N in (256, 1024, 2112, 4096, 7168) for K in (512, 2048, 7168)}
    assert seen == set(ops.A8W8_PATHS.values())
    assert ops.a8w8_path(1 << 24, 1024, 131056) in ops.A8W8_PATHS.values()
