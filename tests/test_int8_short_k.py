"""Shapes of gemm_a8w8 whose K is one or two of the kernels' 128-byte steps, shorter than their rings, per kernel."""
import pytest

from mxfp4_block_scaled_02_amd import ops

SHORT_K = [("skinny_16x16", 17, 33, 128), ("skinny_16x16", 16, 257, 256), ("skinny_32x16", 4099, 1, 384)] + [
    (path, M, 6149, K) for K in (16, 128, 144, 256)
    for path, M in [("ring_32x32", 17), ("ring_64x32", 47), ("ring_64x64", 257), ("ring_128x64", 161),
                    ("ring_128x128", 515), ("ring_128x256", 1030), ("large_256x256", 1283)]]


@pytest.mark.parametrize("path,M,N,K", SHORT_K)
def test_path_of_a_short_k(path, M, N, K):
    assert ops.a8w8_path(M, N, K) == path
