"""Adapters at the sizes that prompts and long rows bring: every form of the launches beside a plain form in 64 bits."""
import ctypes

import pytest
import torch

from mxfp4_block_scaled_02_amd import ops
from tests.test_gpu_lora import TYPES, case, check

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("T", [1023, 1024, 1025, 2047, 2048, 2049])
@pytest.mark.parametrize("n", [1, 6, 700])
def test_rows_at_the_plan_s_borders(T, n):
    c = case(T + n, T, 72, 70, 16, n, BF, F32)
    check(c)
    c["index"][:] = torch.arange(T, device="cuda") * (n + 1) // T - 1   # spans, the first without an adapter
    check(c)


@pytest.mark.parametrize("dtype,out", TYPES)
@pytest.mark.parametrize("T,K,N,R,n", [
    (2000, 4096, 2570, 64, 8), (2000, 4096, 2570, 128, 8),      # whole units of several tiles, long slices of K
    (2000, 4096, 640, 24, 400), (4096, 4096, 200, 64, 700), (4096, 4096, 200, 128, 700),  # units of a few rows
    (16, 4096, 330, 128, 5), (64, 4096, 200, 128, 64),          # many splits, a row's ranks over a wave
    (64, 7168, 200, 64, 2), (64, 7168, 200, 128, 1), (40, 7168, 130, 24, 2),  # units of more than 16 rows, up to 64 in all
    (300, 4096, 2570, 40, 3), (300, 1032, 25 * 256, 128, 16), (300, 1032, 25 * 256, 64, 16),
])
def test_long_rows_and_wide_adapters(T, K, N, R, n, dtype, out):
    check(case(T + K + N + R, T, K, N, R, n, dtype, out))


def test_a_prompt():
    """Rows of a few requests: long slices of K, whole units, splits that one thread adds up."""
    c = case(1, 4096, 7168, 1000, 64, 8, BF, BF)
    c["index"][:] = torch.arange(4096, device="cuda") * 9 // 4096 - 1
    check(c)


@pytest.mark.parametrize("N", [5 * 256, 6 * 256 - 3])
@pytest.mark.parametrize("dtype,out", TYPES)
def test_more_rows_than_a_block_a_tile_or_a_unit_at_a_time(N, dtype, out):
    check(case(N, 9000, 40, N, 24, 8, dtype, out))


class _Params(ctypes.Structure):
    """hipKernelNodeParams of hip_runtime_api.h."""
    _fields_ = [("block", ctypes.c_uint32 * 3), ("extra", ctypes.c_void_p), ("func", ctypes.c_void_p),
                ("grid", ctypes.c_uint32 * 3), ("args", ctypes.c_void_p), ("shared", ctypes.c_uint32)]


def grids(graph):
    """The grids of a captured graph's kernels."""
    with open("/proc/self/maps") as f:
        hip = ctypes.CDLL(next(p.split()[-1] for p in f if "libamdhip64.so" in p))
    g, n = ctypes.c_void_p(graph.raw_cuda_graph()), ctypes.c_size_t(0)
    assert hip.hipGraphGetNodes(g, None, ctypes.byref(n)) == 0
    nodes = (ctypes.c_void_p * n.value)()
    assert hip.hipGraphGetNodes(g, nodes, ctypes.byref(n)) == 0
    out = []
    for node in nodes:
        p = _Params()
        assert hip.hipGraphKernelNodeGetParams(ctypes.c_void_p(node), ctypes.byref(p)) == 0
        out.append(tuple(p.grid))
    return out


@pytest.mark.parametrize("T,N,z", [(4096, 512, 4), (5000, 512, 4), (8192, 512, 4), (8193, 512, 1), (9000, 513, 1), (20000, 256, 4),
                                   (20481, 256, 1), (4096, 1536, 1), (4096, 1280, 4)])
def test_whole_units_are_taken_once_all_blocks_of_rows_fill_the_chip(T, N, z):
    """z workgroups of expand to a unit; 72 units to a block of 4096 rows."""
    c = case(T, T, 8, N, 8, 8, BF, BF)
    check(c)
    graph = torch.cuda.CUDAGraph(keep_graph=True)
    with torch.cuda.graph(graph):
        ops.lora_add(**c)
    blocks = -(-T // 4096)
    assert grids(graph)[-1] == (-(-N // 256), blocks, 72 * z)
