"""Thin ctypes binding of libmxfp4.so (C ABI in include/mxfp4.h).

Argument marshalling only: torch supplies device memory and the current
stream; every step of the computation runs in the library's HIP kernels. There
is no fallback: if the library is missing or a call returns a non-zero status,
these functions raise.
"""
from __future__ import annotations

import ctypes
import functools
import os
import threading

import torch

# MXFP4_LIB names another build of the same library (the sanitizer check build);
# it must exist like the default one.
_LIB_PATH = os.environ.get("MXFP4_LIB") or os.path.join(os.path.dirname(os.path.abspath(__file__)), "libmxfp4.so")
_lib = None
_lock = threading.Lock()

MXFP4_MAX_GROUPS = 32
STATUS = {0: "MXFP4_OK", 1: "MXFP4_ERR_NULL", 2: "MXFP4_ERR_SHAPE", 3: "MXFP4_ERR_ALIGN", 4: "MXFP4_ERR_WORKSPACE",
          5: "MXFP4_ERR_TOO_MANY_GROUPS", 6: "MXFP4_ERR_HIP", 7: "MXFP4_ERR_BUFFER", 8: "MXFP4_ERR_ARG"}
EXPORTED = ["mxfp4_status_str", "mxfp4_quant", "mxfp4_rmsnorm_quant", "mxfp4_pack_B_bytes", "mxfp4_pack_B",
            "gemm_a4w4_workspace_bytes", "gemm_a4w4_fused", "gemm_a4w4_fused_path", "gemm_a4w4_fused_noalloc",
            "gemm_a4w4_fused_dump_bytes",
            "gemm_a4w4_fused_dump",
            "gemm_a4w4", "grouped_gemm_a4w4_workspace_bytes", "grouped_gemm_a4w4", "grouped_gemm_a4w4_dump_bytes",
            "grouped_gemm_a4w4_dump_copies", "grouped_gemm_a4w4_dump", "grouped_gemm_a4w4_mnk", "grouped_gemm_nvfp4",
            "int8_quant", "int8_rmsnorm_quant", "gemm_a8w8", "gemm_a8w8_path", "moe_route", "moe_a16w4_workspace_bytes",
            "moe_a16w4", "lora_add_workspace_bytes", "lora_add"]


class Mxfp4Error(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {lib().mxfp4_status_str(status).decode()} (status {status})")


class GroupMnk(ctypes.Structure):
    """mirror of mxfp4_group_mnk"""
    _fields_ = [("A", ctypes.c_void_p), ("lda", ctypes.c_int64), ("strideA", ctypes.c_int64),
                ("Bp", ctypes.c_void_p), ("strideB", ctypes.c_int64), ("C", ctypes.c_void_p), ("ldc", ctypes.c_int64),
                ("strideC", ctypes.c_int64), ("M", ctypes.c_int64), ("N", ctypes.c_int64), ("K", ctypes.c_int64),
                ("L", ctypes.c_int64)]


class GroupNv(ctypes.Structure):
    """mirror of nvfp4_group"""
    _fields_ = [("Aq", ctypes.c_void_p), ("lda", ctypes.c_int64), ("strideA", ctypes.c_int64),
                ("As", ctypes.c_void_p), ("ldas", ctypes.c_int64), ("strideAs", ctypes.c_int64),
                ("Bq", ctypes.c_void_p), ("ldb", ctypes.c_int64), ("strideB", ctypes.c_int64),
                ("Bs", ctypes.c_void_p), ("ldbs", ctypes.c_int64), ("strideBs", ctypes.c_int64),
                ("C", ctypes.c_void_p), ("ldc", ctypes.c_int64), ("strideC", ctypes.c_int64),
                ("M", ctypes.c_int64), ("N", ctypes.c_int64), ("K", ctypes.c_int64), ("L", ctypes.c_int64)]


class Group(ctypes.Structure):
    """mirror of mxfp4_group"""
    _fields_ = [("A", ctypes.c_void_p), ("lda", ctypes.c_int64), ("Bp", ctypes.c_void_p), ("C", ctypes.c_void_p),
                ("ldc", ctypes.c_int64), ("M", ctypes.c_int64)]


def lib() -> ctypes.CDLL:
    """Load libmxfp4.so (once) and declare the C signatures."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(_LIB_PATH):
            raise RuntimeError(f"{_LIB_PATH} is not built; run `python -m mxfp4_block_scaled_02_amd.build`")
        L = ctypes.CDLL(_LIB_PATH)
        vp, i64, sz, i32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_size_t, ctypes.c_int
        L.mxfp4_status_str.argtypes, L.mxfp4_status_str.restype = [i32], ctypes.c_char_p
        L.mxfp4_quant.argtypes, L.mxfp4_quant.restype = [vp, i64, vp, i64, vp, i64, i64, i64, vp], i32
        L.mxfp4_rmsnorm_quant.argtypes = [vp, i64, vp, ctypes.c_float, vp, i64, vp, i64, i64, i64, vp]
        L.mxfp4_rmsnorm_quant.restype = i32
        L.mxfp4_pack_B_bytes.argtypes, L.mxfp4_pack_B_bytes.restype = [i64, i64], sz
        L.mxfp4_pack_B.argtypes, L.mxfp4_pack_B.restype = [vp, vp, i64, i64, vp, sz, vp], i32
        L.gemm_a4w4_workspace_bytes.argtypes, L.gemm_a4w4_workspace_bytes.restype = [i64, i64, i64], sz
        L.gemm_a4w4_fused.argtypes = [vp, i64, vp, vp, i64, i64, i64, i64, vp, sz, vp]
        L.gemm_a4w4_fused.restype = i32
        L.gemm_a4w4_fused_path.argtypes, L.gemm_a4w4_fused_path.restype = [i64, i64, i64], i32
        L.gemm_a4w4_fused_noalloc.argtypes = [vp, i64, vp, vp, i64, i64, i64, i64, vp]
        L.gemm_a4w4_fused_noalloc.restype = i32
        L.gemm_a4w4_fused_dump_bytes.argtypes, L.gemm_a4w4_fused_dump_bytes.restype = [i64, i64, i64], sz
        L.gemm_a4w4_fused_dump.argtypes = [vp, i64, vp, vp, i64, i64, i64, i64, vp, sz, vp, sz, vp]
        L.gemm_a4w4_fused_dump.restype = i32
        L.grouped_gemm_a4w4_dump_bytes.argtypes = [ctypes.POINTER(Group), i32, i64, i64]
        L.grouped_gemm_a4w4_dump_bytes.restype = sz
        L.grouped_gemm_a4w4_dump_copies.argtypes = [ctypes.POINTER(Group), i32, i64, i64, i32]
        L.grouped_gemm_a4w4_dump_copies.restype = i64
        L.grouped_gemm_a4w4_dump.argtypes = [ctypes.POINTER(Group), i32, i64, i64, vp, sz, vp, sz, vp]
        L.grouped_gemm_a4w4_dump.restype = i32
        L.gemm_a4w4.argtypes = [vp, i64, vp, i64, vp, vp, i64, i64, i64, i64, vp, sz, vp]
        L.gemm_a4w4.restype = i32
        L.grouped_gemm_a4w4_workspace_bytes.argtypes = [ctypes.POINTER(Group), i32, i64, i64]
        L.grouped_gemm_a4w4_workspace_bytes.restype = sz
        L.grouped_gemm_a4w4.argtypes = [ctypes.POINTER(Group), i32, i64, i64, vp, sz, vp]
        L.grouped_gemm_a4w4.restype = i32
        L.grouped_gemm_a4w4_mnk.argtypes = [ctypes.POINTER(GroupMnk), i32, vp]
        L.grouped_gemm_a4w4_mnk.restype = i32
        L.grouped_gemm_nvfp4.argtypes, L.grouped_gemm_nvfp4.restype = [ctypes.POINTER(GroupNv), i32, vp], i32
        L.int8_quant.argtypes, L.int8_quant.restype = [vp, i64, i32, vp, i64, vp, i64, i64, vp], i32
        L.int8_rmsnorm_quant.argtypes = [vp, i64, vp, i64, vp, ctypes.c_float, i32, vp, i64, vp, i64, vp, i64, i64, vp]
        L.int8_rmsnorm_quant.restype = i32
        L.gemm_a8w8.argtypes = [vp, i64, vp, vp, i64, vp, vp, vp, i64, i32, i64, i64, i64, vp]
        L.gemm_a8w8.restype = i32
        L.gemm_a8w8_path.argtypes, L.gemm_a8w8_path.restype = [i64, i64, i64], i32
        L.moe_route.argtypes = [vp, i64, i32, vp, i32, i32, ctypes.c_float, vp, vp, i64, i64, i64, vp]
        L.moe_route.restype = i32
        L.moe_a16w4_workspace_bytes.argtypes, L.moe_a16w4_workspace_bytes.restype = [i64] * 4, sz
        L.moe_a16w4.argtypes = [vp, i64, vp, vp, vp, i64, vp, i64, vp, i64, i64, i64, i64, i64, i64, vp, sz, vp]
        L.moe_a16w4.restype = i32
        L.lora_add_workspace_bytes.argtypes, L.lora_add_workspace_bytes.restype = [i64] * 4, sz
        L.lora_add.argtypes = [vp, i64, i32, vp, i64, i32, vp, vp, vp, vp, i64, i64, i64, i64, i64, vp, sz, vp]
        L.lora_add.restype = i32
        _lib = L
        return L


def _check(status: int, where: str) -> None:
    if status != 0:
        raise Mxfp4Error(status, where)


def _stream(t: torch.Tensor) -> int:
    return torch.cuda.current_stream(t.device).cuda_stream


def _require(t: torch.Tensor, dtype: torch.dtype, name: str) -> None:
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA (HIP) tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if t.dim() != 2 or t.stride(1) != 1:
        raise ValueError(f"{name} must be 2-D with unit column stride")


# Workspace per (device, stream): zeroed once at allocation, grown on demand.
# The library leaves it zeroed after every call, so it is reused without
# clearing. Calls that may overlap need distinct workspaces; calls on one stream
# never overlap, so one buffer per stream is enough. A grown buffer replaces the
# old one only after the stream's earlier work (which may still use the old
# buffer) is ordered before its release by the caching allocator.
_ws: dict = {}


def workspace(device: torch.device, nbytes: int, stream: int | None = None) -> torch.Tensor:
    dev = device.index if device.index is not None else torch.cuda.current_device()
    if stream is None:
        stream = torch.cuda.current_stream(dev).cuda_stream
    key = (dev, int(stream))
    buf = _ws.get(key)
    if nbytes > 0 and (buf is None or buf.numel() < nbytes):
        buf = torch.zeros(max(nbytes, 1 << 20), dtype=torch.uint8, device=device)
        _ws[key] = buf
    return buf


def quant(x: torch.Tensor, out=None):
    """bf16 [M, K] -> (q uint8 [M, K/2], s uint8 [M, K/32]); `out` = (q, s) reuses given buffers."""
    _require(x, torch.bfloat16, "x")
    M, K = x.shape
    if out is None:
        q = torch.empty((M, K // 2), dtype=torch.uint8, device=x.device)
        s = torch.empty((M, K // 32), dtype=torch.uint8, device=x.device)
    else:
        q, s = out
        _require(q, torch.uint8, "q")
        _require(s, torch.uint8, "s")
        if q.shape != (M, K // 2) or s.shape != (M, K // 32):
            raise ValueError("out buffers must be [M, K/2] and [M, K/32]")
    _check(lib().mxfp4_quant(x.data_ptr(), x.stride(0), q.data_ptr(), q.stride(0), s.data_ptr(), s.stride(0), M, K,
                             _stream(x)), "mxfp4_quant")
    return q, s


def rmsnorm_quant(x: torch.Tensor, w: torch.Tensor, eps: float, out=None):
    """RMSNorm of each row of bf16 x [M, K] with bf16 weight w [K], then MXFP4:
    (q uint8 [M, K/2], s uint8 [M, K/32]); `out` = (q, s) reuses given buffers."""
    _require(x, torch.bfloat16, "x")
    M, K = x.shape
    if not w.is_cuda or w.dtype != torch.bfloat16 or w.dim() != 1 or w.shape[0] != K or w.stride(0) != 1:
        raise ValueError("w must be a contiguous bf16 CUDA vector of length K")
    if out is None:
        q = torch.empty((M, K // 2), dtype=torch.uint8, device=x.device)
        s = torch.empty((M, K // 32), dtype=torch.uint8, device=x.device)
    else:
        q, s = out
        _require(q, torch.uint8, "q")
        _require(s, torch.uint8, "s")
        if q.shape != (M, K // 2) or s.shape != (M, K // 32):
            raise ValueError("out buffers must be [M, K/2] and [M, K/32]")
    _check(lib().mxfp4_rmsnorm_quant(x.data_ptr(), x.stride(0), w.data_ptr(), float(eps), q.data_ptr(), q.stride(0),
                                     s.data_ptr(), s.stride(0), M, K, _stream(x)), "mxfp4_rmsnorm_quant")
    return q, s


def pack_B_bytes(N: int, K: int) -> int:
    return int(lib().mxfp4_pack_B_bytes(N, K))


def pack_B(bq: torch.Tensor, bs: torch.Tensor) -> torch.Tensor:
    """fp4x2 [N, K/2] + E8M0 [N, K/32] (both contiguous uint8) -> packed uint8 buffer."""
    _require(bq, torch.uint8, "bq")
    _require(bs, torch.uint8, "bs")
    N, KH = bq.shape
    K = 2 * KH
    if not (bq.is_contiguous() and bs.is_contiguous()) or bs.shape != (N, K // 32):
        raise ValueError("bq [N, K/2] and bs [N, K/32] must be contiguous and agree")
    if bs.get_device() != bq.get_device():
        raise ValueError("bq and bs must be on the same device")
    out = torch.empty(pack_B_bytes(N, K), dtype=torch.uint8, device=bq.device)
    _call(lib().mxfp4_pack_B, "mxfp4_pack_B", bq.get_device(),
          (bq.data_ptr(), bs.data_ptr(), N, K, out.data_ptr(), out.numel(), _stream(bq)))
    return out


PATHS = {1: "splitk", 2: "skinny", 3: "skinny_tiles", 4: "tiled"}


def fused_path(M: int, N: int, K: int) -> str:
    """Name of the kernel gemm_a4w4_fused runs for (M, N, K) ("splitk", "skinny", "skinny_tiles", "tiled");
    raises for a shape the call rejects."""
    p = int(lib().gemm_a4w4_fused_path(M, N, K))
    if p not in PATHS:
        raise ValueError(f"gemm_a4w4_fused rejects M={M} N={N} K={K}")
    return PATHS[p]


def gemm(a: torch.Tensor, bp: torch.Tensor, N: int, out: torch.Tensor | None = None) -> torch.Tensor:
    """C[M, N] = Q(A) . B^T in one fused launch; A bf16 [M, K], bp from pack_B."""
    _require(a, torch.bfloat16, "a")
    M, K = a.shape
    if bp.numel() < pack_B_bytes(N, K):
        raise ValueError("packed B is smaller than pack_B_bytes(N, K)")
    if out is None:
        out = torch.empty((M, N), dtype=torch.bfloat16, device=a.device)
    _require(out, torch.bfloat16, "out")
    wsz = int(lib().gemm_a4w4_workspace_bytes(M, N, K))
    st = _stream(a)
    ws = workspace(a.device, wsz, st)
    _check(lib().gemm_a4w4_fused(a.data_ptr(), a.stride(0), bp.data_ptr(), out.data_ptr(), out.stride(0), M, N, K,
                                 ws.data_ptr() if wsz else None, ws.numel() if wsz else 0, st),
           "gemm_a4w4_fused")
    return out


def gemm_dump(a: torch.Tensor, bp: torch.Tensor, N: int):
    """Verification form of gemm(): returns (C, codes [copies, M, K/2], scales [copies, M, K/32]), the
    quantised A that each N-tile of the fused kernel computed on chip (uint8)."""
    _require(a, torch.bfloat16, "a")
    M, K = a.shape
    if bp.numel() < pack_B_bytes(N, K):
        raise ValueError("packed B is smaller than pack_B_bytes(N, K)")
    out = torch.empty((M, N), dtype=torch.bfloat16, device=a.device)
    wsz = int(lib().gemm_a4w4_workspace_bytes(M, N, K))
    st = _stream(a)
    ws = workspace(a.device, wsz, st)
    dsz = int(lib().gemm_a4w4_fused_dump_bytes(M, N, K))
    copies = dsz // (M * (K // 2 + K // 32))
    dump = torch.full((dsz,), 0xEE, dtype=torch.uint8, device=a.device)
    _check(lib().gemm_a4w4_fused_dump(a.data_ptr(), a.stride(0), bp.data_ptr(), out.data_ptr(), out.stride(0), M, N, K,
                                      ws.data_ptr() if wsz else None, ws.numel() if wsz else 0, dump.data_ptr(), dsz,
                                      st), "gemm_a4w4_fused_dump")
    nq = copies * M * (K // 2)
    return out, dump[:nq].view(copies, M, K // 2), dump[nq:].view(copies, M, K // 32)


def gemm_a4w4(aq: torch.Tensor, a_scale: torch.Tensor, bp: torch.Tensor, N: int,
              out: torch.Tensor | None = None) -> torch.Tensor:
    """C[M, N] = A_q . B^T with A already quantised: aq fp4x2 [M, K/2], a_scale E8M0 [M, K/32] (uint8,
    for example from quant()); bp from pack_B. The unfused comparator of gemm()."""
    _require(aq, torch.uint8, "aq")
    _require(a_scale, torch.uint8, "a_scale")
    M, KH = aq.shape
    K = 2 * KH
    if a_scale.shape[0] != M or a_scale.shape[1] < K // 32:
        raise ValueError("a_scale must be [M, >= K/32]")
    if bp.numel() < pack_B_bytes(N, K):
        raise ValueError("packed B is smaller than pack_B_bytes(N, K)")
    if out is None:
        out = torch.empty((M, N), dtype=torch.bfloat16, device=aq.device)
    _require(out, torch.bfloat16, "out")
    wsz = int(lib().gemm_a4w4_workspace_bytes(M, N, K))
    st = _stream(aq)
    ws = workspace(aq.device, wsz, st)
    _check(lib().gemm_a4w4(aq.data_ptr(), aq.stride(0), a_scale.data_ptr(), a_scale.stride(0), bp.data_ptr(),
                           out.data_ptr(), out.stride(0), M, N, K, ws.data_ptr() if wsz else None,
                           ws.numel() if wsz else 0, st), "gemm_a4w4")
    return out


def grouped_gemm(a_list, bp_list, N: int, out_list=None):
    """One launch over all groups: C_g = Q(A_g) . B_g^T for shared N, K."""
    G = len(a_list)
    if G != len(bp_list):
        raise ValueError("a_list and bp_list differ in length")
    if G < 1 or G > MXFP4_MAX_GROUPS:
        raise ValueError(f"G must be in [1, {MXFP4_MAX_GROUPS}]")
    K = a_list[0].shape[1]
    if out_list is None:
        out_list = [torch.empty((a.shape[0], N), dtype=torch.bfloat16, device=a.device) for a in a_list]
    arr = (Group * G)()
    for g, (a, bp, c) in enumerate(zip(a_list, bp_list, out_list)):
        _require(a, torch.bfloat16, "a_g")
        _require(c, torch.bfloat16, "c_g")
        if a.shape[1] != K:
            raise ValueError("all groups share K")
        arr[g] = Group(a.data_ptr(), a.stride(0), bp.data_ptr(), c.data_ptr(), c.stride(0), a.shape[0])
    wsz = int(lib().grouped_gemm_a4w4_workspace_bytes(arr, G, N, K))
    st = _stream(a_list[0])
    ws = workspace(a_list[0].device, wsz, st)
    _check(lib().grouped_gemm_a4w4(arr, G, N, K, ws.data_ptr() if wsz else None, ws.numel() if wsz else 0, st),
           "grouped_gemm_a4w4")
    return out_list


def grouped_gemm_dump(a_list, bp_list, N: int):
    """Verification form of grouped_gemm(): returns (list of C, list of (codes [copies, M_g, K/2],
    scales [copies, M_g, K/32])), the quantised A each N-tile computed on chip per group."""
    G = len(a_list)
    K = a_list[0].shape[1]
    outs = [torch.empty((a.shape[0], N), dtype=torch.bfloat16, device=a.device) for a in a_list]
    arr = (Group * G)()
    for g, (a, bp, c) in enumerate(zip(a_list, bp_list, outs)):
        _require(a, torch.bfloat16, "a_g")
        arr[g] = Group(a.data_ptr(), a.stride(0), bp.data_ptr(), c.data_ptr(), c.stride(0), a.shape[0])
    dsz = int(lib().grouped_gemm_a4w4_dump_bytes(arr, G, N, K))
    dump = torch.full((dsz,), 0xEE, dtype=torch.uint8, device=a_list[0].device)
    _check(lib().grouped_gemm_a4w4_dump(arr, G, N, K, None, 0, dump.data_ptr(), dsz, _stream(a_list[0])),
           "grouped_gemm_a4w4_dump")
    at, res = 0, []
    for g, a in enumerate(a_list):
        M = a.shape[0]
        copies = int(lib().grouped_gemm_a4w4_dump_copies(arr, G, N, K, g))
        nq, ns = copies * M * (K // 2), copies * M * (K // 32)
        res.append((dump[at:at + nq].view(copies, M, K // 2), dump[at + nq:at + nq + ns].view(copies, M, K // 32)))
        at += nq + ns
    return outs, res


def grouped_gemm_mnk(problems, out_list=None):
    """Groups with their own (M, N, K) and a batch count, in one launch.

    problems: list of (A, Bp, N) with A bf16 [L, M, K] (or [M, K] for L = 1) and
    Bp uint8 [L, pack_B_bytes(N, K)] (or 1-D for L = 1), each batch row-major.
    Returns (or fills `out_list` with) bf16 C tensors [L, M, N] ([M, N] for L = 1).
    """
    descs, outs = [], []
    for gi, (A, Bp, N) in enumerate(problems):
        batched = A.dim() == 3
        A3 = A if batched else A.unsqueeze(0)
        B2 = Bp if Bp.dim() == 2 else Bp.unsqueeze(0)
        L, M, K = A3.shape
        if not A3.is_cuda or A3.dtype != torch.bfloat16 or A3.stride(2) != 1:
            raise ValueError("A must be a bf16 CUDA tensor with unit stride along K")
        if B2.dtype != torch.uint8 or B2.shape[0] != L or B2.shape[1] < pack_B_bytes(N, K) or B2.stride(1) != 1:
            raise ValueError("Bp must be uint8 [L, pack_B_bytes(N, K)]")
        if out_list is None:
            C3 = torch.empty((L, M, N), dtype=torch.bfloat16, device=A.device)
        else:
            C = out_list[gi]
            C3 = C if C.dim() == 3 else C.unsqueeze(0)
            if C3.shape != (L, M, N) or C3.dtype != torch.bfloat16 or C3.stride(2) != 1:
                raise ValueError("out_list[i] must be bf16 [L, M, N]")
        descs.append(GroupMnk(A3.data_ptr(), A3.stride(1), A3.stride(0), B2.data_ptr(), B2.stride(0),
                              C3.data_ptr(), C3.stride(1), C3.stride(0), M, N, K, L))
        outs.append(C3 if batched else C3[0])
    arr = (GroupMnk * len(descs))(*descs)
    _check(lib().grouped_gemm_a4w4_mnk(arr, len(descs), _stream(problems[0][0])), "grouped_gemm_a4w4_mnk")
    return outs if out_list is None else out_list


def grouped_gemm_nvfp4(problems, out_list=None):
    """NVFP4 groups with their own (M, N, K) and a batch count, in one launch.

    problems: list of (aq, a_scale, bq, b_scale): uint8 tensors aq [L, M, K/2]
    (E2M1 codes, low nibble first), a_scale [L, M, K/16] (E4M3), bq [L, N, K/2],
    b_scale [L, N, K/16]; 2-D for L = 1. Rows may be padded (unit stride along
    K). Returns (or fills `out_list` with) float16 C tensors [L, M, N] ([M, N]
    for L = 1).
    """
    def as3(t, name):
        t3 = t if t.dim() == 3 else t.unsqueeze(0)
        if not t3.is_cuda or t3.dtype != torch.uint8 or t3.stride(2) != 1:
            raise ValueError(f"{name} must be a uint8 CUDA tensor with unit stride along K")
        return t3

    descs, outs = [], []
    for gi, (aq, a_s, bq, b_s) in enumerate(problems):
        batched = aq.dim() == 3
        A, As, B, Bs = as3(aq, "aq"), as3(a_s, "a_scale"), as3(bq, "bq"), as3(b_s, "b_scale")
        L, M, KH = A.shape
        N, K = B.shape[1], 2 * KH
        if B.shape != (L, N, KH) or As.shape != (L, M, K // 16) or Bs.shape != (L, N, K // 16):
            raise ValueError("aq [L, M, K/2], a_scale [L, M, K/16], bq [L, N, K/2], b_scale [L, N, K/16] must agree")
        if out_list is None:
            C3 = torch.empty((L, M, N), dtype=torch.float16, device=aq.device)
        else:
            C = out_list[gi]
            C3 = C if C.dim() == 3 else C.unsqueeze(0)
            if C3.shape != (L, M, N) or C3.dtype != torch.float16 or C3.stride(2) != 1:
                raise ValueError("out_list[i] must be float16 [L, M, N]")
        descs.append(GroupNv(A.data_ptr(), A.stride(1), A.stride(0), As.data_ptr(), As.stride(1), As.stride(0),
                             B.data_ptr(), B.stride(1), B.stride(0), Bs.data_ptr(), Bs.stride(1), Bs.stride(0),
                             C3.data_ptr(), C3.stride(1), C3.stride(0), M, N, K, L))
        outs.append(C3 if batched else C3[0])
    arr = (GroupNv * len(descs))(*descs)
    _check(lib().grouped_gemm_nvfp4(arr, len(descs), _stream(problems[0][0])), "grouped_gemm_nvfp4")
    return outs if out_list is None else out_list


# The 8-bit integer path. MXFP4_TYPE_* of include/mxfp4.h by torch type.
TYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}


A8W8_PATHS = dict(enumerate(["skinny_16x16", "skinny_32x16", "skinny_32x32", "ring_32x32", "ring_64x32", "ring_64x64",
                             "ring_128x64", "ring_128x128", "ring_128x256", "large_256x256"], 1))

# These calls are short (the kernels of a decode step take a few microseconds, a launch 2.8), so the host's part is
# kept short too: the raw handle of the current stream spares building a Stream, and one chain of tests passes the
# ordinary call (everything contiguous); what fails it goes through the checks below, which either say what is wrong
# or find the strides.
# (Both names are absent from a torch built without devices, where every tensor is refused before their use.)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_current_device = getattr(torch._C, "_cuda_getDevice", None)
_I8, _F32 = torch.int8, torch.float32


def _matrix(t: torch.Tensor, name: str, dtype: torch.dtype, rows: int, cols: int, device: int) -> int:
    """Checks a [rows, cols] argument with unit column stride and returns its row stride (of one row: its length)."""
    if t.dtype is not dtype or t.get_device() != device or t.shape != (rows, cols):
        raise ValueError(f"{name} must be {dtype} [{rows}, {cols}] on device {device}, "
                         f"got {t.dtype} {list(t.shape)} on {t.device}")
    row, col = t.stride()
    if col != 1 and cols > 1:
        raise ValueError(f"{name} must have unit column stride")
    return row if rows > 1 else cols


def _vector(t: torch.Tensor, name: str, dtype: torch.dtype, n: int, device: int) -> None:
    """Checks a contiguous [n] argument."""
    if t.dtype is not dtype or t.get_device() != device or t.shape != (n,) or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} vector of length {n} on device {device}")


def _typed(x: torch.Tensor, name: str):
    """(MXFP4_TYPE_*, device index, rows, columns) of a 2-D device tensor."""
    dev, dt = x.get_device(), TYPES.get(x.dtype)
    if dev < 0:
        raise ValueError(f"{name} must be a CUDA (HIP) tensor")
    if x.dim() != 2:
        raise ValueError(f"{name} must be 2-D")
    if dt is None:
        raise ValueError(f"{name} must be bfloat16, float16 or float32, got {x.dtype}")
    M, K = x.shape
    return dt, dev, M, K


def _codes(x: torch.Tensor, M: int, K: int, dev: int, out):
    """The (q, s) outputs of a quantising call on x, and q's row stride."""
    if out is None:
        device = x.device
        return torch.empty(M, K, dtype=_I8, device=device), torch.empty(M, dtype=_F32, device=device), K
    q, s = out
    ldq = _matrix(q, "q", _I8, M, K, dev)
    _vector(s, "s", _F32, M, dev)
    return q, s, ldq


def _call(fn, where: str, dev: int, args) -> None:
    """fn(*args) with device `dev` current, whatever device is."""
    if dev == _current_device():
        status = fn(*args)
    else:
        with torch.cuda.device(dev):
            status = fn(*args)
    if status:
        raise Mxfp4Error(status, where)


def int8_quant(x: torch.Tensor, out=None):
    """bf16, fp16 or fp32 [M, K] -> (q int8 [M, K], s float32 [M]), x ~ q * s[:, None]: activations by token,
    or a weight [N, K] by output channel. `out` = (q, s) reuses given buffers."""
    dt, dev, M, K = _typed(x, "x")
    ldx = K if x.is_contiguous() else _matrix(x, "x", x.dtype, M, K, dev)
    q, s, ldq = _codes(x, M, K, dev, out)
    _call((_lib or lib()).int8_quant, "int8_quant", dev,
          (x.data_ptr(), ldx, dt, q.data_ptr(), ldq, s.data_ptr(), M, K, _raw_stream(dev)))
    return q, s


def int8_rmsnorm_quant(x: torch.Tensor, w: torch.Tensor, eps: float, residual: torch.Tensor | None = None, out=None):
    """RMSNorm of each row of x [M, K] (bf16, fp16 or fp32) with weight w [K] of the same type, then int8 codes:
    (q int8 [M, K], s float32 [M]). With a residual [M, K] of the same type the norm is of h = x + residual, and
    (q, s, h) is returned. `out` = (q, s) or (q, s, h) reuses given buffers; h may be x or residual itself."""
    dt, dev, M, K = _typed(x, "x")
    T = x.dtype
    ldx = K if x.is_contiguous() else _matrix(x, "x", T, M, K, dev)
    if not (w.dtype is T and w.get_device() == dev and w.shape == (K,) and w.is_contiguous()):
        _vector(w, "w", T, K, dev)
    h, rp, ldr, hp, ldh = None, None, 0, None, 0
    if residual is None:
        q, s, ldq = _codes(x, M, K, dev, out)
    else:
        if (residual.dtype is T and residual.get_device() == dev and residual.shape == (M, K)
                and residual.is_contiguous()):
            ldr = K
        else:
            ldr = _matrix(residual, "residual", T, M, K, dev)
        rp = residual.data_ptr()
        if out is None:
            h = torch.empty(M, K, dtype=T, device=x.device)
            q, s, ldq = _codes(x, M, K, dev, None)
            ldh = K
        else:
            q, s, h = out
            _, _, ldq = _codes(x, M, K, dev, (q, s))
            ldh = _matrix(h, "h", T, M, K, dev)
        hp = h.data_ptr()
    _call((_lib or lib()).int8_rmsnorm_quant, "int8_rmsnorm_quant", dev,
          (x.data_ptr(), ldx, rp, ldr, w.data_ptr(), float(eps), dt, hp, ldh, q.data_ptr(), ldq, s.data_ptr(), M, K,
           _raw_stream(dev)))
    return (q, s) if residual is None else (q, s, h)


def gemm_a8w8(aq: torch.Tensor, a_scale: torch.Tensor, bq: torch.Tensor, b_scale: torch.Tensor,
              bias: torch.Tensor | None = None, out_dtype: torch.dtype = torch.bfloat16,
              out: torch.Tensor | None = None) -> torch.Tensor:
    """C[M, N] = (aq . bq^T) * a_scale[:, None] * b_scale[None, :] (+ bias): aq int8 [M, K] with a float32 scale per
    token, bq int8 [N, K] with one per output channel (both from int8_quant, for example), bias [N] of the type of C.
    C has `out_dtype` (bf16, fp16 or fp32), or is `out` with its own type."""
    dev = aq.get_device()
    if dev < 0 or aq.dim() != 2 or bq.dim() != 2:
        raise ValueError("aq and bq must be 2-D CUDA (HIP) tensors")
    M, K = aq.shape
    N, lda, ldb = bq.shape[0], K, K
    if not (aq.dtype is _I8 and bq.dtype is _I8 and a_scale.dtype is _F32 and b_scale.dtype is _F32
            and aq.is_contiguous() and bq.is_contiguous() and a_scale.is_contiguous() and b_scale.is_contiguous()
            and bq.get_device() == dev and a_scale.get_device() == dev and b_scale.get_device() == dev
            and bq.shape[1] == K and a_scale.shape == (M,) and b_scale.shape == (N,)):
        lda = _matrix(aq, "aq", _I8, M, K, dev)
        ldb = _matrix(bq, "bq", _I8, N, K, dev)
        _vector(a_scale, "a_scale", _F32, M, dev)
        _vector(b_scale, "b_scale", _F32, N, dev)
    if out is None:
        ct = TYPES.get(out_dtype)
        if ct is None:
            raise ValueError(f"out_dtype must be bfloat16, float16 or float32, got {out_dtype}")
        out, ldc = torch.empty(M, N, dtype=out_dtype, device=aq.device), N
    else:
        ct = _typed(out, "out")[0]
        ldc = _matrix(out, "out", out.dtype, M, N, dev)
    cp = None
    if bias is not None:
        _vector(bias, "bias", out.dtype, N, dev)
        cp = bias.data_ptr()
    _call((_lib or lib()).gemm_a8w8, "gemm_a8w8", dev,
          (aq.data_ptr(), lda, a_scale.data_ptr(), bq.data_ptr(), ldb, b_scale.data_ptr(), cp, out.data_ptr(), ldc, ct,
           M, N, K, _raw_stream(dev)))
    return out


def a8w8_path(M: int, N: int, K: int) -> str:
    """Name of the kernel gemm_a8w8 runs for (M, N, K), rows x columns of C per workgroup; raises for a shape the
    call rejects."""
    p = int(lib().gemm_a8w8_path(M, N, K))
    if p not in A8W8_PATHS:
        raise ValueError(f"gemm_a8w8 rejects M={M} N={N} K={K}")
    return A8W8_PATHS[p]


# Products whose weight is picked row by row. Their scratch is allocated for each call (its contents do not matter): a
# captured graph then holds its own, and graphs that are replayed at the same time do not meet in it.
SCORES = {"softmax": 0, "sigmoid": 1}
_I32, _U8, _BF16 = torch.int32, torch.uint8, torch.bfloat16


# The library's size queries are pure functions of a few integers.
@functools.lru_cache(maxsize=256)
def _expert_bytes(I: int, H: int) -> tuple:
    """Packed bytes of an expert's gate and up rows and of its down rows, and of those with the next I that takes more,
    which a row of bytes stays below: I is not stored with the weights, and a wrong one would find others in their places."""
    size = lib().mxfp4_pack_B_bytes
    return int(size(2 * I, H)), int(size(H, I)), int(size(2 * I + 64, H)), int(size(H, I + 64))


@functools.lru_cache(maxsize=256)
def _moe_scratch(T: int, k: int, H: int, I: int) -> int:
    return int(lib().moe_a16w4_workspace_bytes(T, k, H, I))


@functools.lru_cache(maxsize=256)
def _lora_scratch(T: int, K: int, R: int, n: int) -> int:
    return int(lib().lora_add_workspace_bytes(T, K, R, n))


def _dense(t: torch.Tensor, name: str, dtype: torch.dtype, shape: tuple, device: int) -> None:
    """Checks a contiguous argument of a given shape."""
    if t.dtype is not dtype or t.get_device() != device or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous {dtype} {list(shape)} on device {device}, "
                         f"got {t.dtype} {list(t.shape)} on {t.device}")


def moe_route(logits: torch.Tensor, k: int, bias: torch.Tensor | None = None, score: str = "softmax",
              renormalize: bool = True, scale: float = 1.0, out=None):
    """The k experts of each token and their weights from a router's logits [T, E] (bf16, fp16 or fp32):
    (weights float32 [T, k], ids int32 [T, k]), by falling rank, ties to the lower index, -1 and 0 where nothing is left
    to choose (logits of -inf). The rank is the logit, or score + bias with a float32 bias [E]; the weights are
    scale * score, over their sum if `renormalize`. `out` = (weights, ids) reuses given buffers."""
    dt, dev, T, E = _typed(logits, "logits")
    if score not in SCORES:
        raise ValueError(f"score must be one of {list(SCORES)}, got {score!r}")
    ldl = E if logits.is_contiguous() else _matrix(logits, "logits", logits.dtype, T, E, dev)
    bp = None
    if bias is not None:
        _vector(bias, "bias", _F32, E, dev)
        bp = bias.data_ptr()
    if out is None:
        if k < 1:
            raise ValueError(f"k must be at least 1, got {k}")
        device = logits.device
        weights, ids = torch.empty(T, k, dtype=_F32, device=device), torch.empty(T, k, dtype=_I32, device=device)
    else:
        weights, ids = out
        _dense(weights, "weights", _F32, (T, k), dev)
        _dense(ids, "ids", _I32, (T, k), dev)
    _call((_lib or lib()).moe_route, "moe_route", dev,
          (logits.data_ptr(), ldl, dt, bp, SCORES[score], bool(renormalize), float(scale), weights.data_ptr(),
           ids.data_ptr(), T, E, k, _raw_stream(dev)))
    return weights, ids


def pack_experts(bq: torch.Tensor, bs: torch.Tensor) -> torch.Tensor:
    """pack_B of each expert's weight: fp4x2 [E, N, K/2] and E8M0 [E, N, K/32] (contiguous uint8) -> packed uint8
    [E, pack_B_bytes(N, K)]. Row e is expert e's packed B, for moe_a16w4 and for the grouped calls alike."""
    if bq.dim() != 3 or bs.dim() != 3 or bq.shape[0] != bs.shape[0] or bq.shape[0] < 1:
        raise ValueError("bq must be [E, N, K/2] and bs [E, N, K/32], E at least 1")
    return torch.stack([pack_B(q, s) for q, s in zip(bq, bs)])


def _experts(p: torch.Tensor, name: str, need: int, N: int, K: int, dev: int, below: int | None = None):
    """(number of experts, bytes from one to the next) of packed expert weights; `below`: see _expert_bytes."""
    if (p.dtype is not _U8 or p.get_device() != dev or p.dim() != 2 or need == 0 or p.shape[1] < need
            or p.stride(1) != 1 or (below is not None and p.shape[1] >= below)):
        raise ValueError(f"{name} must be uint8 [E, {need}] (pack_experts of {N} x {K}) on device {dev}, "
                         f"got {p.dtype} {list(p.shape)} on {p.device}")
    return p.shape[0], p.stride(0) if p.shape[0] > 1 else p.shape[1]


def moe_a16w4(x: torch.Tensor, ids: torch.Tensor, weights: torch.Tensor, w13: torch.Tensor, w2: torch.Tensor, I: int,
              out: torch.Tensor | None = None) -> torch.Tensor:
    """The experts' gated MLP for a few tokens: y[t] = sum_j weights[t, j] * W2_e (silu(G_e x[t]) * (U_e x[t])) with
    e = ids[t, j]; ids outside [0, E) are left out. x bf16 [T, H], ids int32 and weights float32 [T, k] (from moe_route,
    for example), w13 and w2 from pack_experts: [E] weights of 2I x H (gate rows G, then up rows U) and of H x I; a row of
    bytes may be longer than its weight by less than the next I would take (of longer ones, pass the columns in front).
    Returns bf16 [T, H], or `out`."""
    dev = x.get_device()
    if dev < 0 or x.dim() != 2:
        raise ValueError("x must be a 2-D CUDA (HIP) tensor")
    T, H = x.shape
    if ids.dim() != 2:
        raise ValueError("ids must be [T, k]")
    k, ldx = ids.shape[1], H
    need13, need2, below13, below2 = _expert_bytes(I, H)
    if (x.dtype is _BF16 and ids.dtype is _I32 and weights.dtype is _F32 and w13.dtype is _U8 and w2.dtype is _U8
            and x.is_contiguous() and ids.is_contiguous() and weights.is_contiguous() and w13.is_contiguous()
            and w2.is_contiguous() and ids.get_device() == dev and weights.get_device() == dev
            and w13.get_device() == dev and w2.get_device() == dev and ids.shape[0] == T and weights.shape == ids.shape
            and need13 and w13.dim() == 2 and w2.dim() == 2 and need13 <= w13.shape[1] < below13
            and need2 <= w2.shape[1] < below2):
        (E, stride13), (E2, stride2) = w13.shape, w2.shape
    else:
        ldx = _matrix(x, "x", _BF16, T, H, dev)
        _dense(ids, "ids", _I32, (T, k), dev)
        _dense(weights, "weights", _F32, (T, k), dev)
        E, stride13 = _experts(w13, "w13", need13, 2 * I, H, dev, below13)
        E2, stride2 = _experts(w2, "w2", need2, H, I, dev, below2)
    if E != E2:
        raise ValueError(f"w13 has {E} experts and w2 {E2}")
    device = x.device
    if out is None:
        out, ldy = torch.empty(T, H, dtype=_BF16, device=device), H
    else:
        ldy = _matrix(out, "out", _BF16, T, H, dev)
    nbytes = _moe_scratch(T, k, H, I)
    ws = torch.empty(nbytes, dtype=_U8, device=device)
    _call((_lib or lib()).moe_a16w4, "moe_a16w4", dev,
          (x.data_ptr(), ldx, ids.data_ptr(), weights.data_ptr(), w13.data_ptr(), stride13, w2.data_ptr(), stride2,
           out.data_ptr(), ldy, T, k, E, H, I, ws.data_ptr(), nbytes, _raw_stream(dev)))
    return out


def lora_add(y: torch.Tensor, x: torch.Tensor, a: torch.Tensor, b: torch.Tensor, index: torch.Tensor,
             scale: torch.Tensor | None = None) -> torch.Tensor:
    """Low-rank adapters of many requests, added in place to a shared projection's product y [T, N]:
    y[t] += scale[i] * (x[t] . a[i]^T) . b[i]^T with i = index[t]; rows whose index is outside [0, n) stay as they are.
    x [T, K], a [n, R, K] and b [n, N, R] bf16 or fp16, y of that type or float32, index int32 [T], scale float32 [n].
    Returns y."""
    yt, dev, T, N = _typed(y, "y")
    if x.dim() != 2 or a.dim() != 3:
        raise ValueError("x must be [T, K] and a [n, R, K]")
    D, K = x.dtype, x.shape[1]
    n, R, ldx, ldy = a.shape[0], a.shape[1], K, N
    if not (y.is_contiguous() and x.is_contiguous() and a.is_contiguous() and b.is_contiguous()
            and index.is_contiguous() and a.dtype is D and b.dtype is D and index.dtype is _I32
            and x.get_device() == dev and a.get_device() == dev and b.get_device() == dev and index.get_device() == dev
            and x.shape[0] == T and a.shape[2] == K and b.shape == (n, N, R) and index.shape == (T,)):
        ldy = _matrix(y, "y", y.dtype, T, N, dev)
        ldx = _matrix(x, "x", D, T, K, dev)
        _dense(a, "a", D, (n, R, K), dev)
        _dense(b, "b", D, (n, N, R), dev)
        _vector(index, "index", _I32, T, dev)
    sp = None
    if scale is not None:
        _vector(scale, "scale", _F32, n, dev)
        sp = scale.data_ptr()
    nbytes = _lora_scratch(T, K, R, n)
    ws = torch.empty(nbytes, dtype=_U8, device=y.device)
    _call((_lib or lib()).lora_add, "lora_add", dev,
          (y.data_ptr(), ldy, yt, x.data_ptr(), ldx, TYPES.get(D, -1), a.data_ptr(), b.data_ptr(), index.data_ptr(), sp,
           T, N, K, R, n, ws.data_ptr(), nbytes, _raw_stream(dev)))
    return y
