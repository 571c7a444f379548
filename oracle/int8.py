"""The 8-bit integer path -- row quantisation, residual RMS norm with
quantisation, and the scaled integer product, from their definitions.

TEST INFRASTRUCTURE ONLY (see ``oracle/__init__.py``): never called by the
product path.

Matrices of values are NumPy float32 arrays that already hold values of the
type named by ``dtype`` ("bf16", "fp16" or "fp32"). The steps that the
definition rounds to fp32 are NumPy float32 operations (each correctly rounded);
sums are exact (``math.fsum`` in float64, Python-sized integers).
"""
from __future__ import annotations

import math

import numpy as np

from .mx import bf16_bits_to_f64, f64_to_bf16_bits

MIN_SCALE = np.float32(2.0 ** -126)
ONE_127TH = np.float32(1.0) / np.float32(127.0)


def round_to(v: np.ndarray, dtype: str) -> np.ndarray:
    """Real values (float32 or float64) rounded once to `dtype`, as float32."""
    v = np.asarray(v)
    with np.errstate(over="ignore"):
        if dtype == "bf16":
            return bf16_bits_to_f64(f64_to_bf16_bits(v.astype(np.float64))).astype(np.float32)
        if dtype == "fp16":
            return v.astype(np.float16).astype(np.float32)
        return v.astype(np.float32)


def row_codes(y: np.ndarray):
    """float32 [M, K] -> (int8 codes [M, K], float32 scales [M])."""
    y = np.asarray(y, dtype=np.float32)
    M, K = y.shape
    q, s = np.zeros((M, K), dtype=np.int8), np.zeros(M, dtype=np.float32)
    for i in range(M):
        if not np.all(np.isfinite(y[i])):
            s[i] = np.nan  # and codes 0
            continue
        s[i] = max(np.float32(np.max(np.abs(y[i])) * ONE_127TH), MIN_SCALE)
        r = np.float32(1.0) / s[i]
        q[i] = np.rint(y[i] * r).astype(np.int8)
    return q, s


def rmsnorm(x: np.ndarray, w: np.ndarray, eps: float, dtype: str, residual=None):
    """(y float32 [M, K], h float32 [M, K] holding values of `dtype`)."""
    x, w = np.asarray(x, np.float32), np.asarray(w, np.float32)
    h = x
    with np.errstate(over="ignore", invalid="ignore"):
        if residual is not None:
            h = np.asarray(x + np.asarray(residual, np.float32), np.float32)
            if dtype != "fp32":
                ok = np.isfinite(h)  # the bf16 conversion takes finite values only
                h = np.where(ok, round_to(np.where(ok, h, 0), dtype), h).astype(np.float32)
        y = np.empty_like(h)
        for i in range(h.shape[0]):
            row = h[i].astype(np.float64)
            ss = math.fsum(row * row) if np.all(np.isfinite(row)) else math.inf
            inv = np.float32(1.0 / np.sqrt(np.float64(ss) / h.shape[1] + np.float64(np.float32(eps))))
            y[i] = (h[i] * inv) * w
    return y, h


def accumulate(aq: np.ndarray, bq: np.ndarray) -> np.ndarray:
    """The integer sums, in float64: every partial sum is a whole number below 2^53, so they are exact."""
    acc = aq.astype(np.float64) @ bq.astype(np.float64).T
    assert np.max(np.abs(acc), initial=0) < 2 ** 31
    return acc


def gemm(aq: np.ndarray, a_s: np.ndarray, bq: np.ndarray, b_s: np.ndarray, bias=None) -> np.ndarray:
    """The fp32 value that C rounds to its type: ((acc * a_s) * b_s) + bias, each step rounded to fp32."""
    acc = accumulate(aq, bq)
    with np.errstate(over="ignore", invalid="ignore"):
        c = acc.astype(np.float32) * a_s[:, None].astype(np.float32) * b_s[None, :].astype(np.float32)
        return c if bias is None else c + bias[None, :].astype(np.float32)


def gemm_f64(aq, a_s, bq, b_s, bias=None) -> np.ndarray:
    """The same in 64 bits, unrounded."""
    c = accumulate(aq, bq) * a_s[:, None].astype(np.float64) * b_s[None, :].astype(np.float64)
    return c if bias is None else c + bias[None, :].astype(np.float64)
