"""Matrices held in 4 bits with a scale for each group: the CPU oracle of the
library's 4-bit quantiser, of its dequantiser and of products with such matrices.

TEST INFRASTRUCTURE ONLY: imported by the tests, never by the product library.

    INT    w = (u - z) * s, u = 0 .. 15, s a bf16 value, z = 8 or a zero point
    MXFP4  w = e2m1(code) * 2^(byte - 127), the E2M1 values and block scales of
           oracle/mx.py

The quantiser's definition is in include/gemm355.h (gemm355_w4_quantize).
Differences and quotients are formed in binary64 and rounded to binary32 (a
quotient of two binary32 values rounded to binary64 first rounds to the same
binary32 value: 53 >= 2 * 24 + 2); the nearest E2M1 code is found by searching
the table of values.
"""
from __future__ import annotations

from typing import Optional, Tuple

import numpy as np

from . import mx


def bf16(x: np.ndarray) -> np.ndarray:
    """Nearest bf16 value (ties to even) of finite binary32 values."""
    b = np.asarray(x, dtype=np.float32).view(np.uint32).astype(np.uint64)
    b = (b + 0x7FFF + ((b >> 16) & 1)) & 0xFFFF0000
    return b.astype(np.uint32).view(np.float32)


def _f32(x: np.ndarray) -> np.ndarray:
    return np.asarray(x, dtype=np.float64).astype(np.float32).astype(np.float64)


def quantize(w: np.ndarray, fmt: str, group: int, zeros: bool = False) -> Tuple[np.ndarray, np.ndarray, Optional[np.ndarray]]:
    """N x K binary32 values -> (codes N x K, scales N x ng, zero points or
    None); scales are binary32 values (INT) or E8M0 bytes (MXFP4)."""
    w = np.asarray(w, dtype=np.float32).astype(np.float64)
    N, K = w.shape
    ng = -(-K // group)
    codes = np.zeros((N, K), np.uint8)
    scales = np.zeros((N, ng), np.uint8 if fmt == "mxfp4" else np.float32)
    zp = np.zeros((N, ng), np.uint8) if zeros else None
    values = mx.decode_e2m1(np.arange(8))
    for n in range(N):
        for g in range(ng):
            x = w[n, g * group:(g + 1) * group]
            sl = slice(g * group, g * group + x.size)
            if fmt == "mxfp4":
                a = float(np.max(np.abs(x)))
                e = max(int(np.floor(np.log2(a))) - 2 + 127, 0) if a > 0 else 0
                scales[n, g] = e
                t = np.abs(np.ldexp(x, 127 - e))
                d = np.abs(np.minimum(t, 6.0)[:, None] - values[None, :])
                best = d.min(axis=1)
                lo = np.argmax(d == best[:, None], axis=1)          # the lower of two at a tie
                tie = (lo < 7) & (d[np.arange(x.size), np.minimum(lo + 1, 7)] == best)
                c = np.where(tie & (lo % 2 == 1), lo + 1, lo)
                codes[n, sl] = c + 8 * np.signbit(x)
                continue
            if zeros:
                lo, hi = min(0.0, float(x.min())), max(0.0, float(x.max()))
                a, steps = float(_f32(hi - lo)), 15.0
            else:
                lo, a, steps = 0.0, float(np.max(np.abs(x))), 7.0
            s = float(bf16(np.float32(_f32(a / steps)))) if a >= 2.0 ** -100 else 1.0
            z = float(np.clip(np.rint(_f32(-lo / s)), 0, 15)) if zeros else 8.0
            codes[n, sl] = np.clip(np.rint(_f32(x / s)) + z, 0, 15).astype(np.uint8)
            scales[n, g] = s
            if zeros:
                zp[n, g] = int(z)
    return codes, scales, zp


def pack(codes: np.ndarray, ldw: int) -> np.ndarray:
    """N x K codes -> N x ldw / 2 bytes, element 2i in the low nibble."""
    c = np.zeros((codes.shape[0], ldw), np.uint8)
    c[:, :codes.shape[1]] = codes
    return (c[:, 0::2] | (c[:, 1::2] << 4)).astype(np.uint8)


def values(codes: np.ndarray, scales: np.ndarray, zeros: Optional[np.ndarray], fmt: str, group: int) -> np.ndarray:
    """N x K binary64 values that the codes stand for."""
    K = codes.shape[1]
    per_k = lambda a: np.repeat(np.asarray(a), group, axis=1)[:, :K]  # noqa: E731
    if fmt == "mxfp4":
        return mx.decode_e2m1(codes) * per_k(mx.decode_e8m0(scales))
    z = per_k(zeros).astype(np.float64) if zeros is not None else 8.0
    return (codes.astype(np.float64) - z) * per_k(scales).astype(np.float64)
