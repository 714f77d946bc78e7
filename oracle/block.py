"""Matrices of E4M3 codes with an fp32 scale for each block of 128 K-values, the
norm that feeds them and the products that read them: the CPU oracle.

TEST INFRASTRUCTURE ONLY: imported by the tests, never by the product library.

The definitions are those of include/gemm355.h (gemm355_block_quantize,
gemm355_rmsnorm, gemm355_block_gemm, gemm355_block_gated), written out in binary64
apart from the steps that the definitions round to binary32.  Scales are held as
[row blocks][K blocks] here, whichever way the library stores them.
"""
from __future__ import annotations

from typing import Optional, Tuple

import numpy as np

from . import quant, reference, w4


def decode(codes: np.ndarray) -> np.ndarray:
    c = np.ascontiguousarray(codes, dtype=np.uint8)
    return reference.decode_e4m3(c).reshape(c.shape)


def spread(scales: np.ndarray, rows: int, K: int, block_rows: int) -> np.ndarray:
    """The scale of every element."""
    s = np.asarray(scales, dtype=np.float64)
    return np.repeat(np.repeat(s, block_rows, 0)[:rows], 128, 1)[:, :K]


def values(codes: np.ndarray, scales: np.ndarray, block_rows: int) -> np.ndarray:
    return decode(codes) * spread(scales, codes.shape[0], codes.shape[1], block_rows)


def scale_of(a: np.ndarray) -> Tuple[np.ndarray, np.ndarray]:
    """Scale and its inverse for largest magnitudes a (binary32)."""
    a = np.asarray(a, dtype=np.float32)
    with np.errstate(divide="ignore"):
        none = a < np.float32(2.0 ** -100)
        s = np.where(none, np.float32(1), a / np.float32(448)).astype(np.float32)
        i = np.where(none, np.float32(1), np.float32(448) / a).astype(np.float32)
    return s, i


def quantize(x: np.ndarray, block_rows: int) -> Tuple[np.ndarray, np.ndarray]:
    """(codes, scales) of binary32 rows."""
    x = np.asarray(x, dtype=np.float32)
    rows, K = x.shape
    nr, nk = -(-rows // block_rows), -(-K // 128)
    codes, scales = np.zeros((rows, K), np.uint8), np.zeros((nr, nk), np.float32)
    for r in range(nr):
        for k in range(nk):
            part = x[r * block_rows:(r + 1) * block_rows, k * 128:(k + 1) * 128]
            s, i = scale_of(np.max(np.abs(part)))
            scales[r, k] = s
            t = np.clip((part * i).astype(np.float32), np.float32(-448), np.float32(448))
            codes[r * block_rows:(r + 1) * block_rows, k * 128:(k + 1) * 128] = quant.encode(t, "e4m3")
    return codes, scales


def norm_input(x: np.ndarray, residual: Optional[np.ndarray], kind: str) -> np.ndarray:
    """h: the binary32 sum, rounded to the residual's type."""
    if residual is None:
        return np.asarray(x, np.float32)
    h = (np.asarray(x, np.float32) + np.asarray(residual, np.float32)).astype(np.float32)
    return w4.bf16(h) if kind == "bf16" else h


def rmsnorm(h: np.ndarray, weight: Optional[np.ndarray], eps: float) -> np.ndarray:
    h = np.asarray(h, dtype=np.float64)
    y = h / np.sqrt(np.mean(h * h, 1, keepdims=True) + float(np.float32(eps)))
    return y if weight is None else y * np.asarray(weight, dtype=np.float64)


def act(g: np.ndarray, kind: str) -> np.ndarray:
    """g / (1 + exp(-z)): z = g for SiLU; (1 + tanh(z / 2)) / 2 is the same quotient,
    without the difference that far below zero loses every digit."""
    g = np.asarray(g, dtype=np.float64)
    z = g if kind == "silu" else 2 * np.sqrt(2 / np.pi) * (g + 0.044715 * g ** 3)
    e = np.exp(-np.abs(z))
    return np.where(z >= 0, g / (1 + e), g * e / (1 + e))
