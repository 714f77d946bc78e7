"""Keys and values in pages of E4M3 codes with one E8M0 scale for each page and
head: the CPU oracle of the library's append and of attention over the cache.

TEST INFRASTRUCTURE ONLY: imported by the tests, never by the product library.

The definitions are those of include/gemm355.h (gemm355_kv_cache,
gemm355_kv_append, gemm355_attention), written out token by token in binary64.
Nearest E4M3 codes come from the table search of oracle/quant.py.
"""
from __future__ import annotations

from typing import List, Optional, Tuple

import numpy as np

from . import quant, reference


def decode(codes: np.ndarray) -> np.ndarray:
    c = np.ascontiguousarray(codes, dtype=np.uint8)
    return reference.decode_e4m3(c).reshape(c.shape)


def encode(x: np.ndarray) -> np.ndarray:
    """Nearest code; infinities to the largest value, NaN to a NaN."""
    x = np.asarray(x, dtype=np.float64)
    nan = np.isnan(x)
    t = np.clip(np.where(nan, 0.0, x), -448.0, 448.0).astype(np.float32)
    return np.where(nan, 0x7F, quant.encode(t, "e4m3")).astype(np.uint8)


def block_exponent(a: float) -> int:
    """Smallest e with a <= 448 * 2^e, in [-100, 120]."""
    e = -100 if a < 1e-25 else 120 if not np.isfinite(a) else max(-100, int(np.floor(np.log2(a))) - 10)
    while e < 120 and a > np.ldexp(448.0, e):
        e += 1
    return min(e, 120)


def rotate(x: np.ndarray, pos: int, cos: np.ndarray, sin: np.ndarray, rot: int, interleaved: bool) -> np.ndarray:
    """heads x D binary64 values of one token -> binary32 values."""
    y = x.astype(np.float64).copy()
    c, s = cos[pos].astype(np.float64), sin[pos].astype(np.float64)
    for i in range(rot // 2):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
        y[:, a] = x[:, a] * c[i] - x[:, b] * s[i]
        y[:, b] = x[:, b] * c[i] + x[:, a] * s[i]
    return y.astype(np.float32)


class Step:
    """A step's indices as the kernels read them: rows, positions and lengths
    with everything out of range brought to the nearest value allowed."""

    def __init__(self, lens, q_start, tokens: int, max_new: int, max_len: int, table, page: int, pages: int):
        self.batch, self.page, self.pages, self.table = len(lens), page, pages, np.asarray(table)
        self.len = [min(max(int(n), 0), max_len) for n in lens]
        self.row: List[int] = []
        self.new: List[int] = []
        self.pos: List[int] = []          # of a sequence's first row
        for b in range(self.batch):
            if q_start is None:
                a, n = b * max_new, max_new
            else:
                a = min(max(int(q_start[b]), 0), tokens)
                n = min(max(int(q_start[b + 1]), a), tokens) - a
            self.row.append(a)
            self.new.append(min(n, max_new))
            self.pos.append(self.len[b] - n)

    def page_id(self, b: int, t: int) -> Optional[int]:
        i = int(self.table[b, t // self.page])
        return i if 0 <= i < self.pages else None


def append(step: Step, k: np.ndarray, v: np.ndarray, ks: np.ndarray, vs: np.ndarray, xk: np.ndarray, xv: np.ndarray,
           cos=None, sin=None, rot: int = 0, interleaved: bool = False) -> None:
    """Updates codes k [pages][H][page][D], v [pages][H][D][page] and scales in
    place; xk, xv: rows x H x D binary64."""
    for b in range(step.batch):
        n, p0 = step.new[b], step.pos[b]
        first = max(p0, 0)
        for base in range(first // step.page * step.page, p0 + n if n else 0, step.page):
            lo, hi = max(first, base), min(p0 + n, base + step.page)
            at = step.page_id(b, base)
            if at is None or lo >= hi:
                continue
            for name in ("k", "v"):
                x, scales = (xk, ks) if name == "k" else (xv, vs)
                rows = [x[step.row[b] + t - p0] for t in range(lo, hi)]
                if name == "k" and rot:
                    rows = [rotate(r, t, cos, sin, rot, interleaved) for r, t in zip(rows, range(lo, hi))]
                new = np.stack(rows).astype(np.float64)                       # tokens, H, D
                for h in range(new.shape[1]):
                    block = k[at, h] if name == "k" else v[at, h].T           # page, D (a view)
                    a = np.abs(new[:, h])
                    e = block_exponent(float(np.max(np.where(np.isnan(a), 0.0, a))))
                    old = int(scales[at, h]) - 127
                    if lo > base:
                        e = max(e, old)
                        if e > old:
                            block[:lo - base] = encode(np.ldexp(decode(block[:lo - base]), old - e))
                    scales[at, h] = e + 127
                    block[lo - base:hi - base] = encode(np.ldexp(new[:, h], -e))


def attention(step: Step, k: np.ndarray, v: np.ndarray, ks: np.ndarray, vs: np.ndarray, q: np.ndarray, scale: float,
              window: int = 0, sinks: int = 0) -> Tuple[np.ndarray, np.ndarray, np.ndarray, np.ndarray]:
    """q: rows x Hq x D binary64 -> (o, lse, W, S): W = sum of weights times
    |v|, S = largest sum of |scale q_d k_d| over the tokens seen (what rounding
    of the weights and of the scores scales with).  Rows that no sequence owns
    are NaN in every output."""
    rows, Hq, D = q.shape
    H = k.shape[1]
    o = np.full((rows, Hq, D), np.nan)
    W = np.full((rows, Hq, D), np.nan)
    lse = np.full((rows, Hq), np.nan)
    S = np.full((rows, Hq), np.nan)
    for b in range(step.batch):
        ids = [step.page_id(b, t) for t in range(step.len[b])]
        held = np.array([t for t, a in enumerate(ids) if a is not None], dtype=np.int64)
        pg, sl = np.array([ids[t] for t in held], dtype=np.int64), held % step.page
        kk = decode(k[pg, :, sl]) * np.ldexp(1.0, ks[pg].astype(int) - 127)[..., None]       # tokens, H, D
        vv = decode(v[pg, :, :, sl]) * np.ldexp(1.0, vs[pg].astype(int) - 127)[..., None]
        for i in range(step.new[b]):
            p, r = step.pos[b] + i, step.row[b] + i
            seen = (held <= p) & ((held > p - window) | (held < sinks) if window else True)
            for j in range(Hq):
                h = j // (Hq // H)
                if not seen.any():
                    o[r, j], W[r, j], lse[r, j], S[r, j] = 0.0, 0.0, -np.inf, 0.0
                    continue
                keys, vals = kk[seen, h], vv[seen, h]
                x = scale * (keys @ q[r, j])
                m = x.max()
                w = np.exp(x - m)
                o[r, j] = w @ vals / w.sum()
                W[r, j] = w @ np.abs(vals) / w.sum()
                lse[r, j] = m + np.log(w.sum())
                S[r, j] = float(np.max(scale * (np.abs(keys) @ np.abs(q[r, j]))))
    return o, lse, W, S
