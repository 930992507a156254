"""Oracle of the microscaled 4-bit Q-pass copy (summary page, Main Findings: a separate low-bit copy
read by the Q pass; the pages give no quantiser).  This build's reading, plain numpy:

  * a block is 32 columns of one row; e = the largest exponent field among its in-window weights, the
    row's window bottom for a block that has none; scale 2^(e - 129);
  * an in-window weight becomes the E2M1 code of the value nearest to weight / scale, ties to the even
    code, magnitudes above 6 to 6; the code's sign bit is the weight's;
  * an escaped slot holds code 0 and stays exact;
  * the scale is stored as the byte e - base + 110.
"""
from __future__ import annotations

from dataclasses import dataclass

import numpy as np

from .w12 import TILE_COLS, TILE_ROWS, W12Record, bf16_to_f64, decode, escaped_mask, padded_rows

MX4_BLOCK = 32
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


@dataclass
class Mx4Copy:
    n: int
    k: int
    code: np.ndarray      # uint8 [n, k], 0..15 (bit 3 the sign)
    scale: np.ndarray     # uint8 [n, k / 32], stored scale bytes


def e2m1_code(mag: float) -> int:
    """The code nearest to a magnitude, ties to the even code (by exhaustive search)."""
    best = 0
    for c in range(1, 8):
        d, b = abs(E2M1[c] - mag), abs(E2M1[best] - mag)
        if d < b or (d == b and c % 2 == 0):
            best = c
    return best


def mx4_copy(rec: W12Record) -> Mx4Copy:
    w = decode(rec)
    n, k = w.shape
    esc = escaped_mask(rec)
    e = ((w >> 7) & 0xFF).astype(np.int64)
    e_in = np.where(esc, 0, e).reshape(n, k // MX4_BLOCK, MX4_BLOCK)
    base = rec.base.astype(np.int64)[:, None]
    big = np.maximum(e_in.max(axis=2), base)
    scale = np.repeat(np.ldexp(1.0, big - 129), MX4_BLOCK, axis=1)
    with np.errstate(invalid="ignore", over="ignore"):
        mag = np.where(esc, 0.0, np.abs(bf16_to_f64(w)) / scale)
    values = np.unique(mag)
    codes = np.array([e2m1_code(v) for v in values], dtype=np.uint8)
    code = codes[np.searchsorted(values, mag)]
    code |= ((w >> 15) << 3).astype(np.uint8)
    code[esc] = 0
    return Mx4Copy(n, k, code, (big - base + 110).astype(np.uint8))


def mx4_weights64(rec: W12Record, cp: Mx4Copy) -> np.ndarray:
    """The weights the Q pass sees: scale * value, escapes exact (float64)."""
    v = np.array(E2M1)[cp.code & 7] * np.where(cp.code & 8, -1.0, 1.0)
    ex = cp.scale.astype(np.int64) + rec.base.astype(np.int64)[:, None] - 239
    w = v * np.repeat(np.ldexp(1.0, ex), MX4_BLOCK, axis=1)
    esc = escaped_mask(rec)
    w[esc] = bf16_to_f64(decode(rec))[esc]
    return w


def mx4_to_storage(cp: Mx4Copy) -> np.ndarray:
    """The copy's tile records, flat uint8 (padding rows zero)."""
    npad = padded_rows(cp.n)
    code = np.zeros((npad, cp.k), dtype=np.uint8)
    code[:cp.n] = cp.code
    scale = np.zeros((npad, cp.k // MX4_BLOCK), dtype=np.uint8)
    scale[:cp.n] = cp.scale
    out = []
    for t in range(npad // TILE_ROWS):
        for b in range(cp.k // TILE_COLS):
            tile = code[TILE_ROWS * t:TILE_ROWS * (t + 1), TILE_COLS * b:TILE_COLS * (b + 1)]
            rec = np.zeros(1088, dtype=np.uint8)
            for g in range(4):
                for r in range(TILE_ROWS):
                    c = tile[r, 32 * g:32 * g + 32]
                    rec[16 * (r + 16 * g):16 * (r + 16 * g) + 16] = c[0::2] | c[1::2] << 4
                    rec[1024 + r + 16 * g] = scale[TILE_ROWS * t + r, 4 * b + g]
            out.append(rec)
    return np.concatenate(out)
