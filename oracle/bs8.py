"""Block-scaled 8-bit KV cache (oracle; test infrastructure only).

E4M3 codes with one power-of-two scale for each block of 16 positions of a kv
head, K and V apart: scale 2^e with the smallest e in [-64, 64] for which no
|x| of the block exceeds 448 * 2^e; code = E4M3 of x * 2^-e, to nearest even,
saturating.  Rows appended to a block that holds earlier rows: the block's e
becomes the larger of the old one and the one the new rows ask for, and the
earlier codes are rounded again after the division by the power of two.

A unit (one page, layer, kv head, K or V) is 256 x 256 codes in cores of
8 positions x 16 dims, then the 16 blocks' scales as float32.
"""
from __future__ import annotations

import math

import numpy as np

from . import fp8

PAGE, DIM, BLOCK = 256, 256, 16
CODE_BYTES = PAGE * DIM
UNIT_BYTES = CODE_BYTES + 4 * (PAGE // BLOCK)
MAX_EXP = 64


def exponent(x: np.ndarray) -> int:
    """e of a block of values (non-finite ones do not count)."""
    a = np.abs(np.asarray(x, np.float64))
    top = float(np.max(np.where(np.isfinite(a), a, 0.0), initial=0.0))
    e = -MAX_EXP
    while e < MAX_EXP and top > math.ldexp(448.0, e):
        e += 1
    return e


def code_offset(row: int, dim: int) -> int:
    """Byte of the code of a page's row and dim within its unit."""
    return ((row // 8) * 16 + dim // 16) * 128 + (row % 8) * 16 + dim % 16


_OFFSETS = np.array([[code_offset(r, d) for d in range(DIM)] for r in range(PAGE)])


class Cache:
    """One kv head of one slot, K or V: codes in position order and an exponent per block."""

    def __init__(self):
        self.codes = np.zeros((0, DIM), np.uint8)
        self.exps: list = []

    def append(self, x: np.ndarray) -> None:
        x = np.asarray(x, np.float32)
        at = 0
        while at < len(x):
            n = len(self.codes)
            used = n % BLOCK
            new = x[at:at + BLOCK - used]
            e = exponent(new)
            if used:
                old = self.exps[-1]
                e = max(e, old)
                if e > old:
                    kept = fp8.decode(self.codes[n - used:]) * math.ldexp(1.0, old - e)
                    self.codes[n - used:] = fp8.encode(kept)[0]
                self.exps[-1] = e
            else:
                self.exps.append(e)
            # the division by a power of two is exact in float64; the float32 it is handed on in loses only what is
            # below 2^-149, far under the smallest code
            scaled = np.clip(np.asarray(new, np.float64) * math.ldexp(1.0, -e), -3.0e38, 3.0e38)
            scaled = np.where(np.isinf(new), new, np.where(np.isnan(new), np.nan, scaled))
            self.codes = np.concatenate([self.codes, fp8.encode(scaled.astype(np.float32))[0]])
            at += len(new)

    def truncate(self, n: int) -> None:
        """Rollback: rows from n on go; the last block keeps its scale."""
        self.codes = self.codes[:n]
        self.exps = self.exps[:(n + BLOCK - 1) // BLOCK]

    def values(self) -> np.ndarray:
        e = np.repeat(np.array(self.exps, np.float64), BLOCK)[:len(self.codes)]
        return fp8.decode(self.codes) * np.exp2(e)[:, None]


def unit_offset(layers: int, heads: int, page, layer: int, head: int, kv: int):
    return (((page * layers + layer) * heads + head) * 2 + kv) * UNIT_BYTES


def read_codes(unit: np.ndarray, rows) -> np.ndarray:
    """Codes [len(rows), 256] of a unit's bytes."""
    return unit[_OFFSETS[rows]]


def read_scales(unit: np.ndarray) -> np.ndarray:
    return unit[CODE_BYTES:].copy().view(np.float32)


def attention(q: np.ndarray, k: np.ndarray, v: np.ndarray, n_ctx: int, group: int = 8) -> np.ndarray:
    """Verify attention of one slot in float64: q [T, Hq, D]; k, v [Hkv, L, D] decoded; token t sees [0, n_ctx + t]."""
    q = np.asarray(q, np.float64)
    T, Hq, D = q.shape
    L = k.shape[1]
    out = np.empty((T, Hq, D))
    hidden = np.arange(L)[None, :] > n_ctx + np.arange(T)[:, None]
    for h in range(Hq):
        s = q[:, h] @ np.asarray(k[h // group], np.float64).T / 16.0
        s[hidden] = -np.inf
        p = np.exp(s - s.max(axis=1, keepdims=True))
        out[:, h] = (p @ np.asarray(v[h // group], np.float64)) / p.sum(axis=1, keepdims=True)
    return out
