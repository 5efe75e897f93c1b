"""Oracle for the e4m3 paths with a scale for each block of 128 (test
infrastructure; see oracle/__init__.py).

Codes and scales in binary32 with correctly rounded quotients, as the GPU path
decides them; products in float64.  A code byte is sign, 4 exponent bits
(bias 7) and 3 mantissa bits; 0x7f / 0xff are NaN and never written.
"""
from __future__ import annotations

import numpy as np

BLOCK = 128
TOP = np.float32(448.0)


def f8_values() -> np.ndarray:
    """The 256 code values in float64 (NaN for 0x7f and 0xff)."""
    out = np.zeros(256)
    for b in range(256):
        e, m = (b >> 3) & 15, b & 7
        v = np.nan if e == 15 and m == 7 else (m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7))
        out[b] = -v if b >= 128 else v
    return out


_VALUES = f8_values()
_POS = _VALUES[:127]          # 0 .. 448, rising with the code


def f8_decode(codes: np.ndarray) -> np.ndarray:
    return _VALUES[codes]


def f8_encode(q: np.ndarray) -> np.ndarray:
    """Nearest code of values in [-448, 448], halves to the even code."""
    q = np.asarray(q, np.float64)
    a = np.abs(q)
    hi = np.clip(np.searchsorted(_POS, a, side="left"), 1, 126)
    lo = hi - 1
    dlo, dhi = a - _POS[lo], _POS[hi] - a       # exact: at most 24 + few bits apart
    up = (dhi < dlo) | ((dhi == dlo) & (hi % 2 == 0))
    code = np.where(up, hi, lo).astype(np.uint8)
    return np.where(np.signbit(q), code | 0x80, code).astype(np.uint8)


def _codes(x: np.ndarray, s: np.ndarray) -> np.ndarray:
    """x float32, s float32 broadcast over it."""
    with np.errstate(divide="ignore", invalid="ignore", over="ignore"):
        q = (x / s).astype(np.float32)
    on = (s > 0) & np.isfinite(s)      # a block with an infinity or NaN: zero codes, s says so
    return np.where(on, f8_encode(np.clip(np.where(on, q, np.float32(0)), -TOP, TOP)), np.uint8(0)).astype(np.uint8)


def blocks(n: int) -> int:
    return (n + BLOCK - 1) // BLOCK


def quantize_f8_g128(x: np.ndarray):
    """x float32 [M, K] -> (codes uint8 [M, K], scales float32 [M, G])."""
    x = np.asarray(x, np.float32)
    M, K = x.shape
    codes, scales = np.zeros((M, K), np.uint8), np.zeros((M, blocks(K)), np.float32)
    for g in range(blocks(K)):
        part = x[:, g * BLOCK:(g + 1) * BLOCK]
        s = (np.abs(part).max(1) / TOP).astype(np.float32)
        scales[:, g] = s
        codes[:, g * BLOCK:(g + 1) * BLOCK] = _codes(part, s[:, None])
    return codes, scales


def quantize_weight_f8_b128(w: np.ndarray):
    """w float32 [K, N] -> (codes uint8 [N, K], scales float32 [B, G])."""
    t = np.ascontiguousarray(np.asarray(w, np.float32).T)
    N, K = t.shape
    codes, scales = np.zeros((N, K), np.uint8), np.zeros((blocks(N), blocks(K)), np.float32)
    for b in range(blocks(N)):
        for g in range(blocks(K)):
            at = (slice(b * BLOCK, (b + 1) * BLOCK), slice(g * BLOCK, (g + 1) * BLOCK))
            s = np.float32(np.abs(t[at]).max() / TOP)
            scales[b, g] = s
            codes[at] = _codes(t[at], s)
    return codes, scales


def gemm_f8_b128(xq, xs, wq, ws):
    """(y, B, D) in float64: the product, the sum of the terms' magnitudes, and
    the sum over runs of 8 inputs of the largest term's magnitude."""
    M, K = xq.shape
    N = wq.shape[0]
    x, w = f8_decode(xq), f8_decode(wq)
    y, B, D = (np.zeros((M, N)) for _ in range(3))
    for g in range(blocks(K)):
        sc = xs[:, g, None].astype(np.float64) * np.repeat(ws[:, g].astype(np.float64), BLOCK)[None, :N]
        for k in range(g * BLOCK, min(K, (g + 1) * BLOCK), 8):
            a, b = x[:, k:k + 8], w[:, k:k + 8]
            y += (a @ b.T) * sc
            B += (np.abs(a) @ np.abs(b).T) * np.abs(sc)
            top = np.zeros((M, N))
            for i in range(a.shape[1]):
                np.maximum(top, np.abs(np.outer(a[:, i], b[:, i])), out=top)
            D += top * np.abs(sc)
    return y, B, D
