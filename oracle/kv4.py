"""Oracle for the 4-bit paged KV cache (test infrastructure; see oracle/__init__.py).

「第4章：量化」 §1.1-1.2: asymmetric codes x_int = round(x / s) + z,
x_hat = (x_int - z) s; 「LLM推理降本五要素」 §5.2: the cache is quantized as it
grows.  Readings:
  * groups of min(D, 128) channels of one position and head; zero lies in every
    group's range, so 0 <= z <= 15; the scale is rounded up to 7 significant
    bits, which keeps (q - z) s exact in 11;
  * decisions in binary32 with correctly rounded quotients, as everywhere here;
  * a scale below 2^-126 counts as zero; a group with a value that is not
    finite is NaN;
  * pages, page table, lengths and offsets as the C header describes them.
Attention and values are binary64.
"""
from __future__ import annotations

import numpy as np

NAN_WORD = 0x7FC00000


def group_width(D: int) -> int:
    return min(D, 128)


def page_words(page: int, D: int) -> int:
    return page * (D // 4 + 2 * (D // group_width(D)))


def round_up_7(t: np.ndarray) -> np.ndarray:
    """float32 >= 0, rounded up to 7 significant bits (a multiple of 2^-132 below 2^-126)."""
    m, e = np.frexp(t.astype(np.float64))
    step = np.ldexp(1.0, np.maximum(e - 7, -132))
    with np.errstate(over="ignore"):
        return (np.ceil(t.astype(np.float64) / step) * step).astype(np.float32)


def quantize_groups(x: np.ndarray):
    """float32 [..., D] -> (codes uint8 [..., D], scale float32 [..., Gd], zero uint8 [..., Gd])."""
    x = np.asarray(x, np.float32)
    D, w = x.shape[-1], group_width(x.shape[-1])
    g = x.reshape(x.shape[:-1] + (D // w, w))
    bad = ~np.isfinite(g).all(-1)
    g = np.where(bad[..., None], np.float32(0), g)
    lo = np.minimum(g.min(-1), np.float32(0))
    hi = np.maximum(g.max(-1), np.float32(0))
    with np.errstate(over="ignore"):
        t = (hi - lo) / np.float32(15)
        bad |= ~np.isfinite(t)
        s = round_up_7(np.where(bad, np.float32(0), t))
    bad |= ~np.isfinite(s)
    s = np.where(bad | (s < np.float32(2.0 ** -126)), np.float32(0), s)
    d = np.where(s > 0, s, np.float32(1))
    z = np.where(s > 0, np.clip(np.rint(-lo / d), 0, 15), 0).astype(np.float32)
    q = np.clip(np.rint(g / d[..., None]) + z[..., None], 0, 15)
    q = np.where((s > 0)[..., None], q, 0).astype(np.uint8)
    return q.reshape(x.shape), np.where(bad, np.float32(np.nan), s), z.astype(np.uint8)


def group_words(scale: np.ndarray, zero: np.ndarray) -> np.ndarray:
    w = np.ascontiguousarray(scale, np.float32).view(np.uint32) | zero.astype(np.uint32)
    return np.where(np.isnan(scale), np.uint32(NAN_WORD), w)


def rotate(x: np.ndarray, pos: np.ndarray, cos: np.ndarray, sin: np.ndarray, interleaved: bool) -> np.ndarray:
    """x float32 [T, H, D] turned by the angles of pos [T], binary32 step by step."""
    x = np.array(x, np.float32)
    half = cos.shape[1]
    i = np.arange(half)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
    c, s = cos[pos][:, None], sin[pos][:, None]
    u, w = x[..., a].copy(), x[..., b].copy()
    x[..., a] = u * c - w * s
    x[..., b] = w * c + u * s
    return x


def rows(T: int, B: int, lengths, offsets=None):
    """[(sequence, position)] of each row; sequence -1 for a row of none."""
    if offsets is None:
        offsets = [i * (T // B) for i in range(B + 1)]
    out = []
    for r in range(T):
        b = next((j for j in range(B) if offsets[j] <= r < offsets[j + 1]), -1)
        out.append((b, int(lengths[b]) - int(offsets[b + 1]) + r if b >= 0 else -1))
    return out


def _place(pos, table_row, page, P):
    """(page id, slot) of a position, or None."""
    if pos < 0 or pos >= len(table_row) * page:
        return None
    i = int(table_row[pos // page])
    return (i, pos % page) if 0 <= i < P else None


def append(pages, page, where, table, k, v):
    """Write k, v float32 [T, H, D] (k rotated) of rows `where` into pages (uint32 [P, H, words], in place)."""
    P, H, _ = pages.shape
    D = k.shape[2]
    c, Gd = D // 8, D // group_width(D)
    for keys, x in ((True, k), (False, v)):
        q, s, z = quantize_groups(x)
        nib = q.reshape(q.shape[:-1] + (c, 8)).astype(np.uint32)
        words = np.zeros(nib.shape[:-1], np.uint32)
        for j in range(8):
            words |= nib[..., j] << np.uint32(4 * j)
        gw = group_words(s, z)
        for r, (b, pos) in enumerate(where):
            at = _place(pos, table[b], page, P) if b >= 0 else None
            if at is None:
                continue
            i, slot = at
            if keys:
                pages[i, :, slot * c:(slot + 1) * c] = words[r]
            else:
                first = page * c + (slot // 4) * 4 * c + slot % 4
                pages[i, :, first:first + 4 * c:4] = words[r]
            first = 2 * page * c + (0 if keys else Gd * page) + slot
            pages[i, :, first:first + Gd * page:page] = gw[r]


def values(pages, page, table_row, positions, D):
    """(k, v) float64 [n, H, D] at positions of one sequence and [n] whether there is a page."""
    P, H, _ = pages.shape
    c, w = D // 8, group_width(D)
    Gd = D // w
    k, v = np.zeros((len(positions), H, D)), np.zeros((len(positions), H, D))
    there = np.zeros(len(positions), bool)
    for n, pos in enumerate(positions):
        at = _place(int(pos), table_row, page, P)
        if at is None:
            continue
        there[n] = True
        i, slot = at
        for keys, out in ((True, k), (False, v)):
            if keys:
                words = pages[i, :, slot * c:(slot + 1) * c]
            else:
                first = page * c + (slot // 4) * 4 * c + slot % 4
                words = pages[i, :, first:first + 4 * c:4]
            first = 2 * page * c + (0 if keys else Gd * page) + slot
            gw = np.ascontiguousarray(pages[i, :, first:first + Gd * page:page])
            s = (gw & np.uint32(0xFFFF0000)).view(np.float32).astype(np.float64)
            z = (gw & np.uint32(15)).astype(np.float64)
            q = np.stack([(words >> np.uint32(4 * j)) & np.uint32(15) for j in range(8)], -1).reshape(H, D)
            out[n] = (q - np.repeat(z, w, 1)) * np.repeat(s, w, 1)
    return k, v, there


def visible(pos, n_keys, there, window, sinks):
    """bool [rows, n_keys]: what rows at positions pos see."""
    j = np.arange(n_keys)[None]
    p = np.asarray(pos)[:, None]
    seen = (j <= p) & there[None]
    if window:
        seen &= (j > p - window) | (j < sinks)
    return seen


def attend(q, k, v, seen, scale):
    """q [n, Hq, D], k, v [L, H, D], seen [n, L], all float64 -> (out, weights [n, Hq, L])."""
    n, Hq, D = q.shape
    L, H, _ = k.shape
    if L == 0:
        return np.zeros((n, Hq, D)), np.zeros((n, Hq, 0))
    G = Hq // H
    any_sees = seen.any(0)
    k, v = (np.where(any_sees[:, None, None], a, 0.0) for a in (k, v))
    x = np.einsum("nhgd,lhd->nhgl", q.reshape(n, H, G, D), k).reshape(n, Hq, L) * scale
    x = np.where(seen[:, None], x, -np.inf)
    top = x.max(-1, keepdims=True)
    w = np.where(seen[:, None], np.exp(x - np.where(np.isfinite(top), top, 0.0)), 0.0)
    w /= np.maximum(w.sum(-1, keepdims=True), 1e-300)
    out = np.einsum("nhgl,lhd->nhgd", w.reshape(n, H, G, L), v).reshape(n, Hq, D)
    return out, w
