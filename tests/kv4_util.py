"""Seeded cases of the 4-bit paged cache for the CPU and GPU tests, and the
bound on what attention over it may be off."""
import numpy as np

import oracle.kv4 as kv4


def make_pool(rng, lengths, page, H, D, spare=2, W=None, fill=True, scale=1.0):
    """Pages (uint32) of random positions and a shuffled page table int32 [B, W]."""
    used = [-(-max(0, int(l)) // page) for l in lengths]
    W = max(used + [1]) if W is None else W
    P = sum(min(u, W) for u in used) + spare
    free = rng.permutation(P).astype(np.int32)
    table = np.full((len(lengths), W), -1, np.int32)
    at = 0
    for b, u in enumerate(used):
        u = min(u, W)
        table[b, :u] = free[at:at + u]
        at += u
    pages = np.zeros((P, H, kv4.page_words(page, D)), np.uint32)
    if fill:
        n = P * page
        mag = np.exp(rng.standard_normal((2, H, D)) * 0.5) * scale
        x = (rng.standard_normal((2, n, H, D)) * mag[:, None]).astype(np.float32)
        # positions 0 .. n-1 of one sequence that owns every page in order
        kv4.append(pages, page, [(0, i) for i in range(n)], np.arange(P, dtype=np.int32)[None], x[0], x[1])
    return pages, table


def attend_case(pages, table, lengths, page, D, q, T, offsets=None, window=0, sinks=0, scale=None):
    """(exact output [T, Hq, D], bound on the error before the output's rounding, rows of a sequence)."""
    B, Hq = len(lengths), q.shape[1]
    G = Hq // pages.shape[1]
    scale = D ** -0.5 if scale is None else scale
    w = kv4.group_width(D)
    out, bound, own = np.zeros((T, Hq, D)), np.zeros((T, Hq, D)), np.zeros(T, bool)
    where = kv4.rows(T, B, lengths, offsets)
    for b in range(B):
        at = [r for r in range(T) if where[r][0] == b]
        if not at:
            continue
        own[at] = True
        pos = np.array([where[r][1] for r in at])
        L = max(0, min(int(pos.max()) + 1, table.shape[1] * page))
        k, v, there = kv4.values(pages, page, table[b], np.arange(L), D)
        seen = kv4.visible(pos, L, there, window, sinks)
        o, p = kv4.attend(q[at], k, v, seen, scale)
        out[at] = o
        bound[at] = error_bound(q[at], k, v, p, seen, o, scale, G, w)
    return out, bound, own


def error_bound(q, k, v, p, seen, o, scale, G, w):
    """What the kernels may be off, to first order, for finite inputs.

    With u = 2^-24 (half a step of binary32), D channels and L positions:
      scores: products of codes and scaled queries are exact; a group's sum of D
        terms, the zero point's term (itself a sum of D) and the factors round at
        most 2 D + 12 times, relative to the sum of the terms' magnitudes
        A_t <= scale * s_t sum_d |q_d| (n_td + z_t) <= scale * 30 s_t sum_d |q_d|
        (n, z <= 15), and s_t is at most a seventh of the group's largest value:
        that has hi or -lo >= 7.5 t >= 7.38 s, hence a code 7 or more off z; as an exponent a score x rounds once more, 2^-24 |x|, and the
        exponential is good to 2^-22.  One weight is off by
        e_t <= (2 D + 12) u A_t + 4 u |x_t| + 2^-22 relatively (|x| <= A).
      weights to binary16: 2^-11 relatively, or 2^-24 of the row's largest
        weight-times-scale (subnormals; the largest is at least 1 when the row's
        unit is set, and at least half its bound after).
      sums over positions: at most L + D roundings of binary32 on codes and zero
        points together, relative to sum_t p_t s_t (n + z) <= sum_t p_t 30 s_t.
      value codes: exact.
    The output is sum p v / sum p: weights off by e_t move it by at most
    sum p_t e_t (|v_t| + |o|).
    """
    n, Hq, D = q.shape
    L, H, _ = k.shape
    u = 2.0 ** -24
    if L == 0:
        return np.zeros((n, Hq, D))
    any_sees = seen.any(0)                                    # what is out of sight may be anything
    k, v = (np.where(any_sees[:, None, None], np.abs(a), 0.0) for a in (k, v))
    sk, sv = (a.reshape(L, H, D // w, w).max(-1) / 7 for a in (k, v))       # at least the scales
    qa = np.abs(q).reshape(n, H, G, D // w, w).sum(-1)
    A = abs(scale) * 30 * np.einsum("nhgc,lhc->nhgl", qa, sk)
    p = p.reshape(n, H, G, L)
    e = (2 * D + 12 + 4) * u * A + 2.0 ** -22
    big = (p[..., None] * sv.transpose(1, 0, 2)[None, :, None]).max(3)      # [n, H, G, Gd]
    per = np.einsum("nhgl,lhd->nhgd", p * (e + 2.0 ** -11), v) + (p * e).sum(-1)[..., None] * np.abs(o).reshape(n, H, G, D)
    seen_by = seen.sum(-1)[:, None, None, None]
    flat = seen_by * 2.0 ** -24 * 16 * big + (L + D) * u * 30 * np.einsum("nhgl,lhc->nhgc", p, sv)
    return (per + np.repeat(flat, w, -1)).reshape(n, Hq, D)
