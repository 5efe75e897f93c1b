"""Oracle for expert routing (test infrastructure; see oracle/__init__.py): one
token and one expert at a time, in float64."""
from __future__ import annotations

import numpy as np


def route_experts(logits, k, bias=None, sigmoid=False, groups=1, top_groups=1, renormalize=True, scale=1.0):
    """logits float32 [T, E] -> (expert int32 [T, k], weight float64 [T, k])."""
    T, E = logits.shape
    expert = np.full((T, k), -1, np.int32)
    weight = np.zeros((T, k))
    for t in range(T):
        x = [float("-inf") if np.isnan(v) else min(float(v), 3.4028234663852886e38) for v in logits[t]]
        is_open = [v > float("-inf") for v in x]
        if sigmoid:
            with np.errstate(over="ignore"):
                p = [float(1 / (1 + np.exp(-np.float64(v)))) for v in x]
        else:
            top = max(x)
            p = [float(np.exp(np.float64(v - top))) if o else 0.0 for v, o in zip(x, is_open)]
            total = sum(p)
            p = [v / total if total > 0 else 0.0 for v in p]
        c = [v if bias is None else v + float(bias[e]) for e, v in enumerate(p)]
        c = [v if o and v > float("-inf") else float("-inf") for v, o in zip(c, is_open)]
        left = set(e for e in range(E) if c[e] > float("-inf"))
        if groups > 1:
            size = E // groups
            value = []
            for g in range(groups):
                best = sorted((c[e] for e in range(g * size, (g + 1) * size) if c[e] > float("-inf")), reverse=True)[:2]
                value.append(sum(best) if best else float("-inf"))
            order = sorted(range(groups), key=lambda g: (-value[g], g))[:top_groups]
            left = set(e for e in left if e // size in order)
        chosen = sorted(left, key=lambda e: (-c[e], e))[:k]
        total = sum(p[e] for e in chosen)
        for j, e in enumerate(chosen):
            expert[t, j] = e
            weight[t, j] = scale * ((p[e] / total if total > 0 else 0.0) if renormalize else p[e])
    return expert, weight


def plan_experts(expert, E):
    """(offsets, row_token, slot) of int32 [T, k]."""
    T, k = expert.shape
    rows = [[] for _ in range(E)]
    for t in range(T):
        for j in range(k):
            if 0 <= expert[t, j] < E:
                rows[expert[t, j]].append((t, j))
    offsets, row_token, slot = np.zeros(E + 1, np.int32), np.full(T * k, -1, np.int32), np.full((T, k), -1, np.int32)
    r = 0
    for e in range(E):
        offsets[e] = r
        for t, j in rows[e]:
            row_token[r], slot[t, j] = t, r
            r += 1
    offsets[E] = r
    return offsets, row_token, slot


def combine_experts(rows, slot, weight):
    """(y, B) in float64: the sums and the sums of the terms' magnitudes."""
    T, k = slot.shape
    y, B = np.zeros((T, rows.shape[1])), np.zeros((T, rows.shape[1]))
    for t in range(T):
        for j in range(k):
            if 0 <= slot[t, j] < rows.shape[0]:
                term = float(weight[t, j]) * rows[slot[t, j]].astype(np.float64)
                y[t] += term
                B[t] += np.abs(term)
    return y, B
