"""Attention over the 4-bit paged cache where positions are of very different kinds: groups
that are not finite in splits of their own, values and keys of far magnitudes."""
import numpy as np
import pytest
import torch

import bit_quantized_gemm_int8_amd as qg
import oracle.kv4 as kv4
from tests.gpu_util import DEV, out_f64
from tests.kv4_util import attend_case
from tests.test_gpu_kv4 import DT, dev
from tests.test_gpu_kv4_runs import i32

pytestmark = pytest.mark.gpu


def cache(k, v, page, W=None):
    """Pages and page table of one sequence with keys and values f32 [L, H, D]."""
    L, H, D = k.shape
    P = -(-L // page)
    pages = np.zeros((P, H, kv4.page_words(page, D)), np.uint32)
    table = np.full((1, W or P), -1, np.int32)
    table[0, :P] = np.random.default_rng(P).permutation(P)
    kv4.append(pages, page, [(0, i) for i in range(L)], table, k, v)
    return pages, table


def attend(q, pages, table, length, fmt, page, window=0, sinks=0):
    """(outputs in binary64, the oracle's, the bound on the error ahead of the output's rounding)."""
    n, Hq, D = q.shape
    q = torch.from_numpy(q).to(DT[fmt])
    print(f"attend {D} {n} {Hq} {fmt} {length}", flush=True)
    got = qg.attend_kv_u4_pages(q.to(DEV), dev(pages), dev(table), i32([length]), window=window, sinks=sinks)
    torch.cuda.synchronize()
    want, bound, _ = attend_case(pages, table, [length], page, D, q.double().numpy(), n, window=window, sinks=sinks)
    return out_f64(got), want, bound


def close(got, want, bound, fmt):
    """The output's rounding on top of the bound; whatever is finite in 64 bits is finite."""
    fin = torch.finfo(DT[fmt])
    off = np.abs(got - want) - (fin.eps / 2 * (np.abs(want) + bound) + bound + fin.smallest_normal * fin.eps)
    assert (off <= 0).all(), (off.max(), np.unravel_index(np.nanargmax(off), off.shape))


# ---- groups that are not finite, by themselves in a split of the positions -----------
# splits of 8 steps of 32 positions for few rows, of 5 to 8 tiles of 64 for many

NAN_AT = [
    # D, tokens, positions, page table in positions, not finite from .. to
    (64, 1, 1793, 2048, 1792, 1793),      # the newest position, the only one of its split
    (128, 1, 1793, 2048, 1792, 1793),
    (256, 1, 1793, 2048, 1792, 1793),
    (128, 1, 257, 768, 256, 257),
    (128, 1, 1793, 2048, 1536, 1792),     # a whole split
    (64, 2, 1800, 2048, 0, 256),          # the first one
    (256, 3, 1793, 2048, 256, 512),
    (128, 200, 1540, 2048, 1344, 1345),   # the first position of a split, which some rows see alone there
    (64, 200, 1540, 2048, 1344, 1345),
    (128, 150, 2000, 2048, 1536, 2000),
    (64, 150, 2000, 2048, 0, 512),
]


@pytest.mark.parametrize("fmt", ["f16", "bf16"])
@pytest.mark.parametrize("case", NAN_AT, ids=range(len(NAN_AT)))
def test_not_finite_in_a_split(case, fmt):
    D, n, L, capacity, lo, hi = case
    page = 64
    rng = np.random.default_rng(L + lo)
    x = rng.standard_normal((2, L, 1, D)).astype(np.float32)
    x[0, lo:hi, 0, 5] = np.inf                       # keys; the whole group is NaN with it
    if D == 256:
        x[0, lo:hi, 0, 200] = np.nan
    pages, table = cache(x[0], x[1], page, capacity // page)
    q = rng.standard_normal((n, 1, D)).astype(np.float32)
    assert qg.attend_kv_u4_pages_workspace_bytes(n, 1, 1, 1, D, page, table.shape[1]) > 0      # there are splits
    got, want, bound = attend(q, pages, table, L, fmt, page)
    sees = L - n + np.arange(n) >= lo
    assert np.isnan(got[sees]).all()
    if not sees.all():
        pages, table = cache(np.where(np.isfinite(x[0]), x[0], 0), x[1], page, capacity // page)
        want, bound, _ = attend_case(pages, table, [L], page, D, torch.from_numpy(q).to(DT[fmt]).double().numpy(), n)
        close(got[~sees], want[~sees], bound[~sees], fmt)


@pytest.mark.parametrize("D,n,L", [(64, 2, 1793), (128, 2, 1793), (256, 2, 1793), (64, 150, 2000), (128, 150, 2000), (128, 3, 200), (128, 150, 200)])
def test_query_that_is_nan(D, n, L):
    """Its row is NaN, split or not; the other rows are as without it."""
    page = 64
    rng = np.random.default_rng(D + n)
    x = rng.standard_normal((2, L, 1, D)).astype(np.float32)
    pages, table = cache(x[0], x[1], page, -(-L // page) + 1)
    q = rng.standard_normal((n, 2, D)).astype(np.float32)
    q[n - 2, 1, 7] = np.nan
    q[0, 0] = np.nan
    got, _, _ = attend(q, pages, table, L, "f16", page)
    bad = np.isnan(q).any(-1)
    assert np.isnan(got[bad]).all()
    want, bound, _ = attend_case(pages, table, [L], page, D, torch.from_numpy(np.where(np.isnan(q), 0, q)).half().double().numpy(), n)
    close(got[~bad], want[~bad], bound[~bad], "f16")


# ---- values of which the first positions say nothing ----------------------------------

def history(D, L, H, rng, first, factors_first, factors_then):
    """Values f32 [L, H, D], each group of channels by its own factor up to position `first` and from there on."""
    v = rng.standard_normal((L, H, D))
    w = kv4.group_width(D)
    for t, f in ((slice(None, first), factors_first), (slice(first, None), factors_then)):
        for g in range(D // w):
            v[t, :, g * w:(g + 1) * w] *= f[g % len(f)]
    return v.astype(np.float32)


def lifted(L, D, H, rng, first, lift):
    """Keys, those from `first` on larger by `lift` in the first channel."""
    k = rng.standard_normal((L, H, D)).astype(np.float32)
    k[first:, :, 0] += lift
    return k


@pytest.mark.parametrize("first", [40, 256, 330])
@pytest.mark.parametrize("D,n", [(64, 2), (128, 2), (256, 2), (128, 40), (256, 40), (64, 150), (128, 150)])
@pytest.mark.parametrize("e0,e1", [(None, 0), (None, 28), (None, 40), (None, 110), (-100, 100), (-60, 30), (-110, 0), (100, -100), (0, -40)])
def test_values_that_grow(D, n, first, e0, e1):
    """Zeros, or far smaller (or larger) values, and then others, the later ones with as much weight or far more."""
    L, page, H = 700, 32, 1
    rng = np.random.default_rng(D + n + first)
    v = history(D, L, H, rng, first, [0.0 if e0 is None else 2.0 ** e0], [2.0 ** e1])
    for lift in (0.0, 30.0):
        pages, table = cache(lifted(L, D, H, rng, first, lift), v, page)
        q = rng.standard_normal((n, 2, D)).astype(np.float32)
        q[:, :, 0] = 10.0
        close(*attend(q, pages, table, L, "bf16", page), "bf16")


@pytest.mark.parametrize("D,n", [(64, 2), (128, 2), (256, 2), (64, 150), (128, 150)])
@pytest.mark.parametrize("e0,e1", [(60, -60), (100, 0), (20, -100)])
def test_values_that_shrink_under_higher_scores(D, n, e0, e1):
    """The later positions have the weight, by some 70 to 110 bits, and the first ones the values."""
    L, page = 700, 32
    rng = np.random.default_rng(D + n)
    for first in (40, 330):
        pages, table = cache(lifted(L, D, 1, rng, first, 50.0 if D == 64 else 60.0), history(D, L, 1, rng, first, [2.0 ** e0], [2.0 ** e1]), page)
        q = rng.standard_normal((n, 2, D)).astype(np.float32)
        q[:, :, 0] = 10.0
        close(*attend(q, pages, table, L, "bf16", page), "bf16")


@pytest.mark.parametrize("D,n", [(64, 2), (128, 2), (256, 2), (64, 12), (64, 150), (128, 150)])
@pytest.mark.parametrize("e0,e1", [(-60, 60), (-100, 24), (-20, 90)])
def test_values_that_grow_under_lower_scores(D, n, e0, e1):
    """The first positions have the weight, by some 112 bits, and the later ones the values, by 110 to 124."""
    L, page = 700, 32
    rng = np.random.default_rng(D + n)
    for first in (40, 330):
        pages, table = cache(lifted(L, D, 1, rng, first, -62.0 * (D / 64) ** 0.5), history(D, L, 1, rng, first, [2.0 ** e0], [2.0 ** e1]), page)
        q = rng.standard_normal((n, 2, D)).astype(np.float32)
        q[:, :, 0] = 10.0
        close(*attend(q, pages, table, L, "bf16", page), "bf16")


# D, tokens, query heads, positions, dtype, window, first positions
GROW = [
    (64, 10, 2, 700, "bf16", 0, 0),          # tiles of 32 rows
    (128, 12, 2, 700, "f16", 0, 0),
    (128, 5, 4, 600, "bf16", 200, 40),
    (64, 2, 1, 700, "f16", 0, 0),
    (128, 3, 1, 3000, "f16", 0, 0),          # positions in splits
    (256, 3, 1, 3000, "f16", 600, 64),
    (128, 150, 1, 2100, "bf16", 0, 0),
    (64, 150, 2, 2100, "f16", 0, 0),
    (128, 70, 4, 900, "f16", 300, 50),
]


@pytest.mark.parametrize("case", GROW, ids=range(len(GROW)))
@pytest.mark.parametrize("e0,e1", [(None, 0), (-40, 0), (6, -14), (-24, 10)])
def test_values_that_grow_more(case, e0, e1):
    D, n, Hq, L, fmt, window, sinks = case
    page = 32
    rng = np.random.default_rng(D + n + L)
    for first in (64, L - 300):
        for lift in (0.0, 20.0):
            v = history(D, L, 1, rng, first, [0.0 if e0 is None else 2.0 ** e0], [2.0 ** e1])
            pages, table = cache(lifted(L, D, 1, rng, first, lift), v, page)
            q = rng.standard_normal((n, Hq, D)).astype(np.float32)
            q[:, :, 0] = 10.0
            close(*attend(q, pages, table, L, fmt, page, window, sinks), fmt)


def test_values_that_grow_eight_waves():
    D, L, page, H = 64, 1100, 64, 256
    rng = np.random.default_rng(1)
    for first, f0, f1 in ((256, 0.0, 2.0 ** 40), (300, 2.0 ** -90, 2.0 ** 60)):
        pages, table = cache(rng.standard_normal((L, H, D)).astype(np.float32), history(D, L, H, rng, first, [f0], [f1]), page)
        close(*attend(rng.standard_normal((1, H, D)).astype(np.float32), pages, table, L, "bf16", page), "bf16")


@pytest.mark.parametrize("fmt", ["f16", "bf16"])
@pytest.mark.parametrize("first", [40, 128, 330])
@pytest.mark.parametrize("f0,f1", [((1, 0), (1, 1)), ((0, 1), (1, 1)), ((1, 2.0 ** -20), (1, 1)), ((1, 1), (1, 2.0 ** 14)), ((2.0 ** -14, 1), (1, 1)),
                                   ((1, 1), (2.0 ** -20, 1)), ((1, 1), (1, 2.0 ** -14)), ((1, 0), (0, 1))])
def test_halves_of_wide_heads(fmt, first, f0, f1):
    """Heads of 256: what one half of the channels holds leaves the other half's outputs alone."""
    D, L, page, H = 256, 600, 32, 1
    rng = np.random.default_rng(first)
    v = history(D, L, H, rng, first, f0, f1)
    for lift in (0.0, 30.0, -30.0):
        pages, table = cache(lifted(L, D, H, rng, first, lift), v, page)
        for n in (1, 30):
            q = rng.standard_normal((n, 2, D)).astype(np.float32)
            q[:, :, 0] = 10.0
            close(*attend(q, pages, table, L, fmt, page), fmt)


def test_halves_of_wide_heads_far_apart():
    D, L, page, H = 256, 600, 32, 1
    rng = np.random.default_rng(7)
    for f0, f1 in (((1, 2.0 ** -30), (1, 2.0 ** 30)), ((2.0 ** 100, 2.0 ** -100), (2.0 ** -100, 2.0 ** 100))):
        v = history(D, L, H, rng, 140, f0, f1)
        pages, table = cache(lifted(L, D, H, rng, 140, 8.0), v, page)
        q = rng.standard_normal((5, 2, D)).astype(np.float32)
        q[:, :, 0] = 10.0
        close(*attend(q, pages, table, L, "bf16", page), "bf16")


# ---- values up to the end of the range -----------------------------------------------

@pytest.mark.parametrize("D,n,L", [(64, 1, 1), (128, 1, 1), (256, 1, 1), (128, 2, 700), (64, 2, 700), (256, 2, 700), (256, 9, 200),
                                   (64, 150, 160), (128, 150, 160), (128, 150, 2000), (64, 150, 2000)])
@pytest.mark.parametrize("top", [1e33, 5e33, 1e36, 1.6e38])
def test_largest_values(D, n, L, top):
    page = 32
    rng = np.random.default_rng(D + n + L)
    k = rng.standard_normal((L, 1, D)).astype(np.float32)
    v = (rng.uniform(-1, 1, (L, 1, D)) * top).astype(np.float32)
    v[:, :, ::5] = np.abs(v[:, :, ::5])               # channels whose sum over the positions is far larger
    v[::3] /= 64
    pages, table = cache(k, v, page)
    for sharp in (1.0, 40.0):
        got, want, bound = attend((rng.standard_normal((n, 2, D)) * sharp).astype(np.float32), pages, table, L, "bf16", page)
        close(got, want, bound, "bf16")


# ---- keys of far magnitudes ------------------------------------------------------------

@pytest.mark.parametrize("D,n", [(64, 2), (128, 2), (256, 2), (64, 150), (128, 150)])
@pytest.mark.parametrize("e,first", [(60, 0), (110, 0), (120, 0), (124, 0), (-60, 0), (-110, 0), (60, 70), (30, 330), (100, 70), (124, 70), (-100, 70)])
def test_keys_far_from_one(D, n, e, first):
    """Keys by 2^e, the first ones zeros, under queries by 2^-e."""
    L, page = 700, 32
    rng = np.random.default_rng(D + n)
    k = np.ldexp(rng.standard_normal((L, 1, D)), e).astype(np.float32)
    k[:first] = 0
    pages, table = cache(k, rng.standard_normal((L, 1, D)).astype(np.float32), page)
    q = np.ldexp(rng.standard_normal((n, 2, D)), -e).astype(np.float32)
    close(*attend(q, pages, table, L, "bf16", page), "bf16")


@pytest.mark.parametrize("n", [1, 9])
def test_queries_of_far_elements(n):
    """Elements of a query below 2^-39 of its largest count as one number in the codes' and in
    the zero points' sums: positions whose keys are zeros there, with a zero point of 15,
    score as the others do.  A score may be off by scale 2^-39 max |q| sum |k|, here 2^-5.1."""
    D, L, page, s = 256, 300, 32, 2.0 ** 34
    rng = np.random.default_rng(n)
    k = np.zeros((L, 1, D), np.float32)
    k[::2, 0, 255] = -15 * s
    v = rng.standard_normal((L, 1, D)).astype(np.float32)
    pages, table = cache(k, v, page)
    q = np.zeros((n, 1, D), np.float32)
    q[:, :, 0] = 1.0
    q[:, :, 128:255] = 2.0 ** -41
    got, want, bound = attend(q, pages, table, L, "bf16", page)
    _, vv, _ = kv4.values(pages, page, table[0], np.arange(L), D)
    off = D ** -0.5 * 2.0 ** -39 * 15 * s                 # of a score; of the weights relatively, both ways
    fin = torch.finfo(torch.bfloat16)
    for r in range(n):
        seen = np.abs(vv[:L - n + r + 1]).mean(0)
        limit = np.expm1(2 * off) * (seen + np.abs(want[r]))
        # the terms of the scores are far below the sums that the bound's own first term counts
        assert (np.abs(got[r] - want[r]) <= limit * (1 + fin.eps) + fin.eps / 2 * np.abs(want[r]) + 2.0 ** -9 * seen).all()
