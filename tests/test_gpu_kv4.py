"""GPU parity of the 4-bit paged cache: appended pages bit for bit, values and
attention against the oracle in 64 bits."""
import numpy as np
import pytest
import torch

import bit_quantized_gemm_int8_amd as qg
import oracle.kv4 as kv4
from tests.gpu_util import DEV, out_f64
from tests.kv4_util import attend_case, make_pool

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def dev(a):
    a = np.ascontiguousarray(a)
    return torch.from_numpy(a.view(np.int32) if a.dtype == np.uint32 else a).to(DEV)


def host_pages(t):
    return t.cpu().numpy().view(np.uint32)


def tables(rng, rows, rot):
    angle = rng.random((rows, rot // 2)) * 6.28
    return np.cos(angle).astype(np.float32), np.sin(angle).astype(np.float32)


# D, page, H, Hq, dtype, rotated channels, interleaved, lengths, offsets (None: one row each)
APPEND = [
    (128, 64, 8, 32, "bf16", 128, False, [1, 64, 65, 300], None),
    (128, 16, 2, 2, "f16", 64, True, [9, 40, 40], [0, 9, 30, 34]),
    (128, 32, 3, 9, "f32", 96, False, [100, 7], [2, 60, 65]),
    (64, 16, 1, 4, "bf16", 64, False, [17, 0, 33], [0, 17, 17, 50]),
    (64, 256, 5, 5, "f16", 16, True, [300], [0, 300]),
    (256, 128, 2, 4, "f32", 256, False, [130, 5], [0, 130, 131]),
    (256, 16, 1, 8, "bf16", 128, True, [31, 2], [0, 31, 33]),
    (256, 64, 1, 0, "f16", 224, False, [10], [0, 4]),
    (128, 64, 4, 0, "bf16", 0, False, [70, 3], [0, 66, 69]),
    (128, 64, 33, 65, "bf16", 128, False, [5, 6], None),
]


@pytest.mark.parametrize("case", APPEND, ids=range(len(APPEND)))
def test_append_bits(case):
    D, page, H, Hq, fmt, rot, inter, lengths, offsets = case
    rng = np.random.default_rng(D + page + H)
    B = len(lengths)
    T = B if offsets is None else offsets[-1] + 3
    pages, table = make_pool(rng, lengths, page, H, D)
    print(f"append {case}", flush=True)
    # a fused projection's rows, some of them larger than others
    x = torch.from_numpy((rng.standard_normal((T, Hq + 2 * H, D)) * np.exp(rng.standard_normal((T, Hq + 2 * H, 1)))).astype(np.float32))
    x[0, -1] = 0
    x = x.to(DT[fmt])
    q, k, v = x.to(DEV).split([Hq, H, H], 1)
    cos, sin = tables(rng, max(lengths) + 1, rot) if rot else (None, None)
    out = torch.full((T, Hq, D), 7.0, dtype=DT[fmt], device=DEV) if Hq else None
    pd = dev(pages)
    args = dict(offsets=None if offsets is None else dev(np.array(offsets, np.int32)),
                cos=None if cos is None else dev(cos), sin=None if sin is None else dev(sin), interleaved=inter)
    got = qg.append_kv_u4_pages(k, v, pd, dev(table), dev(np.array(lengths, np.int32)), q=q if Hq else None, out=out, **args)
    torch.cuda.synchronize()
    where = kv4.rows(T, B, lengths, offsets)
    pos = np.array([max(p, 0) for _, p in where])
    xf = x.float().numpy()
    turn = (lambda a: kv4.rotate(a, pos, cos, sin, inter)) if rot else (lambda a: a)
    kv4.append(pages, page, where, table, turn(xf[:, Hq:Hq + H]), xf[:, Hq + H:])
    np.testing.assert_array_equal(host_pages(pd), pages)
    if not Hq:
        assert got is None
        return
    want = torch.from_numpy(turn(xf[:, :Hq])).to(DT[fmt]).float().numpy()
    own = np.array([b >= 0 for b, _ in where])
    neg = np.array([p < 0 for _, p in where]) & bool(rot)
    want[neg] = 0
    want[~own] = 7.0
    np.testing.assert_array_equal(out_f64(got), want.astype(np.float64))


def test_append_rows_that_do_not_fit():
    """Positions past the page table, past the rotation tables, below zero, and
    table entries that are no page: nothing is written, queries as documented."""
    rng = np.random.default_rng(8)
    D, page, H = 64, 16, 2
    lengths, offsets = [40, 20, 2, 2 ** 31 - 1, -5], [0, 4, 8, 12, 13, 14]
    T = 14
    pages, table = make_pool(rng, [32, 20, 2, 16, 16], page, H, D)
    table[1] = [table[1][0], pages.shape[0]]          # positions 16 .. 19: an id past the pool
    table[4] = [-1, -2 ** 31]
    x = rng.standard_normal((T, 3 * H, D)).astype(np.float32)
    cos, sin = tables(rng, 38, 32)                   # positions 38, 39 have no angle
    q, k, v = torch.from_numpy(x).to(DEV).split(H, 1)
    pd = dev(pages)
    got = qg.append_kv_u4_pages(k, v, pd, dev(table), dev(np.array(lengths, np.int32)),
                                offsets=dev(np.array(offsets, np.int32)), q=q, cos=dev(cos), sin=dev(sin))
    torch.cuda.synchronize()
    where = kv4.rows(T, 5, lengths, offsets)
    pos = np.array([p for _, p in where])
    known = (pos >= 0) & (pos < 38)
    assert pos[:4].tolist() == [36, 37, 38, 39] and pos[8:12].tolist() == [-2, -1, 0, 1]
    at = np.where(known, pos, 0)
    kept = [w if known[i] else (-1, -1) for i, w in enumerate(where)]
    kv4.append(pages, page, kept, table, kv4.rotate(x[:, H:2 * H], at, cos, sin, False), x[:, 2 * H:])
    np.testing.assert_array_equal(host_pages(pd), pages)
    want = kv4.rotate(x[:, :H], at, cos, sin, False)
    want[~known] = 0
    np.testing.assert_array_equal(out_f64(got), want.astype(np.float64))


def test_append_not_finite_and_subnormal():
    rng = np.random.default_rng(9)
    D, page, H, T = 128, 16, 2, 8
    x = rng.standard_normal((T, 2 * H, D)).astype(np.float32)
    x[0, 0, 3], x[1, 1, 100], x[2, 2, 0] = np.inf, np.nan, -np.inf
    x[3, 0, :2] = 3e38, -3e38
    x[4] *= 1e-40
    x[5, 0] = 0
    x[5, 0, 7] = 1.4e-45
    x[6] *= 1e37
    pages, table = make_pool(rng, [T], page, H, D)
    k, v = torch.from_numpy(x).to(DEV).split(H, 1)
    pd = dev(pages)
    qg.append_kv_u4_pages(k, v, pd, dev(table), dev(np.array([T], np.int32)))
    kv4.append(pages, page, kv4.rows(T, 1, [T]), table, x[:, :H], x[:, H:])
    np.testing.assert_array_equal(host_pages(pd), pages)
    a, b = qg.dequantize_kv_u4_pages(pd, dev(table), dev(np.array([T], np.int32)), T, D, out_dtype=torch.float32)
    ka, vb, _ = kv4.values(pages, page, table[0], np.arange(T), D)
    np.testing.assert_array_equal(out_f64(a), ka)
    np.testing.assert_array_equal(out_f64(b), vb)


def test_append_bf16_ties():
    """Small integers and halves: quotients on and near ties, through the exact division."""
    rng = np.random.default_rng(10)
    D, page, H, T = 128, 64, 4, 64
    x = rng.integers(-60, 61, (T, 2 * H, D)).astype(np.float32) / 4
    x[:, :, 0] = 7.5
    x[:, :, 1] = -7.5                                  # s = 1, z = rne(7.5) = 8
    pages, table = make_pool(rng, [T], page, H, D)
    k, v = torch.from_numpy(x).to(torch.bfloat16).to(DEV).split(H, 1)
    pd = dev(pages)
    qg.append_kv_u4_pages(k, v, pd, dev(table), dev(np.array([T], np.int32)))
    kv4.append(pages, page, kv4.rows(T, 1, [T]), table, x[:, :H], x[:, H:])
    np.testing.assert_array_equal(host_pages(pd), pages)


@pytest.mark.parametrize("D,page,H,out", [(64, 16, 3, "f16"), (128, 128, 2, "bf16"), (256, 32, 1, "f32"), (128, 16, 40, "f16")])
def test_dequantize_values(D, page, H, out):
    rng = np.random.default_rng(D + H)
    lengths, offsets = [page + 3, 5, 0, 2 * page + 1], [1, 1 + page + 3, page + 7, page + 7, page + 20]
    T = page + 22
    pages, table = make_pool(rng, lengths, page, H, D)
    table[3, 1] = -1
    print(f"dequantize {D} {page} {H} {out}", flush=True)
    outs = tuple(torch.full((T, H, D), 5.0, dtype=DT[out], device=DEV) for _ in range(2))
    k, v = qg.dequantize_kv_u4_pages(dev(pages), dev(table), dev(np.array(lengths, np.int32)), T, D,
                                     offsets=dev(np.array(offsets, np.int32)), out_dtype=DT[out], out=outs)
    want = np.zeros((2, T, H, D))
    for r, (b, p) in enumerate(kv4.rows(T, 4, lengths, offsets)):
        if b < 0:
            want[:, r] = 5.0
        else:
            a, c, _ = kv4.values(pages, page, table[b], [p], D)
            want[0, r], want[1, r] = a[0], c[0]
    for got, w in ((k, want[0]), (v, want[1])):
        ref = torch.from_numpy(w.astype(np.float32)).to(DT[out]).float().numpy()
        np.testing.assert_array_equal(out_f64(got), ref.astype(np.float64))


# ---- attention -------------------------------------------------------------------

# D, page, H, Hq, dtype, lengths, offsets (None: n rows each), n, window, sinks
ATTEND = [
    (128, 64, 2, 8, "bf16", [1, 33, 700, 64], None, 1, 0, 0),
    (128, 16, 1, 1, "f16", [1, 2, 31, 32, 257], None, 1, 0, 0),
    (128, 32, 3, 9, "f16", [100, 500], None, 3, 0, 0),
    (128, 128, 1, 32, "bf16", [300, 41], None, 2, 0, 0),                 # 32 heads a kv head: several tiles
    (64, 16, 2, 14, "f16", [77, 640, 5], None, 5, 0, 0),
    (64, 256, 4, 4, "bf16", [1500], None, 1, 0, 0),
    (256, 16, 1, 8, "bf16", [513, 20], None, 1, 0, 0),
    (256, 64, 2, 2, "f16", [90, 600], None, 7, 0, 0),
    (128, 16, 2, 4, "f16", [200, 1300], None, 1, 64, 4),                 # window and first positions
    (128, 64, 1, 2, "bf16", [900], None, 40, 100, 0),
    (64, 32, 1, 3, "f16", [700, 90], None, 33, 17, 40),
    (256, 32, 1, 1, "bf16", [400], None, 20, 5, 1),
    (128, 32, 2, 6, "bf16", [900, 1, 64, 300], [0, 64, 65, 65, 200], 0, 0, 0),    # ragged, an empty sequence
    (128, 16, 1, 4, "f16", [35, 500, 2], [3, 38, 39, 41], 0, 33, 2),              # rows of no sequence at both ends
    (64, 64, 2, 2, "bf16", [200, 130], [0, 199, 260], 0, 0, 0),
    (256, 128, 1, 4, "f16", [150, 700], [0, 150, 151], 0, 0, 0),
    (128, 64, 2, 2, "f16", [0, 3, 300], None, 5, 0, 0),                   # fewer positions than rows: rows that see nothing
    (128, 64, 1, 4, "bf16", [257], None, 257, 0, 0),
    (64, 16, 1, 1, "f16", [130], None, 130, 1, 0),                        # only itself
    (128, 32, 1, 1, "bf16", [40], None, 1, 1, 64),
    # many rows of a sequence: the prompt kernel
    (128, 16, 2, 2, "bf16", [333, 200], None, 190, 0, 0),
    (128, 64, 1, 8, "f16", [100, 1000], None, 65, 0, 0),
    (128, 256, 3, 3, "f16", [129], None, 129, 0, 0),
    (64, 32, 2, 6, "bf16", [150, 400], None, 45, 0, 0),
    (64, 64, 1, 2, "f16", [600], None, 300, 64, 8),
    (256, 16, 1, 2, "f16", [260], None, 100, 0, 0),
    (256, 64, 2, 4, "bf16", [300, 500], None, 77, 130, 70),
    (128, 32, 1, 4, "f16", [2000], None, 50, 333, 4),                     # first positions far from the window
    (128, 64, 1, 1, "bf16", [200], None, 200, 1, 0),
    (128, 64, 1, 1, "f16", [700], None, 300, 100, 600),                   # first positions reach into the window
    (128, 64, 2, 2, "bf16", [60, 500], None, 100, 0, 0),                  # rows ahead of position 0
    (128, 32, 2, 4, "f16", [400, 9, 300, 50, 333], [0, 200, 201, 203, 253, 353], 0, 0, 0),   # rows for both kernels
    (64, 16, 20, 20, "f16", [257], None, 257, 0, 0),
    (128, 64, 2, 4, "f16", [2100, 700], None, 130, 0, 0),                 # its positions in splits
    (64, 32, 1, 4, "bf16", [2500], [1, 300], 0, 1500, 30),
    (128, 128, 3, 6, "bf16", [1800, 600, 40], [0, 130, 131, 135], 0, 0, 0),
]


def run_attend(case, seed=0, q_scale=1.0, kv_scale=1.0, scale=None, edit=None):
    D, page, H, Hq, fmt, lengths, offsets, n, window, sinks = case
    rng = np.random.default_rng(seed + D + page + H)
    B = len(lengths)
    T = B * n if offsets is None else offsets[-1] + 2
    pages, table = make_pool(rng, lengths, page, H, D, scale=kv_scale)
    if edit is not None:
        edit(pages, table)
    q = torch.from_numpy((rng.standard_normal((T, Hq, D)) * q_scale).astype(np.float32)).to(DT[fmt])
    print(f"attend {case}", flush=True)
    out = torch.full((T, Hq, D), 3.0, dtype=DT[fmt], device=DEV)
    off = None if offsets is None else np.array(offsets, np.int32)
    got = qg.attend_kv_u4_pages(q.to(DEV), dev(pages), dev(table), dev(np.array(lengths, np.int32)),
                                offsets=None if off is None else dev(off), window=window, sinks=sinks, scale=scale, out=out)
    torch.cuda.synchronize()
    assert got is out
    want, bound, own = attend_case(pages, table, lengths, page, D, q.double().numpy(), T, offsets, window, sinks, scale)
    want[~own] = 3.0
    return out_f64(got), want, bound, torch.finfo(DT[fmt]), own


def check_attend(got, want, bound, fin, own):
    tiny = fin.smallest_normal * fin.eps                  # half a step among subnormal outputs, and more
    worst = np.abs(got - want) - (fin.eps / 2 * (np.abs(want) + bound) + bound + tiny)
    assert (worst <= 0).all(), (worst.max(), np.unravel_index(worst.argmax(), worst.shape))
    assert (got[~own] == 3.0).all()
    # over all outputs: half a step of the output, of the weights, and as much again as either for the rest
    a, b = got[own], want[own]
    if np.linalg.norm(b) > 0:
        assert np.linalg.norm(a - b) <= (fin.eps / 2 + 2.0 ** -10) * np.linalg.norm(b)


@pytest.mark.parametrize("case", ATTEND, ids=range(len(ATTEND)))
def test_attend(case):
    check_attend(*run_attend(case))


@pytest.mark.parametrize("q_scale,kv_scale", [(1e-6, 1.0), (300.0, 1e-3), (1.0, 1e-20), (1e-3, 1e4)])
def test_attend_scales(q_scale, kv_scale):
    """Queries and values far from 1; the scores stay within a few hundred."""
    for n in (2, 70):
        case = (128, 32, 2, 4, "bf16", [300, 45], None, n, 0, 0)
        check_attend(*run_attend(case, q_scale=q_scale, kv_scale=kv_scale, scale=0.09 / (q_scale * kv_scale)))


@pytest.mark.parametrize("n", [3, 64])
def test_attend_sharp_and_negative_scale(n):
    """Scores hundreds apart, both ways round: the running bound rises by large steps."""
    for scale in (20.0, -20.0):
        got, want, bound, fin, own = run_attend((128, 16, 1, 4, "f16", [900, 64], None, n, 0, 0), scale=scale)
        # the weights' own errors grow with the scores and are in the bound; the norm's share is not
        worst = np.abs(got - want) - (fin.eps / 2 * (np.abs(want) + bound) + bound + 1e-7)
        assert (worst <= 0).all()


@pytest.mark.parametrize("D,n", [(128, 4), (128, 90), (256, 90)])
def test_attend_large_values_with_small_weights(D, n):
    """Some positions have values 2^30 times the others' and next to no weight,
    ahead of and behind those that decide."""
    def edit(pages, table):
        c, groups = D // 8, 32 * (D // 128)
        for i in range(pages.shape[0]):
            first = 2 * 32 * c + groups                   # value groups of 32 positions
            w = pages[i, :, first:first + groups].copy()
            s = (w & np.uint32(0xFFFF0000)).view(np.float32) * np.float32(2.0 ** (30 if i % 2 else -3))
            pages[i, :, first:first + groups] = s.view(np.uint32) | (w & np.uint32(15))
            f = 2 * 32 * c                                # key groups: large-valued pages score far lower
            w = pages[i, :, f:f + groups].copy()
            s = (w & np.uint32(0xFFFF0000)).view(np.float32) * np.float32(2.0 ** (-6 if i % 2 else 0))
            pages[i, :, f:f + groups] = s.view(np.uint32) | (w & np.uint32(15))
    got, want, bound, fin, own = run_attend((D, 32, 1, 4, "bf16", [600], None, n, 0, 0), q_scale=30.0, edit=edit)
    worst = np.abs(got - want) - (fin.eps / 2 * (np.abs(want) + bound) + bound)
    assert (worst <= 0).all()


@pytest.mark.parametrize("n", [3, 40, 70])
def test_attend_out_of_sight(n):
    """NaN, infinite and huge groups, and table entries of no page, where no row
    may look: behind the last position, outside the window, in other pages."""
    D, page = 128, 32
    case = (D, page, 2, 4, "bf16", [70, 400], None, n, 50, 2)
    c = D // 8

    def edit(pages, table):
        def spoil(b, lo, hi, word):
            for pos in range(lo, hi):
                i = table[b, pos // page]
                pages[i, :, 2 * page * c + pos % page] = word
                pages[i, :, 2 * page * c + page + pos % page] = word
        spoil(0, 70, 96, np.uint32(0x7FC00000))
        spoil(0, 2, max(2, 70 - n - 50 + 1), np.uint32(0x7F800000))
        spoil(1, 400, 416, np.uint32(0x7F7F000F))
        spoil(1, 2, 400 - n - 50 + 1, np.uint32(0xFFC00000))
        table[1, 2:9] = np.array([-1, 10 ** 9, -7, 2 ** 31 - 1, -2 ** 31, 77, -1], np.int64).astype(np.int32)
        spare = set(range(pages.shape[0])) - set(table.flatten().tolist())
        for i in spare:
            pages[i] = 0xFFFFFFFF
    check_attend(*run_attend(case, edit=edit))


@pytest.mark.parametrize("D,Hq", [(64, 1), (64, 2), (64, 4), (128, 5), (256, 2)])
def test_attend_rows_that_see_nothing_or_nan(D, Hq):
    page, gd = 16, max(1, D // 128)
    c = D // 8

    def edit(pages, table):
        table[0, :] = -1                                   # no pages at all
        i = table[1, 1]
        pages[i, :, 2 * page * c + 3] = 0x7FC00000         # a key of position 19
        i = table[2, 2]
        for g in range(gd):
            pages[i, :, 2 * page * c + (gd + g) * page + 5] = 0x7FC00000  # a value of position 37
    got, want, bound, fin, own = run_attend((D, page, 1, Hq, "f16", [40, 40, 40], None, 40, 0, 0), edit=edit)
    got, want = got.reshape(3, 40, Hq, D), want.reshape(3, 40, Hq, D)
    assert (got[0] == 0).all()
    for b, first in ((1, 19), (2, 37)):
        assert np.isnan(got[b, first:]).all() and np.isfinite(got[b, :first]).all()


def test_attend_past_the_page_table():
    """lengths past W * page: rows see what the table reaches; capacity and window apart."""
    for window in (0, 30):
        case = (128, 16, 1, 4, "bf16", [100, 2 ** 31 - 1], None, 3, window, 4)
        D, page, H, Hq, fmt, lengths, _, n, _, sinks = case
        rng = np.random.default_rng(5)
        pages, table = make_pool(rng, [100, 100], page, H, D, W=4)
        q = torch.from_numpy(rng.standard_normal((6, Hq, D)).astype(np.float32)).to(torch.bfloat16)
        got = out_f64(qg.attend_kv_u4_pages(q.to(DEV), dev(pages), dev(table), dev(np.array(lengths, np.int32)), window=window, sinks=sinks))
        k, v, there = kv4.values(pages, page, table[0], np.arange(64), D)
        for r in range(3):
            seen = kv4.visible([97 + r], 64, there, window, sinks)
            want, _ = kv4.attend(q[r:r + 1].double().numpy(), k, v, seen, D ** -0.5)
            assert np.linalg.norm(got[r] - want[0]) <= (2.0 ** -8 + 2.0 ** -10) * np.linalg.norm(want[0])
        k, v, there = kv4.values(pages, page, table[1], np.arange(64), D)
        seen = there[None] & (np.arange(64)[None] < (sinks if window else 64))
        for r in range(3, 6):
            want, _ = kv4.attend(q[r:r + 1].double().numpy(), k, v, seen, D ** -0.5)
            assert np.linalg.norm(got[r] - want[0]) <= (2.0 ** -8 + 2.0 ** -10) * np.linalg.norm(want[0])


@pytest.mark.parametrize("n", [1, 80])
def test_no_pages(n):
    """An empty pool, and an empty page table: nothing is stored, seen or read back."""
    D, H = 128, 2
    for P, W in ((0, 3), (2, 0)):
        pages = qg.kv_u4_pages(P, H, 32, D)
        table, lengths = torch.zeros((1, W), dtype=torch.int32, device=DEV), torch.tensor([96], dtype=torch.int32, device=DEV)
        x = torch.randn((n, 4 * H, D), device=DEV).half()
        q, k, v = x.split([2 * H, H, H], 1)
        got = qg.append_kv_u4_pages(k, v, pages, table, lengths, q=q)
        assert torch.equal(got, q) and (pages == 0).all()
        assert (qg.attend_kv_u4_pages(got, pages, table, lengths) == 0).all()
        for x in qg.dequantize_kv_u4_pages(pages, table, lengths, n, D):
            assert (x == 0).all()
