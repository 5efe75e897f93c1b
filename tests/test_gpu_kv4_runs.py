"""The 4-bit paged cache as it is used: projections, appending, attention and
reading back in a row; long calls against short ones; captured and on other
streams; pools past 32-bit offsets; scores far apart."""
import numpy as np
import pytest
import torch

import bit_quantized_gemm_int8_amd as qg
import oracle.kv4 as kv4
from tests.gpu_util import DEV, out_f64
from tests.kv4_util import attend_case, make_pool
from tests.test_gpu_kv4 import DT, check_attend, dev, host_pages, run_attend, tables

pytestmark = pytest.mark.gpu


def i32(a):
    return torch.tensor(np.array(a, np.int64).astype(np.int32), device=DEV)


# ---- calls of many rows, which take four positions at a time, against calls of few ----

# D, page, H, Hq, dtype, rotated channels, interleaved, angles of this many positions
LONG = [
    (128, 64, 8, 8, "bf16", 128, False, 10000),
    (128, 16, 8, 8, "f16", 64, True, 2202),
    (64, 32, 9, 30, "f32", 64, False, 1999),
    (256, 16, 4, 0, "f16", 256, False, 10000),
    (256, 256, 3, 6, "bf16", 128, True, 2001),
    (64, 128, 16, 17, "bf16", 0, False, 0),
]


@pytest.mark.parametrize("case", LONG, ids=range(len(LONG)))
def test_many_rows_as_few(case):
    D, page, H, Hq, fmt, rot, inter, angles = case
    rng = np.random.default_rng(page + H)
    # sequences that begin and end anywhere, one of a single row, one of none, one whose first positions are below zero
    lengths = [2203, 900, 77, 5, 1300, 300]
    offsets = [3, 2003, 2004, 2081, 2081, 3302, 3602]
    lengths[5] = 290
    T = 4099
    pages, table = make_pool(rng, lengths, page, H, D, fill=False)
    table[4, 1] = -1
    table[0, -1] = pages.shape[0]
    x = torch.from_numpy((rng.standard_normal((T, Hq + 2 * H, D)) * np.exp(rng.standard_normal((T, Hq + 2 * H, 1)))).astype(np.float32)).to(DT[fmt])
    x[40, -1, 5] = float("nan")
    x[41, -2, 5] = float("inf")
    x[42, -1] = 0
    q, k, v = x.to(DEV).split([Hq, H, H], 1)
    cos, sin = (dev(t) for t in tables(rng, angles, rot)) if rot else (None, None)
    print(f"many rows {case}", flush=True)
    want, got = dev(pages), dev(pages)
    turned = torch.full((2, T, Hq, D), 7.0, dtype=DT[fmt], device=DEV)

    def part(r0, r1):
        """lengths and offsets of rows r0 .. r1 - 1 alone."""
        o = np.clip(offsets, r0, r1)
        return i32(np.array(lengths) - (np.array(offsets[1:]) - o[1:])), i32(o - r0)

    def append(to, y, r0, r1):
        n, o = part(r0, r1)
        qg.append_kv_u4_pages(k[r0:r1], v[r0:r1], to, dev(table), n, offsets=o, q=q[r0:r1] if Hq else None, cos=cos, sin=sin,
                              interleaved=inter, out=y[r0:r1] if Hq else None)
    append(got, turned[0], 0, T)
    for r0 in range(0, T, 301):
        append(want, turned[1], r0, min(r0 + 301, T))
    assert torch.equal(got, want)
    assert (want != 0).any()
    assert torch.equal(turned[0].nan_to_num(9), turned[1].nan_to_num(9))
    assert (turned[0][:3] == 7).all() and (turned[0][3602:] == 7).all()
    for out in ("f32", fmt):
        whole = [torch.full((T, H, D), 5.0, dtype=DT[out], device=DEV) for _ in range(2)]
        parts = [torch.full((T, H, D), 5.0, dtype=DT[out], device=DEV) for _ in range(2)]
        n, o = part(0, T)
        qg.dequantize_kv_u4_pages(got, dev(table), n, T, D, offsets=o, out_dtype=DT[out], out=whole)
        for r0 in range(0, T, 301):
            r1 = min(r0 + 301, T)
            n, o = part(r0, r1)
            qg.dequantize_kv_u4_pages(got, dev(table), n, r1 - r0, D, offsets=o, out_dtype=DT[out], out=[t[r0:r1] for t in parts])
        for a, b in zip(whole, parts):
            assert torch.equal(a.nan_to_num(9), b.nan_to_num(9))
            assert (a[:3] == 5).all() and (a[3602:] == 5).all() and not (a[3:3602] == 5).all()


# ---- attention: kernels and splits that the other tests do not reach ----------------

MORE = [
    # rows of few and of many tokens in one kernel: the sight is short
    (128, 64, 2, 4, "f16", [700, 300, 40], [0, 600, 601, 603], 0, 100, 4),
    (64, 16, 3, 6, "bf16", [0, 500, 1, 260], [2, 2, 400, 401, 441], 0, 0, 0),
    (128, 32, 1, 8, "bf16", [3, 1000], [1, 5, 100], 0, 64, 0),
    # and in two: the sight is long
    (128, 256, 1, 2, "bf16", [4500, 700, 33], [0, 300, 301, 304], 0, 0, 0),
    # tiles of 32 rows of the other kernel
    (128, 64, 2, 8, "f16", [300, 1000], None, 8, 0, 0),
    (64, 32, 1, 4, "bf16", [700, 50], None, 5, 60, 3),
    (128, 32, 1, 4, "bf16", [400, 90, 300], [0, 9, 10, 18], 0, 0, 0),
    (64, 16, 2, 4, "f16", [500, 40], [0, 20, 24], 0, 0, 0),
    # a workgroup of eight waves for each kv head
    (128, 64, 64, 64, "f16", [2200, 1500], None, 1, 0, 0),
    (64, 64, 256, 256, "bf16", [1100], None, 1, 0, 0),
    (64, 128, 128, 256, "f16", [1200, 300], [0, 1, 2], 0, 0, 0),
    (128, 32, 128, 128, "bf16", [2100, 2], None, 1, 1500, 3),
    # many splits of few tiles
    (128, 64, 1, 1, "f16", [4000], None, 130, 0, 0),
    (64, 128, 1, 2, "bf16", [5000], None, 70, 0, 0),
    (256, 64, 1, 1, "f16", [5000], None, 3, 0, 0),
]


@pytest.mark.parametrize("case", MORE, ids=range(len(MORE)))
def test_attend_more(case):
    check_attend(*run_attend(case))


@pytest.mark.parametrize("D,n", [(128, 1), (128, 150), (64, 150), (256, 5)])
def test_attend_short_sequences_under_a_wide_page_table(D, n):
    """Most splits of the positions are empty."""
    page, H, Hq, W, lengths = 64, 1, 2, 128, [n, 70 + n]
    rng = np.random.default_rng(D + n)
    pages, table = make_pool(rng, lengths, page, H, D, W=W)
    q = torch.from_numpy(rng.standard_normal((2 * n, Hq, D)).astype(np.float32)).half()
    assert qg.attend_kv_u4_pages_workspace_bytes(2 * n, 2, Hq, H, D, page, W) > 0
    got = qg.attend_kv_u4_pages(q.to(DEV), dev(pages), dev(table), i32(lengths))
    want, bound, own = attend_case(pages, table, lengths, page, D, q.double().numpy(), 2 * n)
    check_attend(out_f64(got), want, bound, torch.finfo(torch.float16), own)


@pytest.mark.parametrize("n", [1, 150])
def test_attend_lengths_far_past_the_page_table(n):
    """Positions near 2^31 - 1 under windows up to 2^30: the table's positions are behind
    the window, all but the first ones that stay visible."""
    D, H, page = 128, 1, 32
    rng = np.random.default_rng(n)
    pages, table = make_pool(rng, [200], page, H, D)
    q = torch.from_numpy(rng.standard_normal((n, 1, D)).astype(np.float32)).half()
    for length in (2 ** 31 - 1, 2 ** 30 + 2 ** 29):
        for window in (1, 2 ** 29, 2 ** 30):
            for sinks in (0, 3):
                got = out_f64(qg.attend_kv_u4_pages(q.to(DEV), dev(pages), dev(table), i32([length]), window=window, sinks=sinks))
                k, v, _ = kv4.values(pages, page, table[0], np.arange(3), D)
                want, _ = kv4.attend(q.double().numpy(), k, v, np.tile(np.arange(3) < sinks, (n, 1)), D ** -0.5)
                assert np.linalg.norm(got - want) <= (2.0 ** -11 + 2.0 ** -10) * np.linalg.norm(want)


@pytest.mark.parametrize("D,H,Hq,n", [(64, 1, 1024, 1), (128, 1, 300, 1), (128, 512, 512, 1), (256, 1, 130, 2)])
def test_attend_many_heads(D, H, Hq, n):
    """Rows that are nearly all heads of one token, and many kv heads."""
    check_attend(*run_attend((D, 16, H, Hq, "bf16", [45, 20], None, n, 0, 0)))


@pytest.mark.parametrize("D,G", [(64, 1), (128, 5), (256, 2)])
def test_many_ragged_sequences(D, G):
    """150 sequences, of no rows, one, a few, and some of many."""
    rng = np.random.default_rng(D + G)
    B, H, page = 150, 1, 16
    counts = rng.integers(0, 3, B)
    counts[[0, 63, 64, 100, 149]] = [0, 40, 150, 33, 0]
    offsets = np.concatenate([[2], 2 + np.cumsum(counts)])
    lengths = counts + rng.integers(0, 60, B)
    T = int(offsets[-1]) + 3
    pages, table = make_pool(rng, lengths, page, H, D, fill=False)
    x = torch.from_numpy(rng.standard_normal((T, (G + 2) * H, D)).astype(np.float32)).half()
    pd, td, ld, od = dev(pages), dev(table), i32(lengths), i32(offsets)
    old = torch.from_numpy(rng.standard_normal((int(lengths.sum()), 2 * H, D)).astype(np.float32)).half()
    ends = np.concatenate([[0], np.cumsum(lengths)])
    qg.append_kv_u4_pages(*old.to(DEV).split(H, 1), pd, td, ld, offsets=i32(ends))          # all positions
    q = x[:, :G * H]
    qg.append_kv_u4_pages(*x[:, G * H:].to(DEV).split(H, 1), pd, td, ld, offsets=od)        # and the last ones again
    for kv, w, o in ((old, kv4.rows(len(old), B, lengths, ends), 0), (x, kv4.rows(T, B, lengths, offsets), G * H)):
        a = kv.float().numpy()
        kv4.append(pages, page, w, table, a[:, o:o + H], a[:, o + H:])
    np.testing.assert_array_equal(host_pages(pd), pages)
    print(f"ragged {D} {G}", flush=True)
    out = torch.full((T, G * H, D), 3.0, dtype=torch.float16, device=DEV)
    qg.attend_kv_u4_pages(q.to(DEV), pd, td, ld, offsets=od, out=out)
    want, bound, own = attend_case(pages, table, lengths, page, D, q.double().numpy(), T, offsets)
    want[~own] = 3.0
    check_attend(out_f64(out), want, bound, torch.finfo(torch.float16), own)


def geometric(D, page, L, first, ratio, rising):
    """A cache whose position t scores first * ratio^t (rising) or the same from the
    other end, for queries of ones, up to the scales' rounding: keys of one value each
    have codes of 15 or 0, and scales a 64th too large at most."""
    t = np.arange(L) if rising else L - 1 - np.arange(L)
    k = np.repeat((first / D * ratio ** t.astype(np.float64)).astype(np.float32)[:, None, None], D, 2)
    v = np.random.default_rng(3).standard_normal((L, 1, D)).astype(np.float32)
    P = -(-L // page)
    pages, table = np.zeros((P, 1, kv4.page_words(page, D)), np.uint32), np.arange(P, dtype=np.int32)[None]
    kv4.append(pages, page, [(0, i) for i in range(L)], table, k, v)
    return pages, table


@pytest.mark.parametrize("rising", [True, False])
@pytest.mark.parametrize("D,n", [(64, 3), (128, 3), (256, 3), (64, 70), (128, 70)])
def test_attend_scores_in_the_millions(D, n, rising):
    """Scores from 1e3 to 3e6, each a tenth off the last: one position decides, for
    each row its own (the largest so far changes with every position) or the first.
    The others' weights are below exp(-80).  The weight is rounded once, by 2^-11, and
    so is the output."""
    L, page = 85, 32
    pages, table = geometric(D, page, L, 1000.0, 1.1, rising)
    q = torch.ones((n, 2, D), device=DEV, dtype=torch.float16)
    print(f"scores {D} {n} {rising}", flush=True)
    got = out_f64(qg.attend_kv_u4_pages(q, dev(pages), dev(table), i32([L]), scale=1.0))
    torch.cuda.synchronize()
    _, v, _ = kv4.values(pages, page, table[0], np.arange(L), D)
    for r in range(n):
        t = L - n + r if rising else 0
        want = np.repeat(v[t], 2, 0)
        assert (np.abs(got[r] - want) <= (2.0 ** -11 + 2.0 ** -11 + 2.0 ** -20) * np.abs(want) + 2.0 ** -24).all(), (r, t)


def test_scale_of_zero_is_a_mean():
    case = (128, 32, 1, 2, "f16", [77], None, 5, 0, 0)
    check_attend(*run_attend(case, scale=0.0))


# ---- views, room, sizes --------------------------------------------------------------

@pytest.mark.parametrize("T", [3, 130])
def test_views_and_workspaces(T):
    D, H, Hq, page = 128, 2, 4, 32
    rng = np.random.default_rng(T)
    pages, table = make_pool(rng, [2000 + T], page, H, D)
    x = torch.randn((T, Hq + 2 * H, D), device=DEV).half()
    q = x[:, 1:1 + Hq]
    n = i32([2000 + T])
    a = qg.attend_kv_u4_pages(q.contiguous(), dev(pages), dev(table), n)
    assert torch.equal(qg.attend_kv_u4_pages(q, dev(pages), dev(table), n), a)
    need = qg.attend_kv_u4_pages_workspace_bytes(T, 1, Hq, H, D, page, table.shape[1])
    assert need > 0
    ws = torch.full((need + 64,), 0xFF, dtype=torch.uint8, device=DEV)
    assert torch.equal(qg.attend_kv_u4_pages(q, dev(pages), dev(table), n, workspace=ws[:need]), a)
    assert (ws[need:] == 0xFF).all()
    # the rotated queries in the place of the queries
    y = q.contiguous()
    cos, sin = (dev(t) for t in tables(rng, 2200, D))
    want = qg.append_kv_u4_pages(x[:, -2 * H:-H], x[:, -H:], dev(pages), dev(table), n, q=y, cos=cos, sin=sin)
    got = qg.append_kv_u4_pages(x[:, -2 * H:-H], x[:, -H:], dev(pages), dev(table), n, q=y, cos=cos, sin=sin, out=y)
    assert got is y and torch.equal(y, want) and not torch.equal(y, q)


def test_no_rows():
    pages = qg.kv_u4_pages(3, 2, 16, 64)
    table, none, x = torch.zeros((2, 3), dtype=torch.int32, device=DEV), i32([0, 0]), torch.empty((0, 2, 64), device=DEV).half()
    for offsets in (None, i32([0, 0, 0])):
        assert qg.append_kv_u4_pages(x, x, pages, table, none, offsets=offsets, q=x).shape == (0, 2, 64)
        assert qg.attend_kv_u4_pages(x, pages, table, none, offsets=offsets).shape == (0, 2, 64)
        assert qg.dequantize_kv_u4_pages(pages, table, none, 0, 64, offsets=offsets)[0].shape == (0, 2, 64)
    assert (pages == 0).all()
    no = torch.zeros((0, 3), dtype=torch.int32, device=DEV)
    assert qg.attend_kv_u4_pages(x, pages, no, i32([])).shape == (0, 2, 64)


@pytest.mark.parametrize("n", [70, 3])
def test_past_32_bit_offsets(n):
    """A pool of 9 GB and tokens 2^26 elements apart, against a small pool and tokens side by side."""
    D, H, Hq, page, P = 128, 8, 16, 256, 32768
    x = torch.randn((n, Hq + 2 * H, D), device=DEV).bfloat16()
    apart = torch.empty((n << 26,), dtype=torch.bfloat16, device=DEV).view(n, 1 << 26)[:, :x[0].numel()].unflatten(1, x.shape[1:])
    apart.copy_(x)
    big = torch.empty((P, H, qg.kv_u4_page_bytes(page, D) // 4), dtype=torch.int32, device=DEV)
    assert big.numel() > 1 << 31
    small = qg.kv_u4_pages(2, H, page, D)
    lengths = i32([200 + n])
    old = torch.randn((200, 2 * H, D), device=DEV).bfloat16()
    out = []
    for pool, t, y in ((small, i32([[0, 1]]), x), (big, i32([[P - 1, P - 3]]), apart)):
        pool[t[0].long()] = 0
        qg.append_kv_u4_pages(old[:, :H], old[:, H:], pool, t, i32([200]))
        q = qg.append_kv_u4_pages(y[:, Hq:Hq + H], y[:, Hq + H:], pool, t, lengths, q=y[:, :Hq])
        out.append([pool[t[0].long()], q, qg.attend_kv_u4_pages(y[:, :Hq], pool, t, lengths),
                    *qg.dequantize_kv_u4_pages(pool, t, lengths, 200 + n, D)])
    for a, b in zip(*out):
        assert torch.equal(a, b)


# ---- layers --------------------------------------------------------------------------

class Layer:
    """Projection to q, k, v with 4-bit weights, cache, attention, and its way out."""

    def __init__(self, D, H, Hq, page, P, seed, B=3, W=24):
        g = torch.Generator().manual_seed(seed)
        self.D, self.H, self.Hq, self.page, self.K = D, H, Hq, page, 256
        self.qkv = qg.quantize_weight_u4_g128((torch.randn((self.K, (Hq + 2 * H) * D), generator=g) / 16).to(DEV))
        self.back = qg.quantize_weight_u4_g128((torch.randn((Hq * D, self.K), generator=g) / 16).to(DEV))
        self.pages = qg.kv_u4_pages(P, H, page, D)
        self.table = torch.randperm(P, generator=g)[:B * W].reshape(B, W).int().to(DEV)
        rng = np.random.default_rng(seed)
        self.np_angles = tables(rng, W * page, D)
        self.cos, self.sin = (dev(t) for t in self.np_angles)

    def step(self, x, lengths, offsets=None, **kw):
        """x f16 [T, K] -> what the layer puts out, and what it made on the way."""
        y = qg.gemm_w4a16_g128(x, *self.qkv).unflatten(1, (-1, self.D))
        q, k, v = y.split([self.Hq, self.H, self.H], 1)
        q = qg.append_kv_u4_pages(k, v, self.pages, self.table, lengths, offsets=offsets, q=q, cos=self.cos, sin=self.sin)
        o = qg.attend_kv_u4_pages(q, self.pages, self.table, lengths, offsets=offsets, **kw)
        return qg.gemm_w4a16_g128(o.flatten(1), *self.back), y, q, o


@pytest.mark.parametrize("D,H,Hq,page", [(128, 2, 4, 16), (64, 1, 8, 32), (256, 1, 2, 64)])
def test_layer_over_a_generation(D, H, Hq, page):
    """Prompts of three requests, a chunk beside single tokens, drafts, single tokens
    under a window: pages bit for bit, attention and the values read back."""
    W = 24
    layer = Layer(D, H, Hq, page, 3 * W + 2, seed=D, W=W)
    table = layer.table.cpu().numpy()
    pages = host_pages(layer.pages).copy()
    have = np.zeros(3, int)
    rng = np.random.default_rng(D)
    for counts, kw in (([150, 9, 33], {}), ([1, 70, 1], {}), ([4, 4, 4], {}), ([1, 1, 1], dict(window=40, sinks=4)), ([1, 1, 1], {}), ([1, 0, 1], {})):
        offsets = np.concatenate([[0], np.cumsum(counts)])
        have += counts
        T = int(offsets[-1])
        same = len(set(counts)) == 1
        x = torch.from_numpy(rng.standard_normal((T, layer.K)).astype(np.float32)).half().to(DEV)
        print(f"layer {D} {counts} {kw}", flush=True)
        z, y, q, o = layer.step(x, i32(have), None if same else i32(offsets), **kw)
        torch.cuda.synchronize()
        assert torch.isfinite(z).all() and (z != 0).any()
        where = kv4.rows(T, 3, have, offsets)
        pos = np.array([p for _, p in where])
        yn = y.float().cpu().numpy()
        turn = [kv4.rotate(a, pos, *layer.np_angles, False) for a in (yn[:, :Hq], yn[:, Hq:Hq + H])]
        kv4.append(pages, page, where, table, turn[1], yn[:, Hq + H:])
        np.testing.assert_array_equal(host_pages(layer.pages), pages)
        np.testing.assert_array_equal(out_f64(q), torch.from_numpy(turn[0]).half().double().numpy())
        want, bound, own = attend_case(pages, table, have, page, D, out_f64(q), T, offsets, kw.get("window", 0), kw.get("sinks", 0))
        check_attend(out_f64(o), want, bound, torch.finfo(torch.float16), own)
    # all of it read back
    ends = np.concatenate([[0], np.cumsum(have)])
    k, v = qg.dequantize_kv_u4_pages(layer.pages, layer.table, i32(have), int(ends[-1]), D, offsets=i32(ends), out_dtype=torch.float32)
    for b in range(3):
        wk, wv, _ = kv4.values(pages, page, table[b], np.arange(have[b]), D)
        np.testing.assert_array_equal(out_f64(k[ends[b]:ends[b + 1]]), wk)
        np.testing.assert_array_equal(out_f64(v[ends[b]:ends[b + 1]]), wv)


@pytest.mark.parametrize("D,n", [(128, 1), (64, 50), (256, 2)])
def test_layer_captured_and_replayed(D, n):
    """A step in a graph: each replay takes the next tokens, at positions that the graph
    itself moves on, and gives what the eager step gives."""
    a, b = (Layer(D, 1, 4, 32, 80, seed=1) for _ in range(2))
    x = torch.randn((3 * n, a.K), device=DEV).half()
    la, lb = i32([300, 20, 0]), i32([300, 20, 0])
    old = torch.randn((600, 2, D), device=DEV).half()
    for l in (a, b):
        qg.append_kv_u4_pages(old[:, :1], old[:, 1:], l.pages, l.table, la, offsets=i32([0, 300, 320, 320]))
    b.step(x, i32([n, n, n]))          # weights and kernels are there; these positions are written again below
    b.pages.copy_(a.pages)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        lb += n
        out = b.step(x, lb)
        back = qg.dequantize_kv_u4_pages(b.pages, b.table, lb, 3 * n, D)
    for i in range(4):
        la += n
        want = a.step(x, la)
        read = qg.dequantize_kv_u4_pages(a.pages, a.table, la, 3 * n, D)
        g.replay()
        torch.cuda.synchronize()
        for u, w in zip(out + back, want + read):
            assert torch.equal(u, w)
        assert torch.equal(a.pages, b.pages)
        x.copy_(torch.randn_like(x))
        torch.randn((256, 256), device=DEV) @ torch.randn((256, 256), device=DEV)
        torch.cuda.synchronize()


def test_two_graphs_with_one_workspace():
    """Two captured calls whose workspace is the same tensor, replayed in turn."""
    rng = np.random.default_rng(4)
    D, H, Hq, page = 128, 2, 4, 64
    pages, table = make_pool(rng, [3000], page, H, D)
    pages, table = dev(pages), dev(table)
    calls = []
    size = max(qg.attend_kv_u4_pages_workspace_bytes(n, 1, Hq, H, D, page, table.shape[1]) for n in (1, 200))
    ws = torch.empty(size, dtype=torch.uint8, device=DEV)
    for n in (1, 200):
        q, lengths = torch.randn((n, Hq, D), device=DEV).half(), i32([3000])
        want = qg.attend_kv_u4_pages(q, pages, table, lengths)
        out = torch.zeros_like(q)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            qg.attend_kv_u4_pages(q, pages, table, lengths, out=out, workspace=ws)
        calls.append((g, out, want, q, lengths))
    for _ in range(3):
        for g, out, want, *_ in calls:
            out.zero_()
            g.replay()
        torch.cuda.synchronize()
        for g, out, want, *_ in calls:
            assert torch.equal(out, want)


def test_two_streams():
    """Steps on two streams at once, caches and workspaces apart, against the same on one."""
    x = [torch.randn((3, 256), device=DEV).half() for _ in range(2)]
    old = torch.randn((6000, 2, 128), device=DEV).half()

    def run(apart):
        layers = [Layer(128, 1, 8, 128, 60, seed=i, W=17) for i in range(2)]
        lengths = [i32([2000, 2000, 2000]) for _ in range(2)]
        for l, n in zip(layers, lengths):
            qg.append_kv_u4_pages(old[:, :1], old[:, 1:], l.pages, l.table, n)
        torch.cuda.synchronize()
        streams = [torch.cuda.Stream() if apart else torch.cuda.current_stream() for _ in range(2)]
        out = [[], []]
        for _ in range(10):
            for i in range(2):
                with torch.cuda.stream(streams[i]):
                    lengths[i] += 1
                    out[i].append(layers[i].step(x[i], lengths[i])[0])
        torch.cuda.synchronize()
        return out[0] + out[1] + [l.pages for l in layers]
    for a, b in zip(run(True), run(False)):
        assert torch.equal(a, b)


# ---- refusals ------------------------------------------------------------------------

def test_refused_operands():
    D, H = 64, 2
    pages = qg.kv_u4_pages(4, H, 16, D)
    table, lengths, offsets = torch.zeros((2, 4), dtype=torch.int32, device=DEV), i32([9, 9]), i32([0, 2, 4])
    k = torch.zeros((4, H, D), device=DEV).half()
    q = torch.zeros((4, 4, D), device=DEV).half()
    cos = torch.ones((64, 32), device=DEV)

    def append(**kw):
        a = dict(k=k, v=k, pages=pages, page_table=table, lengths=lengths, offsets=offsets, q=q, cos=cos, sin=cos)
        a.update(kw)
        return qg.append_kv_u4_pages(**a)

    def attend(**kw):
        a = dict(q=q, pages=pages, page_table=table, lengths=lengths, offsets=offsets)
        a.update(kw)
        return qg.attend_kv_u4_pages(**a)

    def read(**kw):
        a = dict(pages=pages, page_table=table, lengths=lengths, T=4, D=D, offsets=offsets)
        a.update(kw)
        return qg.dequantize_kv_u4_pages(**a)
    wrong = (TypeError, ValueError, RuntimeError)
    for call in (append, attend, read):
        call()
        for kw in (dict(pages=pages.cpu()), dict(pages=pages.float()), dict(pages=pages[:, :, :-1]), dict(pages=pages[0]), dict(pages=pages[:, ::2]),
                   dict(pages=pages[:, :, :280].contiguous()), dict(page_table=table[0]), dict(page_table=table.long()),
                   dict(page_table=table[:, ::2]), dict(page_table=table.cpu()), dict(page_table=table[:1]), dict(lengths=lengths.long()),
                   dict(lengths=lengths[:1]), dict(lengths=lengths.cpu()), dict(lengths=None), dict(offsets=offsets[:2]),
                   dict(offsets=offsets.long()), dict(offsets=offsets.cpu())):
            with pytest.raises(wrong):
                call(**kw)
    for kw in (dict(k=k[:, :1]), dict(v=k[:3]), dict(v=k.float()), dict(k=k.double(), v=k.double()), dict(k=k[0], v=k[0]), dict(k=k.cpu()),
               dict(k=k.transpose(0, 1).contiguous().transpose(0, 1)), dict(k=k[:1].expand(4, H, D)), dict(q=q.float()), dict(q=q[:3]),
               dict(q=q[:, :, :32]), dict(q=q.cpu()), dict(cos=None), dict(sin=None), dict(cos=cos[:, :30]), dict(cos=cos[:, :4], sin=cos[:, :4]),
               dict(cos=cos.half()), dict(sin=cos[:32]), dict(cos=torch.ones((64, 40), device=DEV), sin=torch.ones((64, 40), device=DEV)),
               dict(out=q.float()), dict(out=q[:3]), dict(q=None, out=q), dict(out=torch.zeros((4, 8, D), device=DEV).half()[:, ::2]),
               dict(k=torch.zeros((4, H * D + 4), device=DEV).half()[:, 4:].unflatten(1, (H, D)))):
        with pytest.raises(wrong):
            append(**kw)
    for kw in (dict(q=q[:, :3]), dict(q=q.float()), dict(q=q[0]), dict(q=q[:, :0]), dict(window=-1), dict(sinks=-1), dict(scale=float("nan")),
               dict(scale=float("inf")), dict(out=q.float()), dict(out=q[:, :2]), dict(workspace=torch.zeros(64, device=DEV)),
               dict(q=q[:3], offsets=None)):
        with pytest.raises(wrong):
            attend(**kw)
    for kw in (dict(D=128), dict(D=96), dict(T=-1), dict(T=3, offsets=None), dict(out_dtype=torch.int32), dict(out=(k, k[:3])), dict(out=(k.float(), k))):
        with pytest.raises(wrong):
            read(**kw)
    long = torch.zeros((2, 4096), dtype=torch.int32, device=DEV)
    need = qg.attend_kv_u4_pages_workspace_bytes(4, 2, 4, H, D, 16, 4096, ragged=True)
    assert need > 0
    with pytest.raises(RuntimeError):
        attend(page_table=long, workspace=torch.empty(need - 1, dtype=torch.uint8, device=DEV))
    for page, d in ((8, 64), (48, 64), (16, 96), (512, 128)):
        with pytest.raises(ValueError):
            qg.kv_u4_pages(1, 1, page, d)


@pytest.mark.parametrize("n", [6, 4097])
def test_offsets_that_leave_the_call(n):
    """Offsets past the call's rows, below zero or falling: undefined rows, and nothing
    outside the buffers or the pages of the sequences."""
    D, H, page = 64, 2, 16
    rng = np.random.default_rng(n)
    pages = qg.kv_u4_pages(700, H, page, D)
    table = i32([np.arange(300), np.arange(300, 600)])
    lengths = i32([n + 90, n + 95])
    x = torch.randn((n, 4 * H, D), device=DEV).half()
    q, k, v = x.split([2 * H, H, H], 1)
    room = torch.full((3, n + 64, 2 * H, D), 3.0, dtype=torch.float16, device=DEV)
    back = torch.full((2, n + 64, H, D), 3.0, dtype=torch.float16, device=DEV)
    for offsets in ([0, n // 2, n + 9], [-8, 5, n + 2 ** 20], [0, n + 3, 2], [n, 3, 1], [-2 ** 31, 0, 2 ** 31 - 1]):
        print(f"offsets {offsets}", flush=True)
        o = i32(offsets)
        qg.append_kv_u4_pages(k, v, pages, table, lengths, offsets=o, q=q, out=room[0, :n])
        qg.attend_kv_u4_pages(q, pages, table, lengths, offsets=o, out=room[1, :n])
        qg.attend_kv_u4_pages(q, pages, table, lengths, offsets=o, window=50, out=room[2, :n])
        qg.dequantize_kv_u4_pages(pages, table, lengths, n, D, offsets=o, out_dtype=torch.float16, out=(back[0, :n], back[1, :n]))
        torch.cuda.synchronize()
        assert (room[:, n:] == 3).all() and (back[:, n:] == 3).all() and (pages[600:] == 0).all()
