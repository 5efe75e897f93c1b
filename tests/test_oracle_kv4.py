"""The oracle of the 4-bit paged cache against closed forms and brute force (CPU)."""
import numpy as np
import pytest

import oracle.kv4 as kv4
from tests.kv4_util import make_pool


def test_round_up_7_closed_forms():
    t = np.array([0.0, 1.0, 1.0 + 2.0 ** -20, 127.0, 127.5, 128.0, 2.0 ** -132, 2.0 ** -140, 3.0e38], np.float32)
    s = kv4.round_up_7(t)
    np.testing.assert_array_equal(s[:8], np.array([0, 1, 1 + 2.0 ** -6, 127, 128, 128, 2.0 ** -132, 2.0 ** -132], np.float32))
    rng = np.random.default_rng(1)
    t = np.abs(rng.standard_normal(2000) * 10.0 ** rng.integers(-30, 30, 2000)).astype(np.float32)
    s = kv4.round_up_7(t)
    assert (s >= t).all() and (s <= t.astype(np.float64) * (1 + 2.0 ** -6)).all()
    assert ((s.view(np.uint32) & 0x1FFFF) == 0).all()


def test_group_code_worked_case():
    x = np.zeros((1, 64), np.float32)
    x[0, :4] = [15.0, 7.4, 7.6, -0.4]                 # t = 15.4 / 15, s = 1.03125 = 66 / 64
    q, s, z = kv4.quantize_groups(x)
    assert s[0, 0] == 66 / 64 and z[0, 0] == 0
    np.testing.assert_array_equal(q[0, :5], [15, 7, 7, 0, 0])
    x[0, :4] = [3.0, -12.0, 1.5, -4.5]                # t = 1: s = 1, z = 12; 1.5 and -4.5 to even
    q, s, z = kv4.quantize_groups(x)
    assert s[0, 0] == 1 and z[0, 0] == 12
    np.testing.assert_array_equal(q[0, :5], [15, 0, 14, 8, 12])


@pytest.mark.parametrize("D", [64, 128, 256])
def test_values_are_near_and_exact_in_f16(D):
    rng = np.random.default_rng(D)
    x = (rng.standard_normal((300, D)) * np.exp(rng.standard_normal((300, 1)) * 2)).astype(np.float32)
    x[0] = 0
    x[1] = np.abs(x[1])
    x[2] = -np.abs(x[2])
    q, s, z = kv4.quantize_groups(x)
    w = kv4.group_width(D)
    v = (q.astype(np.float64) - np.repeat(z, w, -1)) * np.repeat(s, w, -1).astype(np.float64)
    # half a step, and half a step of zero point at the ends of the range
    assert (np.abs(v - x) <= np.repeat(s, w, -1) * (1 + 2.0 ** -20)).all()
    assert (v[0] == 0).all()
    m, e = np.frexp(v)
    assert (m * 2 ** 11 == np.rint(m * 2 ** 11)).all()


def test_not_finite_groups_are_nan():
    x = np.ones((4, 256), np.float32)
    x[0, 3], x[1, 200], x[2, 5] = np.inf, np.nan, 3e38
    x[2, 6] = -3e38                                   # a range past binary32
    q, s, z = kv4.quantize_groups(x)
    assert np.isnan(s).tolist() == [[True, False], [False, True], [True, False], [False, False]]
    assert (q[0, :128] == 0).all() and (kv4.group_words(s, z)[0, 0] == kv4.NAN_WORD)


@pytest.mark.parametrize("D,page", [(64, 16), (128, 32), (256, 64)])
def test_append_and_read_back(D, page):
    rng = np.random.default_rng(3)
    H, lengths, offsets = 2, [page + 5, 3, 2 * page], [1, 8, 10, 12]
    pages, table = make_pool(rng, lengths, page, H, D, fill=False)
    T = 13
    where = kv4.rows(T, 3, lengths, offsets)
    assert where[0] == (-1, -1) and where[12] == (-1, -1) and where[1] == (0, page - 2) and where[11] == (2, 2 * page - 1)
    k, v = (rng.standard_normal((T, H, D)).astype(np.float32) for _ in range(2))
    kv4.append(pages, page, where, table, k, v)
    w = kv4.group_width(D)
    for r, (b, pos) in enumerate(where):
        if b < 0:
            continue
        a, c, there = kv4.values(pages, page, table[b], [pos], D)
        assert there[0]
        for got, x in ((a[0], k[r]), (c[0], v[r])):
            q, s, z = kv4.quantize_groups(x)
            np.testing.assert_array_equal(got, (q - np.repeat(z, w, -1).astype(np.float64)) * np.repeat(s, w, -1))
    # the packed uint4 format: channel 8 i + j in bits 4 j
    i, slot = int(table[2, (2 * page - 1) // page]), (2 * page - 1) % page
    q, _, _ = kv4.quantize_groups(k[11])
    assert int(pages[i, 1, slot * D // 8] >> 4 & 15) == q[1, 1]


def test_rotation_is_a_rotation():
    rng = np.random.default_rng(4)
    x = rng.standard_normal((5, 2, 64)).astype(np.float32)
    angle = rng.random((9, 16))
    cos, sin = np.cos(angle).astype(np.float32), np.sin(angle).astype(np.float32)
    pos = np.array([0, 8, 3, 3, 1])
    for inter in (False, True):
        y = kv4.rotate(x, pos, cos, sin, inter)
        np.testing.assert_array_equal(y[..., 32:], x[..., 32:])
        a = x[..., 0:32:2] + 1j * x[..., 1:32:2] if inter else x[..., :16] + 1j * x[..., 16:32]
        b = y[..., 0:32:2] + 1j * y[..., 1:32:2] if inter else y[..., :16] + 1j * y[..., 16:32]
        np.testing.assert_allclose(b, a * np.exp(1j * angle[pos])[:, None], rtol=0, atol=4 * 2.0 ** -23 * 6)


def test_attend_by_brute_force():
    rng = np.random.default_rng(5)
    q, k, v = rng.standard_normal((3, 4, 64)), rng.standard_normal((6, 2, 64)), rng.standard_normal((6, 2, 64))
    there = np.array([True, True, False, True, True, True])
    seen = kv4.visible([-1, 3, 5], 6, there, 2, 1)
    assert seen.tolist() == [[False] * 6, [True, False, False, True, False, False], [True, False, False, False, True, True]]
    o, p = kv4.attend(q, k, v, seen, 0.5)
    assert (o[0] == 0).all()
    e = [np.exp(0.5 * (q[2, 3] @ k[j, 1])) for j in (0, 4, 5)]
    np.testing.assert_allclose(o[2, 3], sum(a * v[j, 1] for a, j in zip(e, (0, 4, 5))) / sum(e), rtol=1e-12)
