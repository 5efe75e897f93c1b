"""Pins of the e4m3 and routing oracles on the CPU: the code table against
torch's e4m3 type, rounding against brute force over all codes, the quantizers'
invariants, routing and plans against hand-worked cases and torch."""
import numpy as np
import pytest
import torch

from oracle import experts as oe
from oracle import f8


def test_code_table_matches_the_torch_type():
    t = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    v = f8.f8_values()
    assert np.array_equal(np.isnan(t), np.isnan(v))
    assert np.array_equal(t[~np.isnan(t)], v[~np.isnan(v)])
    assert v[0x7e] == 448.0 and v[1] == 2.0 ** -9


def test_encode_is_the_nearest_code_halves_to_even():
    v = f8.f8_values()[:127]
    mid = (v[:-1] + v[1:]) / 2                      # every tie
    even = np.where(np.arange(126) % 2 == 0, np.arange(126), np.arange(1, 127))
    assert np.array_equal(f8.f8_encode(mid), even.astype(np.uint8))
    assert np.array_equal(f8.f8_encode(np.nextafter(mid, 0)), np.arange(126).astype(np.uint8))
    assert np.array_equal(f8.f8_encode(np.nextafter(mid, 1e9)), np.arange(1, 127).astype(np.uint8))
    x = (np.random.default_rng(0).standard_normal(20000) * 100).clip(-448, 448).astype(np.float32)
    t = torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(f8.f8_encode(x), t)


@pytest.mark.parametrize("K", [16, 128, 144, 272])
def test_quantizer_invariants(K):
    rng = np.random.default_rng(K)
    x = (rng.standard_normal((5, K)) * np.exp(rng.standard_normal((5, 1)) * 4)).astype(np.float32)
    x[2] = 0
    q, s = f8.quantize_f8_g128(x)
    back = f8.f8_decode(q)
    for g in range(f8.blocks(K)):
        at = slice(128 * g, 128 * g + 128)
        assert np.all(np.abs(back[:, at]).max(1)[s[:, g] > 0] == 448)
        sc = s[:, g, None].astype(np.float64)
        # half a step of the code (2^-4 of a normal value, 2^-10 below), and
        # the binary32 rounding of the quotient
        step = np.maximum(np.abs(x[:, at]) * 2.0 ** -4, sc * 2.0 ** -10) * (1 + 2.0 ** -20)
        assert np.all(np.abs(back[:, at] * sc - x[:, at]) <= step + 1e-300)
    assert np.all(q[2] == 0) and np.all(s[2] == 0)


def test_weight_blocks_are_the_activation_rule_over_a_block():
    rng = np.random.default_rng(1)
    w = rng.standard_normal((144, 150)).astype(np.float32)
    q, s = f8.quantize_weight_f8_b128(w)
    assert q.shape == (150, 144) and s.shape == (2, 2)
    for b in range(2):
        for g in range(2):
            blk = w.T[128 * b:128 * b + 128, 128 * g:128 * g + 128]
            flat = blk.reshape(1, -1)
            sc = np.float32(np.abs(flat).max() / np.float32(448))
            assert s[b, g] == sc
            assert np.array_equal(q[128 * b:128 * b + 128, 128 * g:128 * g + 128],
                                  f8.f8_encode((blk / sc).clip(-448, 448)))


def test_subnormal_scale_is_clamped():
    x = np.zeros((1, 16), np.float32)
    x[0, 0] = np.float32(700 * 2.0 ** -149)       # s = 2 * 2^-149, quotient 350
    x[0, 1] = np.float32(-600 * 2.0 ** -149)
    q, s = f8.quantize_f8_g128(x)
    assert s[0, 0] == np.float32(2 * 2.0 ** -149) and f8.f8_decode(q)[0, 0] == 352
    x[0, 0] = np.float32(671 * 2.0 ** -149)       # s = 2^-149 (671 / 448 rounds to 1): 671 > 448
    q, s = f8.quantize_f8_g128(x)
    assert s[0, 0] == np.float32(2.0 ** -149) and f8.f8_decode(q)[0, 0] == 448 and f8.f8_decode(q)[0, 1] == -448


def test_product_matches_the_dequantized_matmul():
    rng = np.random.default_rng(2)
    xq, xs = f8.quantize_f8_g128(rng.standard_normal((3, 272)).astype(np.float32))
    wq, ws = f8.quantize_weight_f8_b128(rng.standard_normal((272, 130)).astype(np.float32))
    y, B, D = f8.gemm_f8_b128(xq, xs, wq, ws)
    x = f8.f8_decode(xq) * np.repeat(xs.astype(np.float64), 128, 1)[:, :272]
    w = f8.f8_decode(wq) * np.repeat(np.repeat(ws.astype(np.float64), 128, 0)[:130], 128, 1)[:, :272]
    assert np.allclose(y, x @ w.T, rtol=1e-12, atol=1e-12 * B.max())
    assert np.allclose(B, np.abs(x) @ np.abs(w).T, rtol=1e-12)
    assert np.all(D <= B) and np.all(8 * D >= B * (1 - 1e-12))


def test_route_worked_case():
    # sigmoid is monotone: choices follow logits + bias order; group values are
    # sums of the two largest
    lg = np.array([[2.0, 1.0, 1.5, -np.inf, 3.0, -9.0, 0.0, 0.0]], np.float32)
    e, w = oe.route_experts(lg, 2, sigmoid=True)
    assert e.tolist() == [[4, 0]]
    s = 1 / (1 + np.exp(-np.array([3.0, 2.0])))
    assert np.allclose(w, s / s.sum())
    # groups (2,1) (1.5,closed) (3,-9) (0,0): sums 1.612 0.818 0.953 1.0
    e, _ = oe.route_experts(lg, 2, sigmoid=True, groups=4, top_groups=2)
    assert e.tolist() == [[0, 1]]
    e, w = oe.route_experts(np.full((2, 4), -np.inf, np.float32), 3)
    assert e.tolist() == [[-1] * 3] * 2 and not w.any()
    e, _ = oe.route_experts(np.zeros((1, 6), np.float32), 3)
    assert e.tolist() == [[0, 1, 2]]              # ties to the lowest


@pytest.mark.parametrize("sigmoid", [False, True])
def test_route_matches_torch(sigmoid):
    rng = np.random.default_rng(3)
    lg = rng.standard_normal((20, 24)).astype(np.float32)
    e, w = oe.route_experts(lg, 4, sigmoid=sigmoid, renormalize=False, scale=2.0)
    p = torch.from_numpy(lg).double()
    p = torch.sigmoid(p) if sigmoid else torch.softmax(p, 1)
    v, i = p.topk(4, 1)
    assert np.array_equal(e, i.numpy()) and np.allclose(w, 2 * v.numpy(), rtol=1e-12)


def test_plan_and_combine_worked_case():
    e = np.array([[2, 0], [0, -1], [5, 2]], np.int32)
    off, tok, slot = oe.plan_experts(e, 3)
    assert off.tolist() == [0, 2, 2, 4] and tok.tolist() == [0, 1, 0, 2, -1, -1]
    assert slot.tolist() == [[2, 0], [1, -1], [-1, 3]]
    rows = np.arange(8, dtype=np.float32).reshape(4, 2)
    y, _ = oe.combine_experts(rows, slot, np.array([[1, 2], [3, 4], [5, 6]], np.float32))
    assert y.tolist() == [[4, 5 + 2], [6, 9], [36, 42]]
