"""Every kernel of the e4m3 products where its scales can go wrong: long rows of
scales that differ from stage to stage, row to row and block to block, more
tiles than workgroups, ragged runs, gathered tokens.  Each case says which
kernel it is for, and the library's own rule has to agree."""
import numpy as np
import pytest
import torch

import bit_quantized_gemm_int8_amd as qg
from oracle import f8
from tests.f8_choice import kernel
from tests.gpu_util import to_dev
from tests.test_gpu_f8 import DEV, DT, check_products, dense_f64, exact_case, f8_dev, runs

pytestmark = pytest.mark.gpu

# K = 1376: 11 scales a row, the last block of 96; 1040: 9, of 16; 2064: 17, of
# 16; 2048: 16.  N: rows of y aligned to 16 bytes, to 4 outputs, to neither.
PLAIN = [(200, 2056, 1376, "64x64 by two groups"), (130, 9000, 1040, "64x64"), (250, 10002, 2064, "64x64"),
         (300, 12288, 1376, "128x128"), (300, 12290, 1040, "128x128"), (1030, 4104, 2064, "128x128"), (515, 8196, 2048, "128x128"),
         (1024, 11008, 1376, "256x256"), (770, 12294, 1040, "256x256"), (2050, 4100, 2064, "256x256")]


def draw(rng, rows, K, N, E=None):
    """Quantized random data with outlier channels: scales of any value.  (Every
    fourth expert has the same codes, and scales of its own.)"""
    x = rng.standard_normal((rows, K)).astype(np.float32) * np.exp(rng.standard_normal((rows, 1))).astype(np.float32)
    x[:, rng.permutation(K)[:max(1, K // 100)]] *= 50
    xq, xs = f8.quantize_f8_g128(x)
    w = [rng.standard_normal((K, N)) * 0.02 * np.exp(rng.standard_normal((K, 1))) for _ in range(min(E or 1, 4))]
    wq, ws = zip(*(f8.quantize_weight_f8_b128(m.astype(np.float32)) for m in w))
    if E is None:
        return xq, xs, wq[0], ws[0]
    each = np.exp(rng.standard_normal((E, 1, 1))).astype(np.float32)
    return xq, xs, np.stack([wq[e % 4] for e in range(E)]), np.stack([ws[e % 4] for e in range(E)]) * each


@pytest.mark.parametrize("M,N,K,which", PLAIN)
def test_plain_products(M, N, K, which):
    xq, xs, wq, ws = exact_case(np.random.default_rng(M + N + K), M, N, K)
    ref = torch.from_numpy(dense_f64(xq, xs, wq, ws))
    for out in DT:
        assert kernel(M, N, out) == ("128x128" if which == "256x256" and out == "f32" else which)
        y = qg.gemm_f8_b128(f8_dev(xq), to_dev(xs), f8_dev(wq), to_dev(ws), out_dtype=DT[out])
        assert torch.equal(y.cpu(), ref.to(DT[out])), out


@pytest.mark.parametrize("out", list(DT))
@pytest.mark.parametrize("M,N,K,which", [(130, 9000, 1040, "64x64"), (300, 12288, 1376, "128x128"), (1024, 11008, 1376, "256x256")])
def test_plain_products_of_random_data(M, N, K, which, out):
    """Some rows of each tile row against the oracle."""
    assert kernel(M, N, out) == ("128x128" if which == "256x256" and out == "f32" else which)
    rng = np.random.default_rng(M)
    xq, xs, wq, ws = draw(rng, M, K, N)
    y = qg.gemm_f8_b128(f8_dev(xq), to_dev(xs), f8_dev(wq), to_dev(ws), out_dtype=DT[out])
    at = np.unique(np.concatenate([[0, M - 1], rng.integers(0, M, 6)]))
    check_products(y[at], f8.gemm_f8_b128(xq[at], xs[at], wq, ws), K, out, tile=True)


EXPERTS = [(200, 40, 520, 1376, "stream"), (300, 8, 264, 1376, "64x64 by two groups"), (1500, 40, 520, 1376, "64x64"),
           (2300, 60, 262, 1040, "64x64"), (3000, 64, 1030, 1376, "128x128"), (3000, 64, 1032, 1040, "128x128"),
           (9000, 64, 520, 2064, "128x128"), (6000, 24, 1540, 1376, "128x128")]


@pytest.mark.parametrize("kind", ["ragged", "even", "one"])
@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("R,E,N,K,which", EXPERTS)
def test_experts(R, E, N, K, which, gather, kind):
    rng = np.random.default_rng(R + E + N + K + gather)
    T = R // 3 if gather else R
    xq, xs, wq, ws = exact_case(rng, T, N, K, E)
    off = runs(rng, R, E, kind)
    token = rng.integers(0, T, R).astype(np.int32) if gather else None
    if gather:
        token[::97] = -1
    ref = torch.full((R, N), 3.0, dtype=torch.float64)
    for e in range(E):
        r = np.arange(off[e], off[e + 1])
        t = r if token is None else token[r]
        full = dense_f64(xq[t], xs[t], wq[e], ws[e])
        full[t < 0] = 0
        ref[off[e]:off[e + 1]] = torch.from_numpy(full)
    args = f8_dev(xq), to_dev(xs), f8_dev(wq), to_dev(ws), to_dev(off)
    for out in DT:
        assert kernel(R, N, out, E) == which
        y = torch.full((R, N), 3.0, dtype=DT[out], device=DEV)
        qg.gemm_f8_b128_experts(*args, row_token=None if token is None else to_dev(token), out_dtype=DT[out], out=y)
        assert torch.equal(y.cpu(), ref.to(DT[out])), out


@pytest.mark.parametrize("out", list(DT))
@pytest.mark.parametrize("R,E,N,K,which", [(1500, 40, 520, 1376, "64x64"), (3000, 64, 1032, 1376, "128x128")])
def test_experts_of_random_data(R, E, N, K, which, out):
    assert kernel(R, N, out, E) == which
    rng = np.random.default_rng(R)
    xq, xs, wq, ws = draw(rng, R, K, N, E)
    off = runs(rng, R, E, "ragged")
    y = qg.gemm_f8_b128_experts(f8_dev(xq), to_dev(xs), f8_dev(wq), to_dev(ws), to_dev(off), out_dtype=DT[out])
    for e in range(E):
        at = np.unique(np.linspace(off[e], max(off[e], off[e + 1] - 1), 3).astype(int))[: off[e + 1] - off[e]]
        if len(at):
            check_products(y[at], f8.gemm_f8_b128(xq[at], xs[at], wq[e], ws[e]), K, out, tile=True)


@pytest.mark.parametrize("M,N,K", [(130, 9000, 1040), (300, 12288, 1376), (1024, 11008, 1376)])
def test_products_repeat_themselves(M, N, K):
    """The same call gives the same bits, and so does each of its rows in
    another call of the same kernel."""
    rng = np.random.default_rng(K)
    xq, xs, wq, ws = (to_dev(a) for a in draw(rng, M, K, N))
    xq, wq = xq.view(torch.float8_e4m3fn), wq.view(torch.float8_e4m3fn)
    y = qg.gemm_f8_b128(xq, xs, wq, ws)
    for _ in range(3):
        assert torch.equal(qg.gemm_f8_b128(xq, xs, wq, ws), y)
    flipped = qg.gemm_f8_b128(xq.view(torch.uint8).flip(0).contiguous().view(torch.float8_e4m3fn), xs.flip(0).contiguous(), wq, ws)
    assert torch.equal(flipped.flip(0), y)
