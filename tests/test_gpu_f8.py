"""e4m3 quantizers and products with block scales against the oracle.

Codes and scales are compared bit for bit.  Products:
  * exact data (small integers with power-of-two scales, every sum exact in
    binary32 and every product of 8 within 2^13 of the others): bit for bit,
    whatever the kernel;
  * random data: |y - y_exact| <= u |y_exact| + floor, u half a step of the
    output type.  The floor counts binary32 roundings, each at most 2^-23 of
    the magnitudes B it can touch (matrix cores may truncate): 128 sums inside
    a block, the product with the scale and the sum over the G blocks, the
    product of the two scales, up to 8 sums of partial results.  16-bit outputs
    of the tile kernel add what the 8-bit matrix cores drop: of each product
    at most 2^-13 of the largest of its 8, so 7 * 2^-13 of the sum D of those.
"""
import numpy as np
import pytest
import torch

import bit_quantized_gemm_int8_amd as qg
from oracle import f8
from tests.gpu_util import out_f64, to_dev

pytestmark = pytest.mark.gpu
DEV = "cuda"
DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
HALF_STEP = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}


def codes(t):
    return t.view(torch.uint8).cpu().numpy()


def f8_dev(a):
    return to_dev(a).view(torch.float8_e4m3fn)


def check_products(y, ref, K, out, tile):
    ye, B, D = ref
    n = 128 + 2 * f8.blocks(K) + 12
    bound = HALF_STEP[out] * np.abs(ye) + n * 2.0 ** -23 * B
    if out == "f16":
        bound += 2.0 ** -25                     # half a subnormal step
    if tile and out != "f32":
        bound += 7 * 2.0 ** -13 * D
    bad = np.abs(out_f64(y) - ye) > bound * (1 + HALF_STEP[out])
    assert not bad.any(), (np.argwhere(bad)[:4], out_f64(y)[bad][:4], ye[bad][:4], bound[bad][:4])


# ---- quantizers ----------------------------------------------------------------

@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("M,K", [(1, 16), (1, 128), (3, 144), (5, 4096), (33, 1376), (700, 272), (1, 16384)])
def test_rows_match_the_oracle(M, K, dt):
    rng = np.random.default_rng(M * 1000 + K)
    x = (rng.standard_normal((M, K)) * np.exp(3 * rng.standard_normal((M, 1)))).astype(np.float32)
    x[:, rng.integers(0, K, 2)] *= 50
    x[M // 2] = 0
    xd = torch.from_numpy(x).to(DEV).to(DT[dt])
    q, s = qg.quantize_f8_g128(xd)
    qo, so = f8.quantize_f8_g128(xd.float().cpu().numpy())
    assert np.array_equal(s.cpu().numpy().view(np.int32), so.view(np.int32))
    assert np.array_equal(codes(q), qo)


def test_rows_at_the_ends_of_binary32():
    """Ties, subnormal scales whose quotients pass 448, blocks whose scale is
    0, and the largest finite value."""
    x = np.zeros((6, 256), np.float32)
    v = f8.f8_values()[:127].astype(np.float32)
    x[0, :126] = (v[:-1] + v[1:]) / 2
    x[0, 126] = 448
    x[0, 128:254] = -x[0, :126]
    x[0, 255] = 448
    x[1, :3] = np.array([671, -600, 3], np.float32) * np.float32(2.0 ** -149)
    x[2, 5] = np.float32(200 * 2.0 ** -149)      # 200 / 448 rounds to 0
    x[3, ::3] = np.float32(3.4028234663852886e38)
    x[4, 7], x[4, 200] = np.float32(1e-37), np.float32(-1e37)
    x[5] = np.float32(-0.0)
    q, s = qg.quantize_f8_g128(to_dev(x))
    qo, so = f8.quantize_f8_g128(x)
    assert np.array_equal(s.cpu().numpy(), so)
    assert np.array_equal(f8.f8_decode(codes(q)), f8.f8_decode(qo))


@pytest.mark.parametrize("M", [2, 70])
def test_infinities_and_nan_reach_their_outputs_only(M):
    """A block with an infinity or NaN has zero codes and a scale that is not
    finite: its row's outputs are NaN, the other rows' are as ever."""
    rng = np.random.default_rng(M)
    x = rng.standard_normal((M, 272)).astype(np.float32)
    x[0, 130], x[1, 270] = -np.inf, np.nan
    q, s = qg.quantize_f8_g128(to_dev(x))
    qo, so = f8.quantize_f8_g128(x)
    assert np.array_equal(codes(q), qo) and np.array_equal(s.cpu().numpy(), so, equal_nan=True)
    assert so[0, 1] == np.inf and np.isnan(so[1, 2])
    w = rng.standard_normal((272, 40)).astype(np.float32)
    wq, ws = f8.quantize_weight_f8_b128(w)
    for out in (torch.float32, torch.bfloat16):
        y = qg.gemm_f8_b128(q, s, f8_dev(wq), to_dev(ws), out_dtype=out)
        assert y[:2].isnan().all() and y[2:].isfinite().all()
    # a NaN of any payload stays one in 16-bit outputs
    xs = s.clone()
    xs[0, 1] = torch.tensor([0x7fffffff], dtype=torch.int32).view(torch.float32)[0]
    for out in (torch.float16, torch.bfloat16):
        assert qg.gemm_f8_b128(q, xs, f8_dev(wq), to_dev(ws), out_dtype=out)[:2].isnan().all()
    w[5, 7] = np.nan
    wq, ws = qg.quantize_weight_f8_b128(to_dev(w))
    wo, wso = f8.quantize_weight_f8_b128(w)
    assert np.array_equal(codes(wq), wo) and np.array_equal(ws.cpu().numpy(), wso, equal_nan=True)


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("E,K,N", [(1, 16, 1), (1, 128, 128), (1, 144, 131), (3, 272, 260), (2, 256, 130)])
def test_weights_match_the_oracle(E, K, N, dt):
    rng = np.random.default_rng(K * 7 + N)
    w = (rng.standard_normal((E, K, N)) * 0.02).astype(np.float32)
    w[0, :128, :128] = 0 if K > 128 else w[0, :128, :128]
    wd = torch.from_numpy(w).to(DEV).to(DT[dt])
    q, s = qg.quantize_weight_f8_b128(wd)
    for e in range(E):
        qo, so = f8.quantize_weight_f8_b128(wd[e].float().cpu().numpy())
        assert np.array_equal(s[e].cpu().numpy().view(np.int32), so.view(np.int32))
        assert np.array_equal(codes(q[e]), qo)
    q2, s2 = qg.quantize_weight_f8_b128(wd[0])          # a single matrix
    assert torch.equal(q2.view(torch.uint8), q[0].view(torch.uint8)) and torch.equal(s2, s[0])


# ---- products --------------------------------------------------------------------

def exact_case(rng, M, N, K, E=None):
    """Codes of -2 .. 2 and scales 1/2 .. 2: products up to 4, their sums over
    K below 2^24 halves of 1/4, so every binary32 sum is exact."""
    lead = () if E is None else (E,)
    G, B = f8.blocks(K), f8.blocks(N)
    ints = np.array([0xc0, 0xb8, 0, 0x38, 0x40], np.uint8)       # -2 -1 0 1 2
    xq, wq = ints[rng.integers(0, 5, (M, K))], ints[rng.integers(0, 5, lead + (N, K))]
    xs = np.exp2(rng.integers(-1, 2, (M, G))).astype(np.float32)
    ws = np.exp2(rng.integers(-1, 2, lead + (B, G))).astype(np.float32)
    return xq, xs, wq, ws


def dense_f64(xq, xs, wq, ws):
    x = f8.f8_decode(xq) * np.repeat(xs.astype(np.float64), 128, 1)[:, :xq.shape[1]]
    w = f8.f8_decode(wq) * np.repeat(np.repeat(ws.astype(np.float64), 128, 0)[:wq.shape[0]], 128, 1)[:, :wq.shape[1]]
    return x @ w.T


# the stream kernel (rows up to 16, each width of its launch), every tile size,
# K and N that end inside a block, single rows and columns, rows of y that are
# aligned to 16 bytes, to 4 outputs and to neither
SHAPES = [(1, 1, 16), (1, 4096, 256), (2, 5000, 400), (7, 33, 144), (16, 131, 1376), (16, 9000, 160), (17, 260, 528),
          (31, 12300, 144), (33, 520, 1040), (64, 4100, 272), (50, 13000, 128), (65, 64, 128), (65, 130, 2064), (77, 4100, 288),
          (128, 128, 256), (200, 2052, 400), (257, 4099, 144), (300, 12288, 272), (1030, 4100, 400), (2049, 4400, 144), (2100, 4353, 656), (1024, 11008, 272)]


@pytest.mark.parametrize("out", list(DT))
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_products_of_exact_data(M, N, K, out):
    xq, xs, wq, ws = exact_case(np.random.default_rng(M + N + K), M, N, K)
    args = f8_dev(xq), to_dev(xs), f8_dev(wq), to_dev(ws)
    y = qg.gemm_f8_b128(*args, out_dtype=DT[out])
    ref = torch.from_numpy(dense_f64(xq, xs, wq, ws)).to(DT[out])
    assert torch.equal(y.cpu(), ref)
    again = torch.full_like(y, 3.0)
    assert qg.gemm_f8_b128(*args, out_dtype=DT[out], out=again) is again and torch.equal(again, y)


@pytest.mark.parametrize("out", list(DT))
@pytest.mark.parametrize("M,N,K", [(1, 200, 4096), (5, 144, 1040), (16, 260, 11008), (40, 96, 2048), (64, 130, 1376),
                                   (80, 130, 1376), (130, 260, 4096)])
def test_products_of_random_data(M, N, K, out):
    rng = np.random.default_rng(M * N + K)
    x = rng.standard_normal((M, K)).astype(np.float32)
    x[:, rng.permutation(K)[:max(1, K // 100)]] *= 50
    w = (rng.standard_normal((K, N)) * 0.02).astype(np.float32)
    xq, xs = f8.quantize_f8_g128(x)
    wq, ws = f8.quantize_weight_f8_b128(w)
    y = qg.gemm_f8_b128(f8_dev(xq), to_dev(xs), f8_dev(wq), to_dev(ws), out_dtype=DT[out])
    check_products(y, f8.gemm_f8_b128(xq, xs, wq, ws), K, out, tile=M > 16)


@pytest.mark.parametrize("M", [1, 40, 100])
def test_large_and_subnormal_codes(M):
    """Every code against every code, the largest (448) and the subnormals
    among them; binary32 outputs sum the exact products."""
    rng = np.random.default_rng(M)
    K, N = 256, 144
    pool = np.array([c for c in range(256) if c & 0x7f != 0x7f], np.uint8)
    xq, wq = pool[rng.integers(0, 254, (M, K))], pool[rng.integers(0, 254, (N, K))]
    xs = np.exp(rng.standard_normal((M, 2))).astype(np.float32)
    ws = np.exp(rng.standard_normal((2, 2))).astype(np.float32)
    for out in DT:
        if out == "f16":
            xs = xs * np.float32(2.0 ** -10)
        y = qg.gemm_f8_b128(f8_dev(xq), to_dev(xs), f8_dev(wq), to_dev(ws), out_dtype=DT[out])
        check_products(y, f8.gemm_f8_b128(xq, xs, wq, ws), K, out, tile=M > 16)


# ---- one weight matrix for each run of rows -----------------------------------------

def runs(rng, R, E, kind):
    """E + 1 offsets: even, ragged with empty experts, or all rows with one."""
    if kind == "even":
        return np.linspace(0, R, E + 1).astype(np.int32)
    if kind == "one":
        off = np.zeros(E + 1, np.int32)
        off[E // 2 + 1:] = R
        return off
    cuts = np.sort(rng.integers(0, R + 1, E - 1))
    return np.concatenate([[0], cuts, [R - R // 7]]).clip(0, R - R // 7).astype(np.int32)


@pytest.mark.parametrize("out", list(DT))
@pytest.mark.parametrize("kind", ["even", "ragged", "one"])
@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("R,E,N,K", [(1, 3, 40, 144), (24, 8, 131, 272), (96, 4, 260, 144), (160, 4, 520, 400),
                                     (300, 3, 130, 272), (1500, 9, 516, 144), (700, 1, 128, 128)])
def test_experts_of_exact_data(R, E, N, K, gather, kind, out):
    rng = np.random.default_rng(R + E + N + K + gather)
    T = max(1, R // 3) if gather else R
    xq, xs, wq, ws = exact_case(rng, T, N, K, E)
    off = runs(rng, R, E, kind)
    token = rng.integers(0, T, R).astype(np.int32) if gather else None
    if gather and R > 10:
        token[3], token[7] = -1, T                     # no such token: a row of zeros
    before = torch.full((R, N), 3.0, dtype=DT[out], device=DEV)
    y = qg.gemm_f8_b128_experts(f8_dev(xq), to_dev(xs), f8_dev(wq), to_dev(ws), to_dev(off),
                                row_token=None if token is None else to_dev(token), out_dtype=DT[out], out=before.clone())
    ref = torch.full((R, N), 3.0, dtype=DT[out])
    for e in range(E):
        r = np.arange(off[e], off[e + 1])
        t = r if token is None else token[r]
        ok = (t >= 0) & (t < T)
        full = np.zeros((len(r), N))
        full[ok] = dense_f64(xq[t[ok]], xs[t[ok]], wq[e], ws[e])
        ref[torch.from_numpy(r)] = torch.from_numpy(full).to(DT[out])
    assert torch.equal(y.cpu(), ref)


@pytest.mark.parametrize("R,E", [(40, 8), (2000, 4)])
def test_offsets_out_of_range_are_clamped(R, E):
    """Negative and too large offsets are read as 0 and R; rows that two runs
    name hold, element by element, one run's result (their workgroups write 16
    or 32 columns at a time, in any order)."""
    rng = np.random.default_rng(R)
    N, K = 64, 144
    xq, xs, wq, ws = exact_case(rng, R, N, K, E)
    args = f8_dev(xq), to_dev(xs), f8_dev(wq), to_dev(ws)
    off = np.full(E + 1, 2 ** 31 - 1, np.int32)
    off[0], off[1], off[2] = -5, R // 4, R // 8
    out = torch.full((R, N), 3.0, device=DEV)
    y = qg.gemm_f8_b128_experts(*args, to_dev(off), out_dtype=torch.float32, out=out).cpu()
    for r in range(0, R, 7):
        named = [e for e in range(E) if min(max(off[e], 0), R) <= r < min(max(off[e + 1], 0), R)]
        got = y[r].numpy()
        if not named:
            assert np.all(got == 3.0)
        else:
            each = [dense_f64(xq[r:r + 1], xs[r:r + 1], wq[e], ws[e])[0].astype(np.float32) for e in named]
            assert np.all(np.any([got == v for v in each], axis=0))


def test_empty_calls():
    e8 = torch.empty((0, 128), device=DEV).to(torch.float8_e4m3fn)
    w8 = torch.zeros((2, 16, 128), device=DEV).to(torch.float8_e4m3fn)
    s0, s1 = torch.empty((0, 1), device=DEV), torch.ones((2, 1, 1), device=DEV)
    assert qg.quantize_f8_g128(torch.empty((0, 128), device=DEV))[0].shape == (0, 128)
    assert qg.gemm_f8_b128(e8, s0, w8[0], s1[0]).shape == (0, 16)
    off = torch.zeros(3, dtype=torch.int32, device=DEV)
    assert qg.gemm_f8_b128_experts(e8, s0, w8, s1, off).shape == (0, 16)
    # rows but no run names one
    x8, s = torch.zeros((5, 128), device=DEV).to(torch.float8_e4m3fn), torch.ones((5, 1), device=DEV)
    y = torch.full((5, 16), 2.0, dtype=torch.bfloat16, device=DEV)
    qg.gemm_f8_b128_experts(x8, s, w8, s1, off, out=y)
    assert torch.all(y == 2.0)


def test_refused_operands():
    x8, s = torch.zeros((4, 256), device=DEV).to(torch.float8_e4m3fn), torch.ones((4, 2), device=DEV)
    w8, ws = torch.zeros((32, 256), device=DEV).to(torch.float8_e4m3fn), torch.ones((1, 2), device=DEV)
    off = torch.tensor([0, 4], dtype=torch.int32, device=DEV)
    with pytest.raises(ValueError):
        qg.gemm_f8_b128(x8, s[:, :1].contiguous(), w8, ws)
    with pytest.raises(ValueError):
        qg.gemm_f8_b128(x8, s, w8, ws.t().contiguous())
    with pytest.raises(TypeError):
        qg.gemm_f8_b128(x8.view(torch.int8), s, w8, ws)
    with pytest.raises(TypeError):
        qg.gemm_f8_b128(x8, s, w8, ws, out_dtype=torch.int32)
    with pytest.raises(ValueError):
        qg.gemm_f8_b128(x8, s, w8, ws, out=torch.empty((4, 32), device=DEV))
    with pytest.raises(ValueError):
        qg.gemm_f8_b128_experts(x8, s, w8, ws, off)
    with pytest.raises(ValueError):
        qg.gemm_f8_b128_experts(x8, s, w8[None], ws[None], off[:1].contiguous())
    with pytest.raises(TypeError):
        qg.gemm_f8_b128_experts(x8, s, w8[None], ws[None], off, row_token=off.long())
    with pytest.raises(ValueError):
        qg.quantize_f8_g128(torch.zeros((4, 256), device=DEV)[:, ::2])
    with pytest.raises(RuntimeError):
        qg.quantize_f8_g128(torch.zeros((4, 24), device=DEV))            # K % 16
    with pytest.raises(TypeError):
        qg.quantize_f8_g128(torch.zeros((4, 32), dtype=torch.float64, device=DEV))
