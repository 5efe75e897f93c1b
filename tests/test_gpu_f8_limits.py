"""Sizes whose offsets pass 31 or 32 bits: the far rows and experts hold what a
small call on them gives, bit for bit."""
import pytest
import torch

import bit_quantized_gemm_int8_amd as qg

pytestmark = pytest.mark.gpu
DEV = "cuda"
F8 = torch.float8_e4m3fn


def small_codes(shape, gen):
    """Codes -2 .. 2: sums of a few thousand products are exact in binary32."""
    ints = torch.tensor([0xc0, 0xb8, 0, 0x38, 0x40], dtype=torch.uint8, device=DEV)
    return ints[torch.randint(0, 5, shape, generator=gen, device=DEV)].view(F8)


def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def rows(q, at):
    return q.view(torch.uint8)[at].view(F8)


def test_quantize_rows_beyond_32_bits():
    M, K = 270000, 16384                              # 4.4e9 inputs
    x = torch.zeros((M, K), dtype=torch.bfloat16, device=DEV)
    x[-3:] = torch.randn((3, K), generator=gen(0), device=DEV).bfloat16()
    q, s = qg.quantize_f8_g128(x)
    qs, ss = qg.quantize_f8_g128(x[-3:].contiguous())
    assert torch.equal(q[-3:].view(torch.uint8), qs.view(torch.uint8)) and torch.equal(s[-3:], ss)
    assert not q[:-3][::1000].view(torch.uint8).any() and not s[:-3].any()


def test_product_rows_beyond_31_bits():
    g, M, N, K = gen(1), 524300, 4112, 144            # 2.16e9 outputs
    xq, xs = small_codes((M, K), g), torch.ones((M, 2), device=DEV)
    wq, ws = small_codes((N, K), g), torch.ones((33, 2), device=DEV)
    y = qg.gemm_f8_b128(xq, xs, wq, ws)
    for at in (slice(0, 5), slice(M // 2, M // 2 + 5), slice(M - 5, M)):
        assert torch.equal(y[at], qg.gemm_f8_b128(rows(xq, at), xs[at], wq, ws))
    # the same rows as an expert's, and the weighted sum of far ones
    off = torch.tensor([0, M - 3, M], dtype=torch.int32, device=DEV)
    w2, s2 = torch.stack([wq.view(torch.uint8), wq.view(torch.uint8).flip(0)]).view(F8), torch.stack([ws, ws])
    z = qg.gemm_f8_b128_experts(xq, xs, w2, s2, off)
    at = slice(M - 5, M)
    assert torch.equal(z[M - 5:M - 3], y[M - 5:M - 3])
    assert torch.equal(z[M - 3:], qg.gemm_f8_b128(rows(xq, slice(M - 3, M)), xs[:3], w2[1], ws))
    slot = torch.tensor([[M - 1, M - 4]], dtype=torch.int32, device=DEV)
    out = qg.combine_experts(z, slot, torch.ones((1, 2), device=DEV), out_dtype=torch.float32)
    assert torch.equal(out[0], z[M - 1].float() + z[M - 4].float())


@pytest.mark.parametrize("R", [4, 3000])
def test_experts_weights_beyond_32_bits(R):
    """Both kernels (a mean of 1 and of 300 rows), the last of ten matrices at
    2.4e9 codes and beyond; tokens gathered from just under 2^31 codes."""
    g, E, N, K, T = gen(2), 10, 16400, 16384, 131000
    wq = torch.zeros((E, N, K), dtype=torch.uint8, device=DEV).view(F8)
    wq[-1].view(torch.uint8).copy_(small_codes((N, K), g).view(torch.uint8))
    ws = torch.ones((E, 129, 128), device=DEV)
    xq = torch.zeros((T, K), dtype=torch.uint8, device=DEV).view(F8)
    xq.view(torch.uint8)[-8:] = small_codes((8, K), g).view(torch.uint8)
    xs = torch.ones((T, 128), device=DEV)
    off = torch.zeros(E + 1, dtype=torch.int32, device=DEV)
    off[-1] = R
    token = (T - 1 - torch.arange(R, device=DEV) % 8).int()
    y = qg.gemm_f8_b128_experts(xq, xs, wq, ws, off, row_token=token, out_dtype=torch.float32)
    want = qg.gemm_f8_b128(rows(xq, token[:4].long()), xs[:4], wq[-1], ws[-1], out_dtype=torch.float32)
    assert want.any() and torch.equal(y[:4], want)
    assert torch.equal(y[8:], y[:-8])                  # row r takes the token of row r - 8
    with pytest.raises(RuntimeError):                  # one token more than 2^31 codes
        big = torch.empty((131073, K), dtype=torch.uint8, device=DEV).view(F8)
        qg.gemm_f8_b128_experts(big, torch.empty((131073, 128), device=DEV), wq, ws, off, row_token=token)
