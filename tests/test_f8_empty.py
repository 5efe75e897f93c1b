"""Calls of the experts' product without rows or without tokens."""
import ctypes
import os

import pytest
import torch

import bit_quantized_gemm_int8_amd as qg

DEV = "cuda"
F8 = torch.float8_e4m3fn
A = ctypes.c_void_p(4096)


def test_no_rows_of_some_tokens():
    """Without rows there is nothing to read: a row_token of no rows may be NULL
    whatever T is."""
    if not os.path.exists(qg.LIB_PATH):
        from bit_quantized_gemm_int8_amd.build import build
        build()
    g = qg.load().gemm_f8_b128_experts
    assert g(A, A, A, A, A, None, 7, 0, 2, 4, 16, None, 2, None) == 0
    assert g(A, A, A, A, A, None, 7, 8, 2, 4, 16, A, 2, None) == 2          # rows: T must be R


@pytest.mark.gpu
def test_no_rows_of_some_tokens_from_python():
    xq, xs = torch.zeros((5, 144), device=DEV).to(F8), torch.ones((5, 2), device=DEV)
    wq, ws = torch.zeros((3, 16, 144), device=DEV).to(F8), torch.ones((3, 1, 2), device=DEV)
    none = torch.empty(0, dtype=torch.int32, device=DEV)
    y = qg.gemm_f8_b128_experts(xq, xs, wq, ws, torch.zeros(4, dtype=torch.int32, device=DEV), row_token=none)
    assert y.shape == (0, 16)


@pytest.mark.gpu
@pytest.mark.parametrize("R", [6, 90, 3000])
def test_rows_without_tokens(R):
    """Rows of no token (a fixed-size batch on a GPU that got none) are zeros;
    rows of no run stay as they were.  The stream kernel and both tile sizes."""
    E, N, K = 3, 4100, 272
    xq, xs = torch.empty((0, K), device=DEV).to(F8), torch.empty((0, 3), device=DEV)
    wq, ws = torch.ones((E, N, K), device=DEV).to(F8), torch.ones((E, 33, 3), device=DEV)
    off = torch.tensor([0, R // 3, R // 2, R - 1], dtype=torch.int32, device=DEV)
    for token in (-1, 0):
        out = torch.full((R, N), 3.0, dtype=torch.bfloat16, device=DEV)
        qg.gemm_f8_b128_experts(xq, xs, wq, ws, off, row_token=torch.full((R,), token, dtype=torch.int32, device=DEV), out=out)
        assert not out[:-1].any() and torch.all(out[-1] == 3.0)
