"""Argument checks of the e4m3 and expert entry points, on the host: every call
here fails validation, or is empty, before anything is launched."""
import ctypes
import os

import pytest

OK, NULL, SHAPE, ALIGN, DTYPE, HIP, ARG = range(7)
A, MIS, ODD = ctypes.c_void_p(4096), ctypes.c_void_p(4104), ctypes.c_void_p(4097)
BIG = 2 ** 30 + 1


@pytest.fixture(scope="module")
def lib():
    import bit_quantized_gemm_int8_amd as q
    if not os.path.exists(q.LIB_PATH):
        from bit_quantized_gemm_int8_amd.build import build
        build()
    return q.load()


def test_quantizers(lib):
    f = lib.quantize_f8_g128
    assert f(None, 0, 4, 16, A, A, None) == NULL
    assert f(A, 0, 4, 16, A, None, None) == NULL
    for K in (0, -16, 17, 24, 2 ** 20 + 16):
        assert f(A, 0, 4, K, A, A, None) == SHAPE
    assert f(A, 0, -1, 16, A, A, None) == SHAPE and f(A, 0, BIG, 16, A, A, None) == SHAPE
    assert f(A, 0, 2 ** 30, 16, A, A, None) == SHAPE          # more threads than a launch holds
    assert f(A, 3, 4, 16, A, A, None) == DTYPE
    assert f(MIS, 0, 4, 16, A, A, None) == ALIGN and f(A, 0, 4, 16, MIS, A, None) == ALIGN
    assert f(A, 0, 4, 16, A, ODD, None) == ALIGN
    assert f(None, 0, 0, 16, None, None, None) == OK
    w = lib.quantize_weight_f8_b128
    assert w(None, 0, 1, 16, 4, A, A, None) == NULL
    assert w(A, 0, 1, 24, 4, A, A, None) == SHAPE and w(A, 0, 1025, 16, 4, A, A, None) == SHAPE
    assert w(A, 0, 1024, 2 ** 20, 2 ** 20, A, A, None) == SHAPE
    assert w(A, -1, 1, 16, 4, A, A, None) == DTYPE
    assert w(MIS, 0, 1, 16, 4, A, A, None) == ALIGN
    assert w(None, 0, 0, 16, 4, None, None, None) == OK and w(None, 0, 2, 16, 0, None, None, None) == OK


def test_product(lib):
    g = lib.gemm_f8_b128
    for i in range(4):
        p = [A, A, A, A]
        p[i] = None
        assert g(*p, 4, 4, 16, A, 2, None) == NULL
        p[i] = MIS if i in (0, 2) else ODD
        assert g(*p, 4, 4, 16, A, 2, None) == ALIGN
    assert g(A, A, A, A, 4, 4, 16, None, 2, None) == NULL
    assert g(A, A, A, A, 4, 4, 16, ODD, 2, None) == ALIGN
    assert g(A, A, A, A, 4, 4, 24, A, 2, None) == SHAPE
    assert g(A, A, A, A, BIG, 4, 16, A, 2, None) == SHAPE and g(A, A, A, A, 4, BIG, 16, A, 2, None) == SHAPE
    assert g(A, A, A, A, 2 ** 30, 2 ** 30, 16, A, 2, None) == SHAPE
    assert g(A, A, A, A, 4, 4, 16, A, 3, None) == DTYPE
    assert g(None, None, None, None, 0, 4, 16, None, 2, None) == OK
    assert g(None, None, None, None, 4, 0, 16, None, 2, None) == OK


def test_experts_product(lib):
    g = lib.gemm_f8_b128_experts
    dims = (8, 8, 2, 4, 16)                                    # T R E N K
    for i in range(5):
        p = [A] * 5
        p[i] = None
        assert g(*p, None, *dims, A, 2, None) == NULL
        p[i] = MIS if i in (0, 2) else ODD
        assert g(*p, None, *dims, A, 2, None) == ALIGN
    assert g(*[A] * 5, ODD, *dims, A, 2, None) == ALIGN
    assert g(*[A] * 5, None, *dims, None, 2, None) == NULL
    assert g(*[A] * 5, None, 7, 8, 2, 4, 16, A, 2, None) == SHAPE      # no row_token: T must be R
    assert g(*[A] * 5, A, 2 ** 27, 8, 2, 4, 16, A, 2, None) == SHAPE   # T K reaches 2^31
    for E in (0, -1, 1025):
        assert g(*[A] * 5, None, 8, 8, E, 4, 16, A, 2, None) == SHAPE
    assert g(*[A] * 5, None, 8, 8, 1024, 2 ** 30, 16, A, 2, None) == SHAPE
    assert g(*[A] * 5, None, 8, 8, 2, 4, 8, A, 2, None) == SHAPE
    assert g(*[A] * 5, None, *dims, A, 3, None) == DTYPE
    assert g(*[None] * 6, 0, 0, 2, 4, 16, None, 2, None) == OK
    assert g(*[None] * 6, 8, 8, 2, 0, 16, None, 2, None) == OK


def test_route(lib):
    def f(lg=A, dt=0, bias=None, T=4, E=12, groups=1, top=1, k=2, score=0, renorm=1, e=A, w=A):
        return lib.route_experts(lg, dt, bias, T, E, groups, top, k, score, renorm, 1.0, e, w, None)
    assert f(lg=None) == NULL and f(e=None) == NULL and f(w=None) == NULL
    assert f(lg=ctypes.c_void_p(4098)) == ALIGN and f(bias=ODD) == ALIGN and f(e=ODD) == ALIGN and f(w=ODD) == ALIGN
    assert f(dt=1, lg=ODD) == ALIGN
    for bad in (dict(T=-1), dict(T=BIG), dict(E=0), dict(E=1025), dict(groups=0), dict(groups=5), dict(E=130, groups=65),
                dict(groups=4, top=0), dict(groups=4, top=5), dict(k=0), dict(k=13), dict(E=200, k=65), dict(groups=4, top=1, k=4)):
        assert f(**bad) == SHAPE, bad
    assert f(score=2) == ARG and f(score=-1) == ARG and f(renorm=2) == ARG and f(dt=3) == DTYPE
    assert f(T=0, lg=None, e=None, w=None) == OK


def test_plan_and_combine(lib):
    p = lib.plan_experts
    assert p(None, 4, 2, 3, A, A, A, None) == NULL and p(A, 4, 2, 3, None, A, A, None) == NULL
    assert p(A, 4, 2, 3, A, None, A, None) == NULL and p(A, 4, 2, 3, A, A, None, None) == NULL
    assert p(ODD, 4, 2, 3, A, A, A, None) == ALIGN and p(A, 4, 2, 3, A, A, ODD, None) == ALIGN
    for T, k, E in ((-1, 2, 3), (4, 0, 3), (4, 65, 3), (4, 2, 0), (4, 2, 1025), (2 ** 30, 2, 3)):
        assert p(A, T, k, E, A, A, A, None) == SHAPE
    c = lib.combine_experts
    assert c(None, 0, A, A, 4, 2, 8, 16, A, 0, None) == NULL and c(A, 0, None, A, 4, 2, 8, 16, A, 0, None) == NULL
    assert c(A, 0, A, None, 4, 2, 8, 16, A, 0, None) == NULL and c(A, 0, A, A, 4, 2, 8, 16, None, 0, None) == NULL
    assert c(ODD, 1, A, A, 4, 2, 8, 16, A, 0, None) == ALIGN and c(A, 0, A, A, 4, 2, 8, 16, ODD, 1, None) == ALIGN
    assert c(A, 3, A, A, 4, 2, 8, 16, A, 0, None) == DTYPE and c(A, 0, A, A, 4, 2, 8, 16, A, 3, None) == DTYPE
    for T, k, R, N in ((-1, 2, 8, 16), (4, 0, 8, 16), (4, 65, 8, 16), (4, 2, -1, 16), (4, 2, 8, -1), (2 ** 28, 2, 8, 4096)):
        assert c(A, 0, A, A, T, k, R, N, A, 0, None) == SHAPE
    assert c(None, 0, None, None, 0, 2, 0, 16, None, 0, None) == OK and c(None, 0, None, None, 4, 2, 0, 0, None, 0, None) == OK
