"""Argument checks of the 4-bit paged cache, on the host: every call here fails
validation, or is empty, before anything is launched."""
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


def test_page_bytes(lib):
    f = lib.kv_u4_page_bytes
    assert f(64, 128) == 64 * 136 and f(16, 64) == 16 * 72 and f(256, 256) == 256 * 272
    for page, D in ((0, 128), (8, 128), (48, 128), (512, 128), (-16, 128), (64, 0), (64, 96), (64, 512), (64, -64)):
        assert f(page, D) == 0


WHERE = dict(T=6, H=2, D=128, pages=A, P=5, page=64, table=A, W=3, lengths=A, offsets=None, B=3)
BAD_WHERE = [(dict(T=-1), SHAPE), (dict(T=BIG), SHAPE), (dict(T=7), SHAPE), (dict(H=0), SHAPE), (dict(H=1025), SHAPE),
             (dict(D=96), SHAPE), (dict(D=512), SHAPE), (dict(page=8), SHAPE), (dict(page=48), SHAPE), (dict(page=512), SHAPE),
             (dict(P=-1), SHAPE), (dict(P=BIG), SHAPE), (dict(W=-1), SHAPE), (dict(W=2 ** 24 + 1), SHAPE),
             (dict(B=0), SHAPE), (dict(B=-1), SHAPE), (dict(B=BIG), SHAPE), (dict(pages=None), NULL), (dict(table=None), NULL),
             (dict(lengths=None), NULL), (dict(pages=MIS), ALIGN), (dict(table=ODD), ALIGN), (dict(lengths=ODD), ALIGN),
             (dict(offsets=ODD), ALIGN)]


def append(lib, q=A, qs=512, k=A, ks=256, v=A, vs=256, dtype=2, cos=A, sin=A, rows=64, rot=128, inter=0, Hq=4, out=A, **w):
    w = {**WHERE, **w}
    return lib.append_kv_u4_pages(q, qs, k, ks, v, vs, dtype, cos, sin, rows, rot, inter, w["T"], Hq, w["H"], w["D"], w["pages"],
                                  w["P"], w["page"], w["table"], w["W"], w["lengths"], w["offsets"], w["B"], out, None)


def dequantize(lib, k=A, v=A, dtype=2, **w):
    w = {**WHERE, **w}
    return lib.dequantize_kv_u4_pages(w["pages"], w["P"], w["page"], w["table"], w["W"], w["lengths"], w["offsets"], w["B"],
                                      w["T"], w["H"], w["D"], k, v, dtype, None)


def attend(lib, q=A, qs=512, dtype=2, Hq=4, window=0, sinks=0, scale=0.1, out=A, ws=A, size=1 << 40, **w):
    w = {**WHERE, **w}
    return lib.attend_kv_u4_pages(q, qs, dtype, w["T"], Hq, w["H"], w["D"], w["pages"], w["P"], w["page"], w["table"], w["W"],
                                  w["lengths"], w["offsets"], w["B"], window, sinks, scale, out, ws, size, None)


@pytest.mark.parametrize("call", [append, dequantize, attend])
def test_where(lib, call):
    for bad, code in BAD_WHERE:
        assert call(lib, **bad) == code, bad
    assert call(lib, T=0, B=0, pages=None, table=None, lengths=None, P=0, W=0) == OK


def test_append(lib):
    for bad, code in [(dict(k=None), NULL), (dict(v=None), NULL), (dict(q=None), NULL), (dict(out=None), NULL), (dict(cos=None), NULL),
                      (dict(sin=None), NULL), (dict(k=MIS), ALIGN), (dict(v=MIS), ALIGN), (dict(q=MIS), ALIGN), (dict(out=MIS), ALIGN),
                      (dict(cos=ODD), ALIGN), (dict(sin=ODD), ALIGN), (dict(ks=255), SHAPE), (dict(vs=255), SHAPE), (dict(qs=511), SHAPE),
                      (dict(ks=260), ALIGN), (dict(dtype=0, ks=258), ALIGN), (dict(dtype=3), DTYPE), (dict(dtype=-1), DTYPE),
                      (dict(rot=-16), SHAPE), (dict(rot=24), SHAPE), (dict(rot=144), SHAPE), (dict(rows=-1), SHAPE), (dict(inter=2), ARG),
                      (dict(Hq=-1), SHAPE), (dict(Hq=1025), SHAPE), (dict(T=2 ** 30, B=2 ** 30), SHAPE)]:
        assert append(lib, **bad) == code, bad
    assert append(lib, T=0, k=None, v=None, q=None, out=None, cos=None, sin=None) == OK


def test_dequantize(lib):
    for bad, code in [(dict(k=None), NULL), (dict(v=None), NULL), (dict(k=MIS), ALIGN), (dict(v=MIS), ALIGN), (dict(dtype=3), DTYPE),
                      (dict(T=2 ** 30, B=2 ** 30), SHAPE)]:
        assert dequantize(lib, **bad) == code, bad
    assert dequantize(lib, T=0, k=None, v=None) == OK


def test_attend(lib):
    for bad, code in [(dict(q=None), NULL), (dict(out=None), NULL), (dict(q=MIS), ALIGN), (dict(out=MIS), ALIGN), (dict(ws=MIS), ALIGN),
                      (dict(qs=511), SHAPE), (dict(qs=516), ALIGN), (dict(dtype=0), DTYPE), (dict(dtype=3), DTYPE), (dict(Hq=0), SHAPE),
                      (dict(Hq=5), SHAPE), (dict(Hq=1026), SHAPE), (dict(T=2 ** 29, B=2 ** 29), SHAPE), (dict(window=-1), SHAPE),
                      (dict(sinks=-1), SHAPE), (dict(window=BIG), SHAPE), (dict(sinks=BIG), SHAPE), (dict(scale=float("nan")), ARG),
                      (dict(scale=float("inf")), ARG)]:
        assert attend(lib, **bad) == code, bad
    assert attend(lib, T=0, q=None, out=None, ws=None, size=0) == OK
    # a long cache and one sequence: split, so a workspace is needed
    need = lib.attend_kv_u4_pages_workspace_bytes(1, 1, 4, 2, 128, 64, 512, 0)
    long = dict(T=1, B=1, W=512)
    assert need > 0 and attend(lib, **long, ws=None, size=0) == NULL and attend(lib, **long, size=need - 1) == SHAPE
    # none for a short one, and 0 for sizes that the call refuses
    f = lib.attend_kv_u4_pages_workspace_bytes
    assert f(1, 1, 4, 2, 128, 64, 1, 0) == 0
    for bad in ((-1, 1, 4, 2, 128, 64, 512, 0), (1, 0, 4, 2, 128, 64, 512, 0), (3, 2, 4, 2, 128, 64, 512, 0), (1, 1, 5, 2, 128, 64, 512, 0),
                (1, 1, 4, 2, 96, 64, 512, 0), (1, 1, 4, 2, 128, 48, 512, 0), (1, 1, 4, 2, 128, 64, 2 ** 25, 0)):
        assert f(*bad) == 0, bad
