"""Which kernel an e4m3 product runs on: the library's own rule
(csrc/qg_f8_index.hpp), compiled for the host."""
import ctypes
import functools
import os
import subprocess
import tempfile

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
NAMES = ("stream", "64x64 by two groups", "64x64", "128x128", "256x256")


@functools.lru_cache(None)
def _rule():
    with tempfile.TemporaryDirectory() as at:
        src, lib = os.path.join(at, "choice.cpp"), os.path.join(at, "choice.so")
        with open(src, "w") as f:
            f.write('#include "qg_f8_index.hpp"\n'
                    'extern "C" int choice(int experts, int64_t R, int64_t E, int64_t N, int wide) {\n'
                    "  return (int)qg::f8_kernel(experts, R, E, N, wide);\n}\n")
        subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-I", os.path.join(ROOT, "bit_quantized_gemm_int8_amd", "csrc"),
                        src, "-o", lib], check=True, capture_output=True, text=True)
        f = ctypes.CDLL(lib).choice
    f.argtypes = [ctypes.c_int, ctypes.c_int64, ctypes.c_int64, ctypes.c_int64, ctypes.c_int]
    return f


def kernel(M, N, out, E=None):
    """Name of the kernel for M rows (of E experts) of N outputs of type `out`."""
    return NAMES[_rule()(E is not None, M, 1 if E is None else E, N, out == "f32")]
