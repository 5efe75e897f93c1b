"""Index arithmetic of the e4m3 tile kernels (csrc/qg_f8_index.hpp), compiled
for the host and walked there."""
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "bit_quantized_gemm_int8_amd", "csrc")


def run_host(tmp_path, body):
    """Output of a C++ program that includes the header."""
    src, exe = tmp_path / "walk.cpp", tmp_path / "walk"
    src.write_text('#include <cstdio>\n#include <initializer_list>\n#include "qg_f8_index.hpp"\nusing namespace qg;\nint main() {\n' + body + "\n}\n")
    subprocess.run(["g++", "-std=c++17", "-O1", "-I", CSRC, str(src), "-o", str(exe)], check=True, capture_output=True, text=True)
    return subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout


# Counts dwords that a load would touch past the array, and scales in use that
# it would not deliver, if the range check knew the vector offset only.
WALK = """
  long past = 0, lost = 0;
  for (int stages = 1; stages <= 4; stages += 3)
    for (int rows = 1; rows <= 5; ++rows)
      for (int G = 1; G <= 40; ++G)
        for (int r = -1; r < rows; ++r)
          for (int g = 0; g < G; g += stages) {
            const uint64_t size = 4ull * rows * G;
            const F8ScaleLoad at = %s;
            for (int i = 0; i < stages; ++i) {
              const uint64_t v = (uint64_t)at.voffset + 4 * i, byte = v + at.soffset;
              const bool read = v + 4 <= size;
              past += read && byte + 4 > size;
              if (r < 0) past += read;
              else if (g + i < G) lost += !(read && byte == 4ull * (r * G + g + i));
            }
          }
  printf("%%ld %%ld", past, lost);
"""
ROW = "r < 0 ? 0x80000000u : 4u * r * G"


def test_scale_loads_stay_inside_by_their_vector_offset(tmp_path):
    assert run_host(tmp_path, WALK % f"f8_scale_load({ROW}, g, stages)") == "0 0"


def test_the_walk_sees_a_stage_in_the_scalar_offset(tmp_path):
    past, lost = run_host(tmp_path, WALK % f"(F8ScaleLoad{{{ROW}, 4 * g}})").split()
    assert int(past) > 0 and int(lost) == 0


def test_places_in_the_tile_list_never_pass_31_bits(tmp_path):
    """The list of the experts' tiles saturates (offsets that do not rise can
    name rows many times over), and a workgroup that steps past its end still
    holds a positive place."""
    out = run_host(tmp_path, """
  long bad = 0;
  for (int tiles_n : {1, 2, 3, 7, 64, 1000, 8388608, 16777216})
    for (int grid : {8, 16, 256, 512, 1024}) {
      const int64_t end = (int64_t)f8_most_tile_rows(tiles_n, grid) * tiles_n;
      bad += end < 1 || end + grid / 8 + 1 > INT32_MAX || end + grid + tiles_n < INT32_MAX;
    }
  printf("%ld", bad);
""")
    assert out == "0"
