"""The layer norm kernels read nothing outside x, dy and dres: their rule for rows that share 16-byte units with their
neighbours (csrc/srnl_norm.h), compiled here and followed over every unit of short buffers."""
import os
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "self_referential_nested_b200", "csrc")

PROGRAM = r"""
#include <cstdio>
#include "srnl_norm.h"
int main() {
  int bad = 0, shared = 0;
  for (int V = 4; V <= 8; V += 4)
    for (int dim = 1; dim <= 3 * V + 1; ++dim)
      for (long rows = 1; rows <= 40; ++rows)
        for (long r = 0; r < rows; ++r) {
          const int room = srnl::row_room(r, rows, dim);
          const int sh = (int)(r * dim % V);
          for (int c = -sh; c < dim; c += V)
            for (int clips = 0; clips < 2; ++clips) {
              if (!srnl::unit_in_one_piece(c, V, dim, room, clips != 0)) continue;
              const long from = r * dim + c;
              if (from < 0 || from + V > rows * dim || from % V != 0) {
                if (bad++ < 5) std::printf("V %d dim %d rows %ld row %ld column %d\n", V, dim, rows, r, c);
              }
              if (c < 0 || c + V > dim) {
                ++shared;
                if (!clips) ++bad;
              }
            }
        }
  std::printf("%d out of range, %d shared\n", bad, shared);
  return bad != 0 || shared == 0;
}
"""


def test_units_that_are_read_whole_lie_in_the_buffer(tmp_path):
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no C++ compiler")
    src, exe = tmp_path / "reads.cpp", tmp_path / "reads"
    src.write_text(PROGRAM)
    subprocess.run([cxx, "-std=c++17", "-I", CSRC, str(src), "-o", str(exe)], check=True)
    done = subprocess.run([str(exe)], capture_output=True, text=True)
    assert done.returncode == 0, done.stdout
