"""CPU check of the sampling's reads: no 16-byte piece that is fetched whole leaves the logits' own range of addresses."""
import ctypes
import os
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "rl_post_trainer_gb300", "csrc")

SOURCE = r"""
#include "slice_edges.h"
// The first fault of a matrix whose first element lies `base` elements into a piece, its rows cut for `ctas` CTAs; 0: none.
extern "C" int faults(uint32_t rows, uint32_t vocab, uint64_t stride, uint32_t base, uint32_t ctas, uint32_t piece) {
  const uint64_t span = (rows - 1) * stride + vocab;
  const uint32_t per = ((vocab + ctas - 1) / ctas + piece - 1) / piece * piece;
  for (uint32_t row = 0; row < rows; ++row)
    for (uint32_t rank = 0; rank < ctas; ++rank) {
      const uint32_t begin = rank * per < vocab ? rank * per : vocab, count = vocab - begin < per ? vocab - begin : per;
      const uint64_t at = row * stride + begin;
      const uint32_t lead = uint32_t((base + at) % piece);
      const pulse::SliceEdges e = pulse::slice_edges(at, count, lead, piece, span);
      if (uint64_t(e.pieces) * piece < lead + count || (count && uint64_t(e.pieces) * piece >= lead + count + piece)) return 1;
      for (uint32_t i = 0; i < e.pieces; ++i) {
        const int64_t from = int64_t(at) - lead + int64_t(i) * piece;
        const bool inside = from >= 0 && from + piece <= int64_t(span);
        const bool edge = (i == 0 && e.low) || (i + 1 == e.pieces && e.high);
        if (!inside && !edge) return 2;  // fetched whole, and not all of it the matrix's
        if (inside && edge) return 3;    // by elements without need
      }
    }
  return 0;
}
"""


@pytest.fixture(scope="module")
def faults(tmp_path_factory):
    gxx = shutil.which("g++")
    assert gxx, "g++ not found"
    d = tmp_path_factory.mktemp("edges")
    (d / "edges.cc").write_text(SOURCE)
    subprocess.run([gxx, "-O2", "-std=c++17", "-Wall", "-Werror", "-shared", "-fPIC", "-I", CSRC, "-o", str(d / "edges.so"), str(d / "edges.cc")], check=True)
    f = ctypes.CDLL(str(d / "edges.so")).faults
    f.argtypes = [ctypes.c_uint32, ctypes.c_uint32, ctypes.c_uint64, ctypes.c_uint32, ctypes.c_uint32, ctypes.c_uint32]
    return f


@pytest.mark.parametrize("piece", [4, 8])
def test_pieces_stay_inside(faults, piece):
    for rows in (1, 2, 3, 5, 9):
        for vocab in list(range(1, 30)) + [63, 64, 65, 127, 1000]:
            for extra in (0, 1, 2, 3, 7, 8, 40):
                for base in range(piece):
                    for ctas in (1, 2, 4, 16):
                        assert faults(rows, vocab, vocab + extra, base, ctas, piece) == 0, (rows, vocab, extra, base, ctas)


def test_far_rows(faults):
    """Rows whose offsets pass 2^32 elements."""
    for rows, vocab, stride in ((4, 1003, 1500000000), (3, 200003, 1 << 39), (2, 1 << 30, 1 << 31)):
        for base in range(8):
            for ctas in (1, 16):
                assert faults(rows, vocab, stride, base, ctas, 8) == 0
