"""CPU-only: the scale loads of the MXFP4 forward tiles stay inside their arrays.

The loads add the chunk as a scalar offset, which the buffer's range check need
not see, so the lanes' own offsets must be in bounds in every chunk, the last one
among them.  The header that forms them is compiled for the host and walked over
every lane of every tile.
"""

import os
import shutil
import subprocess

import pytest

from bit_nf4_quantized_08_amd import build

WALK = r"""
#include <stdio.h>
#include "qn_mx_scales.h"

// Tiles of `tile` rows over a matrix of `rows` rows in `chunks` chunks: 0 when all is well.
static int walk(long rows, long chunks, int tile) {
  for (long first = 0; first < rows; first += tile)
    for (int group = 0; group < tile; group += 128)
      for (int lane = 0; lane < 64; ++lane) {
        const long row = first + group + 2 * lane;
        const long off = qn::mx_scale_pair(row, rows);
        if (row < rows && off != row * 8) return 1;                   // a row's own scales
        const long end = (chunks - 1) * rows * 8 + off + 16;          // in the last chunk
        if (end > chunks * rows * 8 + (rows % 2 ? 8 : 0)) return 2;   // inside the array
      }
  return 0;
}

int main() {
  for (int tile = 128; tile <= 256; tile += 128)
    for (long chunks = 1; chunks <= 33; chunks += 8) {
      for (long m = 33; m <= 1100; ++m)       // rows of X
        if (int e = walk(m, chunks, tile)) return printf("X rows %ld chunks %ld tile %d: %d\n", m, chunks, tile, e), 1;
      for (long n = 64; n <= 9000; n += 64)   // rows of the weight
        if (int e = walk(n, chunks, tile)) return printf("W rows %ld chunks %ld tile %d: %d\n", n, chunks, tile, e), 1;
    }
  return 0;
}
"""


@pytest.mark.skipif(shutil.which("g++") is None, reason="no host compiler")
def test_scale_loads_stay_inside(tmp_path):
    src, exe = tmp_path / "walk.cpp", tmp_path / "walk"
    src.write_text(WALK)
    r = subprocess.run(["g++", "-std=c++17", "-O1", "-I", build.CSRC, str(src), "-o", str(exe)], capture_output=True,
                       text=True)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0, r.stdout


def test_the_forward_tiles_use_them():
    """The kernel forms its offsets with that function, and X^'s codes follow its scales in the workspace."""
    with open(os.path.join(build.CSRC, "k_mx.hip")) as f:
        src = f.read()
    assert "const uint32_t eo = mx_scale_pair(" in src
    assert src.index("p.xs = c.take<uint8_t>") < src.index("p.xc = c.take<uint8_t>")
