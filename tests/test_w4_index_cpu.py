"""Where the 4-bit products' loads of scales and zeros start (csrc/fm_w4_index.hpp), over
the sizes at which a block of columns ends inside or before one of its tiles.  The scalar
part of a buffer load's offset is taken from the resource's size before the lane's part is
compared with what is left: it must never be past the resource."""
import os
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "tile_gemm_communication_amd", "csrc")

PROGRAM = r"""
#include <cstdio>
#include <initializer_list>
#include "fm_w4_index.hpp"
int main() {
  int bad = 0;
  for (int groups = 0; groups <= 9; ++groups)
    for (int N = 8; N <= 400; N += 8)
      for (int columns : {16, 32, 48, 64, 128})        // of a block
        for (int n0 = 0; n0 < N; n0 += columns)
          for (int tile = 0; tile < columns; tile += 16)
            for (int group = 0; group < groups + 4; ++group) {
              const int at = fm::scale_offset(group, groups, fm::tile_column(n0, tile, N), N, groups > 0);
              const int bytes = groups * N * 2;
              const int want = ((group < groups ? group : groups - 1) * N + n0 + tile) * 2;
              if (at < 0 || at > bytes || (groups > 0 && at >= bytes) ||
                  (groups > 0 && n0 + tile < N && at != want)) {
                if (!bad++) std::printf("groups %d N %d block %d from %d tile %d group %d: %d of %d bytes\n",
                                        groups, N, columns, n0, tile, group, at, bytes);
              }
            }
  return bad != 0;
}
"""


@pytest.mark.skipif(shutil.which("g++") is None, reason="no host compiler")
def test_scale_offsets_stay_in_the_matrix(tmp_path):
    src = tmp_path / "index.cpp"
    src.write_text(PROGRAM)
    exe = tmp_path / "index"
    subprocess.run(["g++", "-std=c++17", "-Wall", "-Werror", "-I", CSRC, str(src), "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout
