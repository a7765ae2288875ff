"""The macro-tile of an 8-bit product (csrc/fm_i8_choice.hpp) for the sizes by which the GPU
tests run each of them, on a chip of 256 compute units: a size whose choice moves would
leave its tile untested under the old name."""
import os
import shutil
import subprocess

import pytest

from test_gpu_i8 import ROUNDS, TILED

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "tile_gemm_communication_amd", "csrc")
UNITS = 256

PROGRAM = r"""
#include <cstdio>
#include "fm_i8_choice.hpp"
int main() {
  long long M, N, K;
  int cus;
  while (std::scanf("%lld %lld %lld %d", &M, &N, &K, &cus) == 4) {
    const fm::TileChoice& c = fm::kTileChoices[fm::choose_tile(M, N, K, cus)];
    std::printf("%dx%d %d\n", c.bm, c.bn, c.resident);
  }
}
"""


@pytest.fixture(scope="module")
def choose(tmp_path_factory):
    """(tile, blocks on a unit) of sizes (M, N, K)."""
    if shutil.which("g++") is None:
        pytest.skip("no host compiler")
    d = tmp_path_factory.mktemp("choice")
    (d / "choice.cpp").write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-Wall", "-Werror", "-I", CSRC, str(d / "choice.cpp"), "-o",
                    str(d / "choice")], check=True)

    def run(sizes):
        lines = "".join(f"{M} {N} {K} {UNITS}\n" for M, N, K in sizes)
        out = subprocess.run([str(d / "choice")], input=lines, capture_output=True, text=True, check=True).stdout
        return [(t, int(r)) for t, r in (line.split() for line in out.splitlines())]

    return run


@pytest.mark.parametrize("tile", TILED)
def test_sizes_take_the_tile_they_are_named_for(choose, tile):
    assert [t for t, _ in choose(TILED[tile])] == [tile] * len(TILED[tile])


@pytest.mark.parametrize("tile", ROUNDS)
def test_sizes_take_several_tiles_a_block(choose, tile):
    bm, bn = map(int, tile.split("x"))
    for (M, N, K), (got, resident) in zip(ROUNDS[tile], choose(ROUNDS[tile])):
        tiles = -(-M // bm) * -(-N // bn)
        assert got == tile and tiles > UNITS * resident and tiles % (UNITS * resident), (M, N, K, got)
