"""Host-side arithmetic of the operators' kernels, compiled with the host compiler and
run on the CPU."""
import ctypes
import os
import subprocess

import numpy as np
import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "mixture_experts_layer_stable_gb300", "csrc")


def compiled(tmp_path, source, *flags):
    """The shared library of a C++ source that may include the kernels' host headers."""
    src, so = tmp_path / "t.cpp", tmp_path / "t.so"
    src.write_text(source)
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", "-shared", "-fPIC", "-I", CSRC, str(src), "-o",
                    str(so), *flags], check=True)
    return ctypes.CDLL(str(so))


TILES = """
#include "row_tiles.h"
extern "C" int max_tok() { return moe::kMaxTok; }
extern "C" int tiles(int c) { return moe::tok_tiles(c); }
extern "C" int most(int c) { return moe::tok_most(c); }
extern "C" void starts(int c, int* out) {
  const int n = moe::tok_tiles(c);
  for (int t = 0; t < n; ++t) out[t] = moe::tok_start(c, n, t);
}
"""


@pytest.fixture(scope="module")
def tiles(tmp_path_factory):
    return compiled(tmp_path_factory.mktemp("tiles"), TILES)


@pytest.mark.parametrize("counts", [range(0, 1300), [5136960, 5136961, 6000000, (1 << 24) + 1, 100000007],
                                    [(1 << 28) - 191, (1 << 28) - 1, 1 << 28]])
def test_tiles_cover_an_expert_s_rows(tiles, counts):
    """Tiles begin at 0, on multiples of 64, and none is empty or longer than the largest."""
    for c in counts:
        n, most = tiles.tiles(c), tiles.most(c)
        assert n == -(-c // tiles.max_tok()) and most <= tiles.max_tok()
        if n == 0:
            assert most == 0
            continue
        s = np.zeros(n, dtype=np.int32)
        tiles.starts(c, s.ctypes.data_as(ctypes.c_void_p))
        rows = np.diff(np.append(s.astype(np.int64), c))
        assert s[0] == 0 and not (s % 64).any() and rows.min() >= 1, c
        assert rows.max() == most if n <= 4 else rows.max() <= most, c
        # 128-row scale tiles that a tile touches: one where the largest tile has up to 128 rows, else two
        assert (s % 128 + rows).max() <= (128 if most <= 128 else 256), c
