"""Which tile the library computes an e4m3 product with: its own choice
(csrc/fp8_tiles.h, host code without GPU headers), compiled with g++."""
from __future__ import annotations

import ctypes
import functools
import os
import subprocess
import tempfile
from typing import NamedTuple

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "quantized_latent_moe_amd", "csrc")
DENSE, DENSE_EXACT, GATED, GATED_EXACT = range(4)

_SOURCE = """
#include "fp8_tiles.h"
extern "C" void choose(int product, int64_t T, int N, int nb, int num_cus, int64_t* out) {
  const int v = latmoe::fp8_pick_tile(product, T, N, nb, num_cus);
  const latmoe::Fp8Tile t = latmoe::kFp8Tiles[product][v];
  out[0] = v, out[1] = t.cols(), out[2] = t.tokens, out[3] = t.count(T, N), out[4] = t.stays();
}
"""


class Choice(NamedTuple):
    variant: int
    cols: int
    tokens: int
    tiles: int
    stays: bool   # workgroups take one tile after the other


@functools.lru_cache(None)
def _lib():
    with tempfile.TemporaryDirectory() as d:
        src, so = os.path.join(d, "t.cpp"), os.path.join(d, "t.so")
        with open(src, "w") as f:
            f.write(_SOURCE)
        subprocess.check_call(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", "-shared", "-fPIC", "-I", CSRC, "-o", so, src])
        c = ctypes.CDLL(so)
    c.choose.argtypes = [ctypes.c_int, ctypes.c_int64, ctypes.c_int, ctypes.c_int, ctypes.c_int,
                         ctypes.POINTER(ctypes.c_int64)]
    c.choose.restype = None
    return c


def choose(product: int, T: int, N: int, K: int, num_cus: int = 256) -> Choice:
    """The tile of a product of T rows with N weight rows (gated: N columns of H) and K columns."""
    out = (ctypes.c_int64 * 5)()
    _lib().choose(product, T, N, -(-K // 128), num_cus, out)
    return Choice(out[0], out[1], out[2], out[3], bool(out[4]))


# Products whose workgroups take a second tile, with steps in several runs of
# four, the last one not full, and ragged ends of T, N and K: (product, cols and
# tokens of the tile, T, N, K).  Every tile whose workgroups stay, twice.
WALKS = [
    (DENSE, (256, 128), 5987, 2050, 656), (DENSE, (256, 128), 9100, 1300, 1136),
    (DENSE, (128, 128), 5003, 2100, 720), (DENSE, (128, 128), 4490, 2340, 528),
    (DENSE_EXACT, (128, 192), 5003, 2100, 720), (DENSE_EXACT, (128, 192), 9001, 1041, 1136),
    (DENSE_EXACT, (128, 128), 8190, 1571, 720), (DENSE_EXACT, (128, 128), 5990, 2050, 656),
    (GATED, (128, 128), 5987, 1040, 656), (GATED, (128, 128), 6100, 1040, 1168),
    (GATED, (128, 64), 4133, 1104, 720), (GATED, (128, 64), 2099, 2064, 528),
    (GATED_EXACT, (128, 64), 4133, 1104, 720), (GATED_EXACT, (128, 64), 2500, 1040, 1168),
]
