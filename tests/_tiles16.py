"""How the library computes a 16-bit product: its own choice
(csrc/dense16_tiles.h, host code without GPU headers), compiled with g++."""
from __future__ import annotations

import ctypes
import functools
import os
import subprocess
import tempfile

from tests._tiles import CSRC

_SOURCE = """
#include "dense16_tiles.h"
using namespace latmoe;
// -1 and the rows of a workgroup for the kernel that streams the weights, else the first launch: variant, tokens
extern "C" void choose(int64_t T, int64_t rows, int K, int num_cus, int64_t* out) {
  if (dense16_small(T, rows, num_cus)) {
    out[0] = -1, out[1] = dense16_small_rows(T, rows, num_cus);
    return;
  }
  const Dense16Launch p = dense16_plan(T, rows, (K + 63) / 64, num_cus);
  out[0] = p.variant, out[1] = p.tokens;
}
"""


@functools.lru_cache(None)
def _lib():
    with tempfile.TemporaryDirectory() as d:
        src, so = os.path.join(d, "t.cpp"), os.path.join(d, "t.so")
        with open(src, "w") as f:
            f.write(_SOURCE)
        subprocess.check_call(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", "-shared", "-fPIC", "-I", CSRC, "-o", so, src])
        c = ctypes.CDLL(so)
    c.choose.argtypes = [ctypes.c_int64, ctypes.c_int64, ctypes.c_int, ctypes.c_int, ctypes.POINTER(ctypes.c_int64)]
    c.choose.restype = None
    return c


def launches(T: int, rows: int, K: int, num_cus: int = 256) -> list:
    """(variant, tokens) of each launch; variant -1 is the streaming kernel, then with its rows a workgroup."""
    out, got = (ctypes.c_int64 * 2)(), []
    while T > 0:
        _lib().choose(T, rows, K, num_cus, out)
        if out[0] < 0:
            return got + [(-1, out[1])]
        got.append((out[0], out[1]))
        T -= out[1]
    return got


# Products, ragged in every direction, and the variants of their launches:
# (T, weight rows, K), the rows even so that a gated pair has them too.
RAGGED = [
    ((4978, 2370, 72), [0]), ((7875, 1962, 712), [0]), ((6007, 1298, 72), [1]), ((4913, 4470, 688), [1]),
    ((3135, 1302, 72), [2]), ((2887, 5430, 632), [2]), ((329, 5746, 72), [3]), ((2097, 1898, 688), [3]),
    ((914, 4260, 80), [4]), ((1577, 2558, 680), [4]), ((4353, 68, 72), [5]), ((497, 3966, 712), [5]),
    ((38, 1470, 72), [6]), ((508, 998, 688), [6]),
    ((4990, 5002, 4088), [0, 1]), ((2950, 8182, 4088), [0, 2]), ((6001, 3110, 2056), [0, 3]),
    ((4133, 4102, 2056), [0, 4]), ((4100, 8182, 2056), [0, -1]),
]
