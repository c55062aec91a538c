"""The 64-bit exp of the routing by scores (CPU): the library's own code
(csrc/exp64.h, host code without GPU headers), compiled with g++ and compared
with exp in 60 decimal digits.

Its bound is 5e-16: of the polynomial 3.3e-16 at the ends of |r| <= ln 2 / 2
(where exp(r) is 0.71 or 1.41: half a step of it is 0.8e-16 of itself), of its
last step 0.8e-16, of the step before 0.3e-16, and of the rounding of r, half a
step of 0.35, 0.3e-16; further inside the polynomial is nearer, and half a step
is 1.1e-16.  The two parts of ln 2 leave 1e-30.
"""
import ctypes
import decimal
import os
import random
import subprocess

import pytest

from tests._tiles import CSRC

BOUND = decimal.Decimal("5e-16")
_SOURCE = """
#include <cmath>
#include "exp64.h"
using namespace latmoe;
extern "C" double own_exp(double x) {
  const double n = exp64_power(x);
  return std::ldexp(exp64_series(kExp64, exp64_rest(x, n)), (int)n);
}
"""


@pytest.fixture(scope="module")
def own_exp(tmp_path_factory):
    d = tmp_path_factory.mktemp("exp64")
    src, so = os.path.join(d, "t.cpp"), os.path.join(d, "t.so")
    with open(src, "w") as f:
        f.write(_SOURCE)
    subprocess.check_call(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", "-Wno-unknown-pragmas", "-ffp-contract=off", "-shared", "-fPIC", "-I", CSRC,
                           "-o", so, src])
    f = ctypes.CDLL(so).own_exp
    f.argtypes, f.restype = [ctypes.c_double], ctypes.c_double
    return f


@pytest.mark.parametrize("size", [1e-9, 0.3, 1.0, 10.0, 50.0, 300.0, 700.0])
def test_within_its_bound(own_exp, size):
    rng = random.Random(int(size * 100))
    with decimal.localcontext() as ctx:
        ctx.prec = 60
        for _ in range(1500):
            x = rng.choice([-1, 1]) * size * rng.uniform(0.8, 1.0)
            want = decimal.Decimal(x).exp()
            assert abs(decimal.Decimal(own_exp(x)) - want) <= want * BOUND, x


def test_ends_and_zero(own_exp):
    assert own_exp(0.0) == 1.0
    for x in (700.0, -700.0, 0.34657359027997264, -0.34657359027997264, 0.34657359027997270):
        want = decimal.Decimal(x).exp(decimal.Context(prec=60))
        assert abs(decimal.Decimal(own_exp(x)) / want - 1) <= BOUND
