"""The remainder of a probability, max(p - A q, 0) in units of 2^-44, from the
kernel's own source compiled for the host: never negative, and near the exact
one."""
import ctypes
import os
import subprocess
from fractions import Fraction

import numpy as np
import pytest

from paged_kv_cache_177_gb300.build import CSRC
from tests.test_gpu_verify_exact import TINY

SOURCE = r"""
#include <cmath>
#include <cstdint>
#include <cstring>
static float __uint_as_float(uint32_t u) { float f; std::memcpy(&f, &u, 4); return f; }
static uint32_t __float_as_uint(float f) { uint32_t u; std::memcpy(&u, &f, 4); return u; }
static float __fmul_rn(float a, float b) { return a * b; }
using std::fmaf;
using std::fmaxf;
using std::fminf;
@BODY@
extern "C" long long remainder_units(float p, float q, long long a) { return residual(p, q, to_multiple(a)); }
"""


@pytest.fixture(scope="module")
def units(tmp_path_factory):
    with open(os.path.join(CSRC, "pkv_verify.cuh")) as f:
        text = f.read()
    body = text[text.index("using Fixed = long long;"):text.index("template <typename T>\n__device__ __forceinline__ float prob")]
    where = tmp_path_factory.mktemp("residual")
    src, so = where / "residual.cpp", where / "residual.so"
    src.write_text(SOURCE.replace("@BODY@", body.replace("__device__ __forceinline__ ", "static ")))
    # (no sum and product may be fused that the source does not fuse, as some hosts' compilers do)
    subprocess.check_call(["g++", "-O1", "-ffp-contract=off", "-std=c++17", "-shared", "-fPIC", str(src), "-o", str(so)])
    f = ctypes.CDLL(str(so)).remainder_units
    f.restype, f.argtypes = ctypes.c_longlong, [ctypes.c_float, ctypes.c_float, ctypes.c_longlong]
    return f


def test_what_came_out_below_zero(units):
    one = 1 << 44
    for a, p, q in ([float.fromhex(x) for x in t] for t in TINY):
        cut = lambda x: int(round(Fraction(x) * one))
        big_a = one + 4 * (cut(a) - cut(0.25)) + cut(p) - cut(q)
        assert units(a, 0.25, big_a) == 0
        assert 0 < Fraction(p) * one - Fraction(big_a, one) * Fraction(q) * one < 1 and units(p, q, big_a) == 0


def test_next_to_nothing(units):
    """p around A q, of every magnitude: not negative, and within 2 units of the exact remainder (p, and A q in two parts,
    are rounded to units, half a unit each; A q is 2^-48 of it off; less than a unit counts as 0)."""
    rng = np.random.default_rng(2)
    one = 1 << 44
    seen = 0
    for _ in range(60000):
        big_a = one + int(rng.integers(0, 1 << int(rng.integers(1, 46))))
        q = np.float32(2.0 ** -rng.uniform(2, 40))
        p = np.float32(float(Fraction(big_a, one) * Fraction(float(q))))
        for _ in range(int(rng.integers(0, 3))):
            p = np.nextafter(p, np.float32(rng.integers(0, 2)))
        got = units(p, q, big_a)
        exact = max(Fraction(float(p)) * one - big_a * Fraction(float(q)), Fraction(0))
        assert got >= 0 and abs(got - exact) <= 2, (p, q, big_a)
        seen += got > 0
    assert seen > 1000
