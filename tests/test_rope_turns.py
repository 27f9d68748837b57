"""The rotation's frequencies as 64-bit fractions of a turn (rope_turns.h, host code): against integers."""
import ctypes
import os
import shutil
import subprocess
from fractions import Fraction

import numpy as np
import pytest

from exact_io_aware_06_gb300 import _build


@pytest.fixture(scope="module")
def turns(tmp_path_factory):
    d = tmp_path_factory.mktemp("turns")
    src, out = d / "t.cpp", d / "t.so"
    src.write_text('#include "rope_turns.h"\n'
                   'extern "C" void turns(const double* f, uint64_t* t, int n) {\n'
                   '    for (int i = 0; i < n; ++i) t[i] = fa::rope_turns(f[i]);\n}\n')
    cxx = os.environ.get("CXX") or shutil.which("g++")
    subprocess.run([cxx, "-O2", "-std=c++17", "-Wall", "-Werror", "-shared", "-fPIC", "-I", _build.CSRC, str(src), "-o", str(out)],
                   check=True)
    fn = ctypes.CDLL(str(out)).turns

    def call(f):
        f, t = np.ascontiguousarray(f, dtype=np.float64), np.zeros(len(f), dtype=np.uint64)
        fn(f.ctypes.data_as(ctypes.c_void_p), t.ctypes.data_as(ctypes.c_void_p), len(f))
        return t

    return call


def two_pi(bits):
    """2 pi 2^bits by Machin's formula, off by a few hundred."""
    atan = lambda x: sum((-1) ** k * ((1 << bits) // ((2 * k + 1) * x ** (2 * k + 1))) for k in range(bits // 4))  # noqa: E731
    return 8 * (4 * atan(5) - atan(239))


def test_fractions_of_a_turn(turns):
    rng = np.random.default_rng(1)
    f = np.concatenate([[0.0, 1.0, -1.0, 5e-324, -5e-324, 2.0 ** 64, -2.0 ** 64, 2.0 ** -64, 2 * np.pi, np.pi, np.nextafter(2.0 ** 64, 0)],
                        10000.0 ** -(np.arange(64) / 64), 2.0 ** np.arange(-90, 65), 10.0 ** np.arange(0, 20),
                        rng.standard_normal(2000) * 2.0 ** rng.integers(-80, 61, 2000)])
    pi2 = two_pi(700)
    one = 1 << 64
    for x, got in zip(f, turns(f)):
        q = Fraction(float(x)) * (1 << 700) / pi2  # turns, to 2^-600
        off = (Fraction(int(got)) - q * one) % one
        off = min(off, one - off)
        assert off < 4, (x, float(off))  # units of 2^-64: five pieces rounded by half of one each
