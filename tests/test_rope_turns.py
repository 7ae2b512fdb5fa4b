"""The rotation's frequencies of the decoder calls (csrc/rope_turns.h, host code)
against 60-digit arithmetic."""
import ctypes
import os
import subprocess
from decimal import Decimal, getcontext

import numpy as np
import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PI = Decimal("3.14159265358979323846264338327950288419716939937510582097494459230781640628620899862803")
SOURCE = """
#include "%s"
extern "C" void turns(double base, int rope_dims, double* hi, float* lo) {
  vattn::host::rope_turns(base, rope_dims, hi, lo);
}
"""


@pytest.fixture(scope="module")
def turns(tmp_path_factory):
    d = tmp_path_factory.mktemp("turns")
    header = os.path.join(ROOT, "vision_encoder_flash_gb300", "csrc", "rope_turns.h")
    (d / "turns.cpp").write_text(SOURCE % header)
    subprocess.run(["g++", "-O3", "-std=c++17", "-shared", "-fPIC", "-o", str(d / "turns.so"), str(d / "turns.cpp")],
                   check=True)
    lib = ctypes.CDLL(str(d / "turns.so"))

    def run(base, rope_dims):
        hi, lo = np.zeros(64), np.zeros(64, np.float32)
        lib.turns(ctypes.c_double(base), ctypes.c_int(rope_dims), ctypes.c_void_p(hi.ctypes.data),
                  ctypes.c_void_p(lo.ctypes.data))
        return hi, lo

    return run


@pytest.mark.parametrize("base", [10000.0, 500000.0, 1e6, 1.0, 2.0, 0.001, 1e-12, 1e12, 1.0000001, 1e300, 1e-200, 3.7e17])
@pytest.mark.parametrize("rope_dims", [1, 2, 3, 48, 64, 72, 127, 128])
def test_more_digits_than_a_double(turns, base, rope_dims):
    getcontext().prec = 60
    hi, lo = turns(base, rope_dims)
    half = rope_dims // 2
    assert not hi[half:].any() and not lo[half:].any()
    for i in range(half):
        want = (Decimal(base).ln() * Decimal(-2 * i) / Decimal(rope_dims)).exp() / (2 * PI)
        got = Decimal(float(hi[i])) + Decimal(float(lo[i]))
        # lo has 24 digits below hi's 53; what is computed is good to some 2^-95
        if want < 2 ** 59:
            assert abs(got - want) <= want * Decimal(2) ** -76 + Decimal(2) ** -140, (i, got, want)
        else:
            assert np.isfinite(hi[i]) and lo[i] in (0, np.float32(lo[i]))
