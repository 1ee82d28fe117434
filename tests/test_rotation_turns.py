"""The frequencies of the position rotation, compiled alone, against 80 digits (no GPU)."""

import ctypes
import struct
import subprocess
from decimal import Decimal, getcontext

import pytest

from speculative_drafting_pe_gb300 import build

TWO_PI = 2 * Decimal("3.14159265358979323846264338327950288419716939937510582097494459230781640628620899862803482534")


@pytest.fixture(scope="module")
def turns(tmp_path_factory):
    at = tmp_path_factory.mktemp("rotation")
    (at / "turns.cpp").write_text('#include "rotation.h"\n'
                                  'extern "C" void turns(float theta, int hd, unsigned long long* out) {\n'
                                  '    pe::rotation_turns(theta, hd, out);\n}\n')
    subprocess.run(["g++", "-O3", "-std=c++17", "-shared", "-fPIC", "-I" + build.CSRC, str(at / "turns.cpp"), "-o",
                    str(at / "turns.so")], check=True)
    lib = ctypes.CDLL(str(at / "turns.so"))

    def call(theta, hd):
        out = (ctypes.c_uint64 * 64)()
        lib.turns(ctypes.c_float(theta), hd, out)
        return list(out)[:hd // 2]
    return call


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("theta", [1.0, 1.0000001, 2.0, 1e4, 150000.0, 5e5, 1e6, 12345.678, 3e38])
def test_turns_per_position(turns, theta, hd):
    getcontext().prec = 80
    exact = Decimal(struct.unpack("f", struct.pack("f", theta))[0])
    for i, got in enumerate(turns(theta, hd)):
        want = exact ** (Decimal(-2 * i) / hd) / TWO_PI * 2 ** 64
        # the nearest whole number, but for what the products of some 2^-100 of themselves each move
        assert abs(got - want) <= Decimal(0.5) + Decimal(2) ** -30, i


def test_a_base_after_another(turns):
    first = turns(1e4, 128)
    assert turns(1e6, 128) != first and turns(1e4, 128) == first and turns(1e4, 64) == first[::2]
