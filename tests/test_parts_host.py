"""The rule for the parts of a contraction (csrc/kernels/parts.hpp), which several kernels work
out for themselves: compiled with and without fused multiply-adds, against exact fractions."""

import ctypes
import os
import shutil
import subprocess
from fractions import Fraction

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
KERNELS = os.path.join(ROOT, "w4a16_gemm_amd", "csrc", "kernels")

SOURCE = """
#include "parts.hpp"
extern "C" int parts_of(int rest, int most, int side, int outputs) { return w4a16::parts_of(rest, most, side, outputs); }
static_assert(w4a16::parts_of(4, 32, 32, 1 << 24) == 8, "a constant expression");
"""


@pytest.fixture(scope="module", params=["off", "fast"])
def rule(request, tmp_path_factory):
    if shutil.which("g++") is None:
        pytest.skip("g++ is not available")
    folder = tmp_path_factory.mktemp("parts")
    (folder / "parts.cpp").write_text(SOURCE)
    subprocess.run(["g++", "-std=c++17", "-O2", "-Wall", "-Werror", "-mfma", f"-ffp-contract={request.param}", "-shared", "-fPIC",
                    "-I", KERNELS, str(folder / "parts.cpp"), "-o", str(folder / "parts.so")], check=True)
    return ctypes.CDLL(str(folder / "parts.so")).parts_of


def exact(rest, most, side, outputs):
    """The parts of least time, of equal ones the fewest."""
    def time(f):
        rounds = Fraction(3, 5) if side == 64 and f * rest <= 32 else -(-f * rest // side)
        return Fraction(rounds) / f + Fraction(16 * rest * f, outputs)
    return min((f for f in range(1, most + 1) if f == 1 or f * rest <= 2 * side), key=lambda f: (time(f), f))


# near ties, where a fused and a plain multiply-add choose differently in 32-bit floats
TIES = [(1, 32, 896), (1, 32, 3840), (1, 32, 9600), (1, 32, 14880), (2, 32, 1792), (2, 32, 7680), (3, 32, 2688), (4, 32, 3584),
        (1, 64, 3520), (1, 64, 14720), (2, 64, 7040)]


@pytest.mark.parametrize("rest,side,outputs", TIES)
def test_near_ties(rule, rest, side, outputs):
    for most in range(1, 33):
        assert rule(rest, most, side, outputs) == exact(rest, most, side, outputs), most


@pytest.mark.parametrize("side", [32, 64])
def test_every_rest(rule, side):
    for rest in range(1, side):
        for outputs in (8, 64, 520, 1000, 1536, 4096, 8960, 10112, 11008, 14336, 28672, 151936, 1 << 20, (1 << 24) - 8, 1 << 24):
            for most in (1, 2, 7, 32):
                assert rule(rest, most, side, outputs) == exact(rest, most, side, outputs), (rest, outputs, most)


def test_nothing_left(rule):
    assert rule(0, 32, 32, 4096) == rule(0, 32, 64, 4096) == 1
