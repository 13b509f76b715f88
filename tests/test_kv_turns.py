"""The frequencies of rotary positions in turns (kv_plan.h, compiled by the
host compiler) against rational arithmetic."""
import os
import shutil
import subprocess
from fractions import Fraction

import pytest

from exact_angle import PI, cos_sin, turns

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "dynamic_quantized_gemm_amd", "csrc")
FREQS = [1.0, 0.7, 10000.0 ** -0.37, 1e-9, 1e3, 1e6, 123456789.123, 1e9, -1e9, 2.0 ** -30, 0.0, 1e-300]


def test_pi_and_the_reduction():
    assert 0 <= PI - Fraction("3.14159265358979323846264338327950288419716939937510") < Fraction(1, 10 ** 50)
    assert cos_sin(0, 0.3) == (1.0, 0.0)
    c, s = cos_sin(5, 0.25)
    assert abs(c - 0.3153223623952687) < 1e-15 and abs(s - 0.9489846193555862) < 1e-15


@pytest.mark.skipif(not shutil.which("g++"), reason="g++ not available")
def test_frequencies_in_turns(tmp_path):
    exe = str(tmp_path / "kv_turns_check")
    subprocess.run(["g++", "-std=c++17", "-O2", "-ffp-contract=off", "-Wall", "-Wextra", "-Werror", f"-I{CSRC}",
                    os.path.join(HERE, "kv_turns_check.cpp"), "-o", exe], check=True)
    out = subprocess.run([exe, *map(repr, FREQS)], capture_output=True, text=True, check=True, timeout=60).stdout
    for f, line in zip(FREQS, out.splitlines()):
        hi, lo = (float.fromhex(x) for x in line.split())
        # the position's 31 bits times this stay far below a turn; 2^-1074 is fp64's least step
        assert abs(Fraction(hi) + Fraction(lo) - turns(f)) <= abs(Fraction(f)) * Fraction(1, 2 ** 105) + Fraction(1, 2 ** 1073)
        assert abs(lo) <= abs(hi) * 2.0 ** -51 + 2.0 ** -1073
