"""The paged cache's index arithmetic on the CPU: kv_plan.h, which the kernels
include as it is, compiled by the host compiler with its sanitizers and
checked exhaustively over small sizes, bad block table entries among them."""
import os
import shutil
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "dynamic_quantized_gemm_amd", "csrc")


def test_rows_pairs_and_shares(tmp_path):
    if not shutil.which("g++"):
        pytest.skip("g++ not available")
    exe = str(tmp_path / "kv_plan_check")
    subprocess.run(["g++", "-std=c++17", "-O1", "-g", "-Wall", "-Wextra", "-Werror", "-fsanitize=address,undefined",
                    "-fno-sanitize-recover=all", f"-I{CSRC}", os.path.join(HERE, "kv_plan_check.cpp"), "-o", exe],
                   check=True)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=300,
                       env={**os.environ, "ASAN_OPTIONS": "detect_leaks=0"})
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stdout + r.stderr
