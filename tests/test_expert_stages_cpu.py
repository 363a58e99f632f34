"""Stages of a sum of up to 2^31 - 1 rows (csrc/expert_rows.h), which the
weights' gradient takes where rows are narrow enough, compiled with g++ and
its overflow checks."""

import os
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_stages_of_the_longest_sums(tmp_path):
    exe = str(tmp_path / "expert_stages_check")
    src = os.path.join(ROOT, "tests", "c_abi", "expert_stages_check.cpp")
    r = subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", "-ftrapv", src, "-o", exe],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([exe], capture_output=True, text=True)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stdout + r.stderr
