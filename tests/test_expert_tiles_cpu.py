"""Row tiles of an expert from offsets of any value (csrc/expert_rows.h),
compiled with g++ and its overflow checks: counted without wrapping, and each
tile's rows inside the buffer."""

import os
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_tiles_of_wild_offsets(tmp_path):
    exe = str(tmp_path / "expert_tiles_check")
    src = os.path.join(ROOT, "tests", "c_abi", "expert_tiles_check.cpp")
    r = subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", "-ftrapv", src, "-o", exe],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([exe], capture_output=True, text=True)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stdout + r.stderr
