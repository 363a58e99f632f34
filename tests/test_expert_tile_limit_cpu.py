"""The number of tiles of a launch from offsets of any value
(csrc/expert_rows.h), compiled with g++: all of them, or none where they reach
2^30, and never a part."""

import os
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_all_tiles_or_none(tmp_path):
    exe = str(tmp_path / "expert_tile_limit_check")
    src = os.path.join(ROOT, "tests", "c_abi", "expert_tile_limit_check.cpp")
    r = subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", "-ftrapv", src, "-o", exe],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([exe], capture_output=True, text=True)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stdout + r.stderr
