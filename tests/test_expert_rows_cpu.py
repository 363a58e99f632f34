"""The rows of an expert from two offsets of any value (csrc/expert_rows.h),
compiled with g++ and its overflow checks: always inside the buffer."""

import itertools
import os
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LOW, HIGH = -2 ** 31, 2 ** 31 - 1


def test_spans_stay_inside_the_buffer(tmp_path):
    exe = str(tmp_path / "expert_rows_check")
    src = os.path.join(ROOT, "tests", "c_abi", "expert_rows_check.cpp")
    r = subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", "-ftrapv", src, "-o", exe],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    ends = [LOW, LOW + 1, -400, -1, 0, 1, 3, 50, 399, 400, 401, 100000, HIGH - 1, HIGH]
    cases = list(itertools.product(ends, ends, [0, 1, 400, 2 ** 27]))
    r = subprocess.run([exe] + [str(v) for c in cases for v in c], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    got = [tuple(int(v) for v in line.split()) for line in r.stdout.splitlines()]
    assert len(got) == len(cases)
    for (begin, end, rows), (first, count) in zip(cases, got):
        want = min(max(begin, 0), rows)
        assert (first, count) == (want, max(min(end, rows) - want, 0)), (begin, end, rows)
