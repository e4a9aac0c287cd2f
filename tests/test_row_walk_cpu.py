"""Pad rows of a group up to the last row index that the calls accept (2^31 - 1)
are shared out within the group: the host code of the walk, compiled alone."""
import os
import re
import shutil
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "..", "precision_rl_amd", "csrc")
pytestmark = pytest.mark.cpu

LAST = 2 ** 31 - 1
# (first row, end, threads): no pads where T k = 2^31 - 128 rows fill their groups of 128
# exactly, up to 127 of them before the last index, with a lane a row (256 and 1024
# threads) and a wave a row (4, 16, and 64 waves of several workgroups)
CASES = [(LAST - 127, LAST - 127, n) for n in (256, 1024, 4, 16, 64)] + \
        [(LAST - 127, LAST, n) for n in (256, 1024, 4, 16, 64)] + \
        [(LAST - 1, LAST, 256), (LAST, LAST, 1024), (0, 0, 256), (5, 5, 4), (5, 132, 4), (5, 132, 256), (0, 127, 64)]


@pytest.mark.skipif(shutil.which("g++") is None, reason="needs a host C++ compiler")
def test_rows_of_a_group_are_visited_once_and_no_others(tmp_path):
    exe = str(tmp_path / "row_walk_check")
    # -fwrapv: a sum of 32 bits wraps here as it does on the GPU; conversions to 32 bits show in the values
    subprocess.run(["g++", "-O1", "-std=c++17", "-fwrapv", "-Wall", "-Werror", os.path.join(HERE, "row_walk_check.cpp"),
                    "-o", exe], check=True)
    # a walk in range takes at most 32 steps of a thread with 4 threads; 8 are followed, so those cases
    # are cut to the last rows
    cases = [(max(r0, r1 - 8 * n), r1, n) for r0, r1, n in CASES]
    out = subprocess.run([exe, *(str(v) for c in cases for v in c)], check=True, capture_output=True, text=True).stdout
    lines = [tuple(map(int, line.split())) for line in out.splitlines()]
    assert [line[:3] for line in lines] == cases
    for r0, r1, n, visited, inside in lines:
        assert inside and visited == r1 - r0, (r0, r1, n)


def test_the_kernels_use_this_walk():
    """Both loops over a group's pad rows of the dispatch, and no row counter of 32 bits beside it."""
    with open(os.path.join(CSRC, "dispatch.hip")) as f:
        text = f.read()
    assert len(re.findall(r"\bwalk_rows\(", text)) >= 2
    assert not re.search(r"for \(int r\b", text)
