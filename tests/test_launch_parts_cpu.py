"""Grids beyond what one launch holds (2^32 threads) are split: the host code of
the split, compiled alone."""
import os
import shutil
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
pytestmark = pytest.mark.cpu


@pytest.mark.skipif(shutil.which("g++") is None, reason="needs a host C++ compiler")
def test_parts_cover_the_grid_within_a_launch(tmp_path):
    exe = str(tmp_path / "launch_parts_check")
    subprocess.run(["g++", "-O1", "-std=c++17", "-Wall", "-Werror", os.path.join(HERE, "launch_parts_check.cpp"),
                    "-o", exe], check=True)
    # workgroups of 512: 2^30 + 300 rows in tiles of 128; of 256: 2^31 - 1 rows; of 1024: 2^30 columns in tiles of 256
    cases = [(512, 1, 1), (512, 2 ** 23 - 8, 1), (512, 2 ** 23 - 7, 2), (512, 2 ** 23 + 3, 2), (256, 2 ** 24, 2),
             (1024, 2 ** 22, 2), (1024, 2 ** 24 + 1, 5), (64, 1024, 1), (256, 0, 0)]
    out = subprocess.run([exe, *(str(v) for threads, total, _ in cases for v in (threads, total))], check=True,
                         capture_output=True, text=True).stdout
    lines = [tuple(map(int, line.split())) for line in out.splitlines()]
    assert [(t, n) for t, n, *_ in lines] == [(t, n) for t, n, _ in cases]
    for (threads, total, launches), (_, _, got, covered, most) in zip(cases, lines):
        assert got == launches and covered and most < 2 ** 32, (threads, total)
