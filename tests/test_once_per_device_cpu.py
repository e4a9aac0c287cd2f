"""What a kernel needs set on a device is set on every device the process launches on:
the host code that keeps count, compiled alone, and no other place that sets it."""
import os
import shutil
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "precision_rl_amd", "csrc")
pytestmark = pytest.mark.cpu


@pytest.mark.skipif(shutil.which("g++") is None, reason="needs a host C++ compiler")
def test_each_device_is_set_once(tmp_path):
    exe = str(tmp_path / "once_per_device_check")
    subprocess.run(["g++", "-O1", "-std=c++17", "-Wall", "-Werror", os.path.join(HERE, "once_per_device_check.cpp"),
                    "-o", exe], check=True)
    # (device, success, runs so far); a failure is tried again, and so is a device past the 64th
    steps = [(0, 1, 1), (0, 1, 1), (1, 1, 1), (0, 1, 1), (1, 1, 1), (63, 1, 1), (63, 1, 1), (64, 1, 1), (64, 1, 2),
             (-7, 0, 1), (-7, 0, 2), (7, 1, 3), (7, 1, 3)]
    out = subprocess.run([exe, *(str(s[0]) for s in steps)], check=True, capture_output=True, text=True).stdout
    assert [tuple(map(int, line.split())) for line in out.splitlines()] == [s[1:] for s in steps]


def test_lds_limits_are_set_per_device():
    for name in os.listdir(CSRC):
        with open(os.path.join(CSRC, name)) as f:
            text = f.read()
        assert "static const hipError_t" not in text, name
        assert ("hipFuncSetAttribute" in text) == (name == "internal.h"), name
