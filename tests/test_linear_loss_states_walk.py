"""As test_linear_loss_walk.py, for the states that fp16 rows' factors are joined with."""

import os
import subprocess

import pytest

from test_linear_loss_walk import CSRC, ROOT, call, follow, shutil


@pytest.fixture(scope="module")
def walker(tmp_path_factory):
    if not shutil.which("g++") or not os.path.isdir("/opt/rocm/include/hip"):
        pytest.skip("g++ and the HIP headers are needed")
    out = str(tmp_path_factory.mktemp("walk") / "walk")
    subprocess.run(["g++", "-O2", "-std=c++17", "-Wall", "-Werror", "-D__HIP_PLATFORM_AMD__", "-isystem", "/opt/rocm/include",
                    f"-I{ROOT}/include", f"-I{CSRC}", os.path.join(CSRC, "linear_loss.cpp"),
                    os.path.join(ROOT, "tests", "linear_loss_states_walk.cpp"), "-o", out], check=True)
    return out


@pytest.mark.parametrize("op", [0, 1])
def test_states_of_rows_with_factors(walker, op):
    # without dX the calls that are followed have a factor a row
    follow(walker, [call(op, 1, 2, T, V, D, pad_x=pad, shift_x=shift, need_x=0)
                    for T in (1, 15, 16, 17, 33, 128, 300, 70000) for V, D in ((5, 1), (100, 7), (300, 64), (65, 1000))
                    for pad, shift in ((0, 0), (3, 1), (24, 8))])
