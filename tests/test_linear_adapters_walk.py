"""Every address that the loads and stores of the projection with adapters
reach, followed on the host (tests/linear_adapters_walk.cpp): the entry points'
own plans and the loads' own walk, with the kernels' launches replaced by checks
that each access lies in what the call was given."""

import os
import random
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "tiled_gemm_tgemm_amd", "csrc")


@pytest.fixture(scope="module")
def walker(tmp_path_factory):
    if not shutil.which("g++") or not os.path.isdir("/opt/rocm/include/hip"):
        pytest.skip("g++ and the HIP headers are needed")
    out = str(tmp_path_factory.mktemp("walk") / "walk")
    cmd = ["g++", "-O2", "-std=c++17", "-Wall", "-Werror", "-D__HIP_PLATFORM_AMD__", "-isystem", "/opt/rocm/include",
           f"-I{ROOT}/include", f"-I{CSRC}", os.path.join(CSRC, "linear_adapters.cpp"),
           os.path.join(ROOT, "tests", "linear_adapters_walk.cpp"), "-o", out]
    subprocess.run(cmd, check=True)
    return out


def follow(walker, calls):
    text = "".join(" ".join(map(str, c)) + "\n" for c in calls)
    r = subprocess.run([walker], input=text, capture_output=True, text=True)
    assert r.returncode == 0, r.stdout[-2000:] + r.stderr[-500:]
    assert r.stdout.startswith(f"{len(calls)} calls")


def call(need, dtype, T, N, D, L=3, r=8, pads=(0, 0, 0, 0, 0), shift=0, hidden=1):
    return (need, dtype, T, N, D, L, r, *pads, shift, hidden)


ROWS = [1, 16, 17, 64, 65, 96, 128, 129, 200, 256, 257, 300, 700, 2100]
SIDES = [1, 7, 8, 63, 64, 65, 72, 128, 129, 257, 1000]


@pytest.mark.parametrize("dtype", [0, 1, 2])
def test_sizes_around_the_tiles(walker, dtype):
    r = random.Random(dtype)
    follow(walker, [call(need, dtype, T, N, r.choice(SIDES), r.choice([1, 3, 20]), r.choice([1, 8, 10, 33, 64]))
                    for T in ROWS for N in SIDES for need in (0, 15)])


@pytest.mark.parametrize("dtype", [0, 1, 2])
def test_strides_alignment_and_parts_of_a_call(walker, dtype):
    r = random.Random(10 + dtype)
    follow(walker, [call(r.choice([0, 0, 0, *range(1, 16)]), dtype, r.choice(ROWS), r.choice(SIDES), r.choice(SIDES), r.choice([1, 2, 50]),
                         r.choice([1, 4, 16, 40, 200]), [r.choice([0, 1, 4, 8, 24]) for _ in range(5)], r.choice([0, 1, 4, 8]), r.randint(0, 1))
                    for _ in range(400)])


def test_no_rows(walker):
    follow(walker, [call(need, dtype, 0, 70, 90) for need in (2, 4, 8, 15) for dtype in (0, 1)])


def test_large_sizes(walker):
    sizes = [(1, 4096, 4096, 8, 16), (48, 8192, 2048, 32, 16), (8192, 16384, 4096, 8, 32), (8192, 64, 16384, 1, 1024), (65, 200000, 64, 4, 4),
             (100000, 300, 64, 32767, 1), (131100, 300, 64, 32767, 1), (20000, 5000, 1000, 1000, 16), (513, 72, 1 << 18, 2, 128),
             (2048, 1024, 1024, 2, 8), (4100, 320, 448, 3, 40), (1025, 64, 64, 1, 16)]
    follow(walker, [call(need, dtype, *s) for need in (0, 15) for dtype in (0, 1) for s in sizes])
