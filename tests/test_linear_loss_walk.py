"""Every address that the loss operators' loads and stores reach, followed on
the host (tests/linear_loss_walk.cpp): the entry points' own plans and the
loads' own walk, with the kernels' launches replaced by checks that each access
lies in what the call was given."""

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
           f"-I{ROOT}/include", f"-I{CSRC}", os.path.join(CSRC, "linear_loss.cpp"),
           os.path.join(ROOT, "tests", "linear_loss_walk.cpp"), "-o", out]
    subprocess.run(cmd, check=True)
    return out


def follow(walker, calls):
    text = "".join(" ".join(map(str, c)) + "\n" for c in calls)
    r = subprocess.run([walker], input=text, capture_output=True, text=True)
    assert r.returncode == 0, r.stdout[-2000:] + r.stderr[-500:]
    assert r.stdout.startswith(f"{len(calls)} calls")


def call(op, backward, dtype, T, V, D, pad_x=0, pad_w=0, shift_x=0, shift_w=0, K=5, need_x=1, need_w=1, pad_dx=0, pad_dw=0):
    return (op, backward, dtype, T, V, D, D + pad_x, D + pad_w, shift_x, shift_w, K, need_x, need_w, D + pad_dx, D + pad_dw)


# rows around the tiles' and the steps' sizes, words and widths likewise
ROWS = [1, 16, 31, 32, 33, 63, 64, 65, 96, 97, 128, 129, 200, 256, 257, 300, 700, 2100]
WORDS = [1, 63, 64, 65, 127, 128, 129, 255, 257, 1000, 5003]
WIDTHS = [1, 7, 8, 63, 64, 72, 128, 200, 1000]


@pytest.mark.parametrize("dtype", [0, 1, 2])
@pytest.mark.parametrize("op", [0, 1])
def test_sizes_around_the_tiles(walker, dtype, op):
    r = random.Random(dtype * 2 + op)
    calls = []
    for T in ROWS:
        for V in WORDS:
            D = r.choice(WIDTHS)
            for backward in (0, 1):
                calls.append(call(op, backward, dtype, T, V, D))
    follow(walker, calls)


@pytest.mark.parametrize("dtype", [0, 1, 2])
def test_strides_alignment_and_parts_of_a_call(walker, dtype):
    r = random.Random(10 + dtype)
    calls = []
    for _ in range(150):
        T, V, D = r.choice(ROWS), r.choice(WORDS), r.choice(WIDTHS)
        pads = [r.choice([0, 1, 4, 8, 24]) for _ in range(4)]
        shifts = [r.choice([0, 1, 4, 8]) for _ in range(2)]
        need = r.choice([(1, 1), (1, 0), (0, 1)])
        for backward in (0, 1):
            calls.append(call(r.randint(0, 1), backward, dtype, T, V, D, pads[0], pads[1], *shifts, r.choice([1, 3, 64, 1024]),
                              *need, pads[2], pads[3]))
    follow(walker, calls)


@pytest.mark.parametrize("dtype", [0, 1, 2])
def test_large_sizes(walker, dtype):
    calls = []
    for T, V, D in [(1, 131072, 4096), (33, 32000, 4096), (8192, 20003, 64), (4096, 32768, 2048), (8192, 131072, 4096),
                    (20000, 5000, 1000), (512, 16384, 1024), (65, 1 << 20, 64), (5, 1 << 24, 8), (100000, 300, 64),
                    (3, 1000, 1 << 20)]:
        for backward in (0, 1):
            calls.append(call(0, backward, dtype, T, V, D))
    follow(walker, calls)


def test_random_sizes(walker):
    r = random.Random(99)
    calls = []
    for _ in range(400):
        T, V, D = (int(2 ** r.uniform(0, 11)) for _ in range(3))
        calls.append(call(r.randint(0, 1), r.randint(0, 1), r.randint(0, 2), T, V, D, K=r.randint(1, 100)))
    follow(walker, calls)
