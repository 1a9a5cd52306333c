"""Which sizes the loss operators take, and what they plan for them."""

import os
import shutil
import subprocess

import pytest

import tiled_gemm_tgemm_amd as tg
from test_linear_loss import BIG, ce_forward, kd_forward, lib, size  # noqa: F401
from test_linear_loss_walk import CSRC


@pytest.mark.parametrize("T,V,D", [(1 << 22, 131072, 64), (1 << 20, 1 << 20, 64), ((1 << 24) - 1, 1 << 22, 8), (1 << 20, 131072, 4096)])
@pytest.mark.parametrize("dtype", [0, 1, 2])
def test_many_tiles_are_taken(T, V, D, dtype):
    for K in (0, 5):
        assert size(dtype=dtype, T=T, V=V, D=D, ldx=D, ldw=D, K=K) > T * V // 8  # a pair of floats a row and 64 words
        assert size(dtype=dtype, T=T, V=V, D=D, ldx=D, ldw=D, K=K, backward=1) > 0


@pytest.mark.parametrize("call", [ce_forward, kd_forward])
def test_too_many_tiles_are_refused(call):
    # 2^16 by 2^15 tiles of 256×256 and one row of tiles fewer; the latter is taken but for its workspace
    T, V = (1 << 24) - 1, 1 << 23
    assert call(T=T, V=V) == tg.TGEMM_ERROR_NOT_SUPPORTED and size(T=T, V=V) == 0
    assert size(T=T - 256, V=V) > BIG and call(T=T - 256, V=V) == tg.TGEMM_ERROR_INVALID_VALUE


def test_a_tiles_place(tmp_path):
    if not shutil.which("g++"):
        pytest.skip("g++ is needed")
    out = str(tmp_path / "place")
    subprocess.run(["g++", "-O1", "-std=c++17", "-Wall", "-Werror", "-fsanitize=undefined", "-fno-sanitize-recover=all", f"-I{CSRC}",
                    os.path.join(os.path.dirname(__file__), "tile_place.cpp"), "-o", out], check=True)
    products = [(1, 1, 1), (1, 9, 3), (8, 8, 1), (9, 7, 5), (65535, 32768, 1), (16384, 512, 1), (32768, 65535, 1),
                (1024, 32767, 64), (46340, 46340, 1)]
    r = subprocess.run([out], input="".join("%d %d %d\n" % p for p in products), capture_output=True, text=True)
    assert r.returncode == 0 and r.stdout == f"{len(products)} products\n", (r.returncode, r.stderr[-500:])


@pytest.mark.parametrize("dtype,value", [(0, 6), (1, 2), (2, 2)])
@pytest.mark.parametrize("T", [1000, 21000, 65536, 100000, 262144, 1 << 20])
@pytest.mark.parametrize("V,D", [(131072, 64), (32768, 1024), (1000, 256)])
def test_what_a_backward_call_holds(dtype, value, T, V, D):
    """A piece of the logits' gradient as tgemm.h bounds it (a row of it is up to 128 words longer than its words, a
    multiple of 256), X, and the sums of dX and dW, which are taken in parts where their tiles are few."""
    piece = max(256 << 20, 2048 * T * value, 256 * T * value)
    piece = min(piece, (V + 255) // 256 * 256 * T * value) + 128 * (T + 64) * value
    x = (T + 64) * D * (6 if dtype == 0 else 2)
    w = V * D * 6 if dtype == 0 else 0
    need = size(dtype=dtype, T=T, V=V, D=D, ldx=D, ldw=D, backward=1)
    sums = need - (piece + x + w + 12 * (T + 64) + 4096)
    # in parts only up to a few rounds of the 256 tiles of 256×256 that the GPU holds
    rounds = 4 * 256 * 256 * 256 * 4
    assert sums <= max(4 * (T + 64) * D, rounds) + rounds
    if T >= 262144 and dtype:
        assert need >= min(V, 2048) * T * value


@pytest.mark.parametrize("V,D", [(5000, 1000), (131072, 4096)])
def test_what_operands_take(V, D):
    """tgemm.h: float32 in planes, 16-bit ones that lie apart in a copy, others and few rows nothing."""
    T, planes = 64, 6 * V * D
    at = dict(T=T, V=V, D=D, ldx=D, ldw=D)
    apart = dict(at, ldw=D + 1)
    for backward in (0, 1):
        stored, copied, float32 = (size(**a, backward=backward) for a in (at, apart, dict(at, dtype=0)))
        assert 2 * V * D <= copied - stored <= 2 * V * (D + 64) and planes <= float32
    assert size(**dict(at, T=32, dtype=0)) < planes // 6


def test_outputs_between_an_inputs_rows_are_refused():
    """tgemm.h: arrays are taken with what lies between their rows."""
    from test_linear_loss import DX, X_, ce_backward

    assert ce_backward(ldx=128, dX=X_ + 128, lddx=128) == tg.TGEMM_ERROR_INVALID_VALUE
    assert ce_backward(dX=DX, lddx=128, dW=DX + 128, lddw=128) == tg.TGEMM_ERROR_INVALID_VALUE

