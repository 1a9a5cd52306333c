"""The Newton-Schulz operator without a GPU: every refusal comes back before
any HIP call, for the C entry point (with addresses that are never read) and
for the torch call."""

import ctypes
import os

import pytest

import tiled_gemm_tgemm_amd as tg
from tiled_gemm_tgemm_amd import _lib

OK, INVALID, UNSUPPORTED = tg.TGEMM_SUCCESS, tg.TGEMM_ERROR_INVALID_VALUE, tg.TGEMM_ERROR_NOT_SUPPORTED
G_, O_, WS = (i << 40 for i in range(1, 4))
BIG = 1 << 39
NUMBERS = (ctypes.c_float * 96)(*([3.4445, -4.775, 2.0315] * 32))


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not os.path.exists(_lib.LIBRARY):
        from tiled_gemm_tgemm_amd import build

        build.build()
    return tg.library()


def call(dtype=1, batch=2, M=100, N=80, G=G_, ldg=80, sg=8000, steps=5, numbers=NUMBERS, eps=1e-7, out=O_, ldo=80, so=8000, ws=WS,
         room=BIG):
    return tg.tgemm_orthogonalize(dtype, batch, M, N, G, ldg, sg, steps, numbers, eps, out, ldo, so, ws, room)


@pytest.mark.parametrize("change,status", [
    (dict(batch=-1), INVALID), (dict(M=-1), INVALID), (dict(N=-1), INVALID), (dict(steps=0), INVALID), (dict(steps=-3), INVALID),
    (dict(eps=-1e-7), INVALID), (dict(eps=float("inf")), INVALID), (dict(eps=float("nan")), INVALID), (dict(numbers=None), INVALID),
    (dict(ldg=79), INVALID), (dict(ldo=79), INVALID), (dict(sg=-1), INVALID), (dict(so=-1), INVALID),
    (dict(so=7999), INVALID),                      # results that overlap one another
    (dict(G=0), INVALID), (dict(out=0), INVALID), (dict(G=G_ + 1), INVALID), (dict(dtype=0, G=G_ + 2), INVALID),
    (dict(out=G_), INVALID), (dict(out=G_ + 2 * 15998), INVALID), (dict(ws=G_), INVALID), (dict(ws=O_), INVALID),
    (dict(ws=0), INVALID), (dict(ws=WS + 8), INVALID), (dict(room=1000), INVALID),
    (dict(G=(1 << 64) - 4096), INVALID),
    (dict(dtype=3), UNSUPPORTED), (dict(dtype=-1), UNSUPPORTED), (dict(batch=65536), UNSUPPORTED), (dict(steps=33), UNSUPPORTED),
    (dict(M=(1 << 20) + 1), UNSUPPORTED), (dict(N=(1 << 20) + 1, ldg=1 << 21, ldo=1 << 21), UNSUPPORTED),
    (dict(ldg=(1 << 40) + 1), UNSUPPORTED), (dict(so=(1 << 40) + 1), UNSUPPORTED),
    (dict(batch=0, G=0, out=0, ws=0, room=0), OK), (dict(M=0, G=0, out=0, ws=0, room=0), OK),
    (dict(N=0, ldg=0, ldo=0, G=0, out=0, ws=0, room=0), OK),
])
def test_refusals(change, status):
    assert call(**change) == status


def test_too_many_tiles_are_refused():
    # 4097x4097 tiles of 256 in each of 65535 matrices
    n = 1 << 20
    assert call(batch=65535, M=n, N=n, ldg=n, ldo=n, sg=0, so=1 << 40) == UNSUPPORTED
    assert tg.tgemm_orthogonalize_workspace_size(1, 65535, n, n, 5) == 0


def test_workspace_sizes():
    size = tg.tgemm_orthogonalize_workspace_size
    assert size(1, 0, 10, 10, 5) == size(1, 1, 0, 10, 5) == size(1, 1, 10, 10, 0) == size(7, 1, 10, 10, 5) == 0
    assert 0 < size(1, 1, 64, 4096, 5) < 1 << 20
    # two fp16 planes of X twice, of S and of Q
    exact = 2 * (2 * 2 * 1024 * 4096) + 2 * (2 * 2 * 1024 * 1024)
    assert exact <= size(1, 1, 1024, 4096, 5)
    assert size(1, 1, 4096, 1024, 5) >= exact and size(1, 1, 1024, 4096, 1) < size(1, 1, 1024, 4096, 2)
    assert size(0, 8, 1024, 4096, 5) >= 8 * exact


def test_the_torch_call_refuses():
    torch = pytest.importorskip("torch")
    t = torch.zeros
    with pytest.raises(TypeError):
        tg.orthogonalize(t(4, 4))  # the host's
    with pytest.raises(TypeError):
        tg.orthogonalize(t(4, 4, dtype=torch.float64))
    with pytest.raises(TypeError):
        tg.orthogonalize(t(4))
    with pytest.raises(TypeError):
        tg.orthogonalize([[1.0]])


def test_coefficients():
    from tiled_gemm_tgemm_amd import newton_schulz as ns

    one = ns._coefficients((1.0, 2.0, 3.0), 2)
    assert list(one) == [1, 2, 3, 1, 2, 3]
    assert list(ns._coefficients(((1.0, 2.0, 3.0), (4.0, 5.0, 6.0)), 2)) == [1, 2, 3, 4, 5, 6]
    with pytest.raises(ValueError):
        ns._coefficients(((1.0, 2.0, 3.0),), 2)
    with pytest.raises(ValueError):
        ns._coefficients((1.0, 2.0), 2)
