"""Stacks of matrices that lie side by side, each row of one next to the same row of
the others, as operands and as results; and those that share elements."""

import pytest

torch = pytest.importorskip("torch")

import tiled_gemm_tgemm_amd as tg  # noqa: E402
from test_gpu_linear_adapters import layer  # noqa: E402
from test_gpu_orthogonalize import TYPES, gradient  # noqa: E402

pytestmark = pytest.mark.gpu


def beside(t, more=0):
    """The same stack side by side, `more` elements after each row of all, and the memory, in which those hold 7."""
    count, rows, cols = t.shape
    room = torch.full((rows, count * cols + more), 7.0, dtype=t.dtype, device="cuda")
    inner = room[:, :count * cols].unflatten(1, (count, cols)).transpose(0, 1)
    inner.copy_(t)
    assert rows == 1 or inner.stride() == (cols, count * cols + more, 1)
    return inner, room


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("shape", [(3, 33, 70), (4, 70, 33), (3, 100, 131), (5, 130, 90), (2, 1, 9)])
@pytest.mark.parametrize("more", [0, 5])
def test_updates(shape, dtype, more):
    G = gradient(shape, dtype, 51)
    want = tg.orthogonalize(G)
    out, room = beside(torch.zeros_like(G), more)
    assert tg.orthogonalize(beside(G, more)[0], out=out) is out
    assert torch.equal(out, want) and bool((room[:, room.shape[1] - more:] == 7).all())


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T", [20, 150, 1300])
@pytest.mark.parametrize("more", [0, 8])
def test_adapters(T, dtype, more):
    X, W, A, B, ids, scales, dY = layer(T, 96, 64, 3, 16, dtype, 52)
    want = tg.linear_adapters_backward(dY, X, W, A, B, ids, scales=scales)
    (dA, room_a), (dB, room_b) = beside(torch.zeros_like(A), more), beside(torch.zeros_like(B), more)
    got = tg.linear_adapters_backward(dY, X, W, beside(A, more)[0], beside(B, more)[0], ids, scales=scales, dA=dA, dB=dB)
    assert got[2] is dA and got[3] is dB
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    for room in (room_a, room_b):
        assert bool((room[:, room.shape[1] - more:] == 7).all())
    assert torch.equal(tg.linear_adapters(X, W, beside(A, more)[0], beside(B, more)[0], ids, scales=scales),
                       tg.linear_adapters(X, W, A, B, ids, scales=scales))


def test_results_that_share_elements_are_refused():
    G = gradient((3, 40, 50), torch.float32, 53)
    for strides in ((0, 50, 1), (49, 150, 1), (50, 149, 1), (40 * 50 - 1, 50, 1), (50, 50, 1)):
        out = torch.empty(3 * 40 * 60, device="cuda").as_strided((3, 40, 50), strides)
        with pytest.raises(tg.TgemmError):
            tg.orthogonalize(G, out=out)
    X, W, A, B, ids, scales, dY = layer(30, 96, 64, 3, 16, torch.float32, 54)
    for strides in ((0, 64, 1), (63, 192, 1), (64, 191, 1)):
        with pytest.raises(tg.TgemmError):
            tg.linear_adapters_backward(dY, X, W, A, B, ids, dA=torch.empty(3 * 16 * 80, device="cuda").as_strided((3, 16, 64), strides))
