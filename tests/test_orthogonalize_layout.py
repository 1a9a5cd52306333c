"""Where the Newton-Schulz operator's matrices and its workspace lie, on the host."""

import pytest

import tiled_gemm_tgemm_amd as tg
from test_orthogonalize import lib  # noqa: F401  (the library is built)
from test_orthogonalize_walk import call, follow, walker  # noqa: F401


def test_results_side_by_side(walker):  # noqa: F811
    """Each row of a matrix next to the same row of the others: no address leaves the result's memory."""
    calls = []
    for dtype in (0, 1, 2):
        for batch, M, N, pad in [(3, 33, 70, 0), (4, 70, 33, 3), (3, 100, 131, 0), (5, 130, 90, 7), (2, 1, 9, 0), (7, 300, 65, 1)]:
            c = list(call(dtype, batch, M, N))
            c[8:10] = batch * N + pad, N
            calls.append(tuple(c))
    follow(walker, calls)
