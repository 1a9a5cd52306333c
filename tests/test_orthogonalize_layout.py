"""Where the Newton-Schulz operator's matrices and its workspace lie, on the host."""

import random

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


def test_the_workspace_is_what_the_header_says(lib):  # noqa: F811
    up = lambda v: (v + 63) // 64 * 64
    r = random.Random(0)
    for _ in range(1000):
        dtype, batch, steps = r.randint(0, 2), r.choice([1, 1, 2, 8, 24, 100]), r.choice([1, 5])
        M, N = (int(65 * 2 ** (8 * r.random())) for _ in range(2))
        need = tg.tgemm_orthogonalize_workspace_size(dtype, batch, M, N, steps)
        planes = (8 if steps > 1 else 4)
        assert batch * (planes * M * N + 8 * min(M, N) ** 2) <= need
        assert need <= batch * (planes * up(M) * up(N) + 8 * up(min(M, N)) ** 2 + 1024) + (1 << 28)
    for M, N, steps in ((8192, 8192, 5), (4096, 16384, 5), (8192, 8192, 1)):
        exact = (8 if steps > 1 else 4) * M * N + 8 * min(M, N) ** 2
        assert exact <= tg.tgemm_orthogonalize_workspace_size(1, 1, M, N, steps) <= 1.25 * exact
    assert tg.tgemm_orthogonalize_workspace_size(1, 1, 300, 1000, 5) <= 8 * 320 * 1024 + 8 * 320 ** 2 + (4 << 20)
