"""Adapters and orthogonalised updates at the ends of what they take: many adapters
in random order over many tokens, and long matrices with a small side."""

import pytest

torch = pytest.importorskip("torch")

import tiled_gemm_tgemm_amd as tg  # noqa: E402
import test_gpu_linear_adapters as adapters  # noqa: E402
import test_gpu_orthogonalize_rounding as updates  # noqa: E402
from test_gpu_orthogonalize import TYPES, chain, error, gradient  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("size", [  # T, N, D, L, r
    (1100, 600, 200, 33, 16),       # more than the few adapters that one work-group groups
    (4096, 4096, 256, 64, 8),       # 256x256 tiles, whose rows are taken adapter by adapter
    (5000, 2048, 520, 300, 5),
    (2500, 130, 70, 700, 3),        # about as many adapters as an adapter has tokens, and fewer
    (8193, 264, 64, 17, 32),        # one past what one work-group groups
])
def test_many_adapters_in_random_order(size, dtype):
    args = adapters.layer(*size, dtype, 61, "random")
    first = adapters.check(args)
    again = adapters.check(args)
    assert torch.equal(first[0], again[0]) and all(torch.equal(a, b) for a, b in zip(first[1], again[1]))


@pytest.mark.parametrize("dtype", TYPES[:2])
def test_more_adapters_than_tokens(dtype):
    adapters.check(adapters.layer(200, 40, 24, 20000, 2, dtype, 62))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("shape", [(64, 1 << 17), ((1 << 17) + 3, 33), (7, 300001), (1, 1 << 20), (1 << 20, 2), (2, 16, 100003), (65, 1 << 16), (40003, 70)])
def test_a_small_side_and_a_long_one(shape, dtype):
    updates.check(gradient(shape, dtype, 63))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("shape", [(300, 65), (257, 700), (4, 130, 140), (1500, 1100)])
# (the last one's a is added to the products and not to Q's diagonal; three such steps would take singular values past
# 1000, which overflows: 2.9 after the first, 1580 after the second)
@pytest.mark.parametrize("coefficients", [updates.MUON, updates.PER_STEP[:3], [(20.0, -30.0, 11.0), (0.3, -0.01, 0.0), (1.5, -0.5, 0.0)]])
def test_the_same_bits_from_any_workspace(shape, dtype, coefficients):
    G, k = gradient(shape, dtype, 64), dict(steps=3, coefficients=coefficients)
    batch = shape[0] if len(shape) == 3 else 1
    need = tg.tgemm_orthogonalize_workspace_size({torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}[dtype], batch, *shape[-2:], 3)
    first = tg.orthogonalize(G, **k)
    for fill in (0xFF, 0x00):
        room = torch.full((need,), fill, dtype=torch.uint8, device="cuda")
        assert torch.equal(first, tg.orthogonalize(G, workspace=room, **k))
    assert first.isfinite().all() and error(first, chain(G, **k)) < 0.02


@pytest.mark.parametrize("dtype", TYPES[:2])
@pytest.mark.parametrize("sizes", [(600, 256, 192, 1000, 4, 16), (1300, 200, 264, 777, 2, 80)])
def test_updates_of_the_gradients_of_a_step(sizes, dtype):
    """Through a projection with adapters and an output head's loss: no further off than their rounding either."""
    from test_gpu_adapter_training import model, step

    args = model(*sizes, dtype, 65)
    args[2].requires_grad_(), args[3].requires_grad_()
    _, dA, dB, uA, uB = step(*args)
    for grad, got in ((dA, uA), (dB, uB)):
        updates.check(grad)
        assert torch.equal(got, tg.orthogonalize(grad))
