"""The loss operators at sizes whose logits would not fit a GPU many times over."""

import pytest

torch = pytest.importorskip("torch")

import tiled_gemm_tgemm_amd as tg  # noqa: E402
from loss_reference import Reference  # noqa: E402
from test_gpu_linear_loss import gpu, log  # noqa: E402,F401

pytestmark = pytest.mark.gpu


def test_more_tiles_than_2_to_the_23rd():
    """2^22 rows of 2^17 words (2^39 logits, 64 GiB of partial statistics): rows from all over against 64 bits."""
    T, V, D = 1 << 22, 1 << 17, 64
    if torch.cuda.mem_get_info()[0] < 90 << 30:
        pytest.skip("needs 90 GiB of free memory")
    log(f"{T}x{V}x{D}")
    g = torch.Generator(device="cuda").manual_seed(51)
    X = torch.randn((T, D), generator=g, device="cuda", dtype=torch.bfloat16)
    W = torch.randn((V, D), generator=g, device="cuda", dtype=torch.bfloat16) * 0.25
    y = torch.randint(0, V, (T,), generator=g, device="cuda")
    loss, lse = tg.linear_cross_entropy_forward(X, W, y)
    torch.cuda.synchronize()
    rows = torch.cat([torch.tensor([0, 255, 256, T // 2 - 1, T // 2, T - 257, T - 256, T - 1], device="cuda"),
                      torch.randint(0, T, (120,), generator=g, device="cuda")])
    Reference(X[rows], W, y[rows]).check_rows(loss[rows], lse[rows])
    assert bool(torch.isfinite(loss).all())
    torch.cuda.empty_cache()
