"""Indices that are not contiguous: the differentiable calls keep a copy for the
backward pass, which may run on another stream, late, when the graph that held
the copy is gone and its memory would be handed out again."""

import pytest

torch = pytest.importorskip("torch")

import tiled_gemm_tgemm_amd as tg  # noqa: E402
from test_gpu_linear_adapters import layer  # noqa: E402
from test_gpu_linear_loss_streams import later  # noqa: E402

pytestmark = pytest.mark.gpu


def strided(t):
    return torch.stack([t, t], dim=1)[:, 0]


def backward_under_a_late_stream(make, up):
    """The gradients of the result that make() gives, from its node by hand under a stream that is behind; the graph is
    dropped and memory of the copy's size allocated and written to before they are worked out."""
    result = make()
    side = torch.cuda.Stream()
    held = later(side)
    with torch.cuda.stream(side):
        got = result.grad_fn.apply(up)
    del result
    junk = [torch.zeros(up.shape[0] if up.dim() else 600, dtype=torch.int64, device="cuda") for _ in range(64)]
    torch.cuda.synchronize()
    del held, junk
    return got


@pytest.mark.parametrize("T", [90, 600, 1500])
def test_adapters(T):
    X, W, A, B, ids, scales, dY = layer(T, 256, 192, 3, 8, torch.bfloat16, 41)
    want = tg.linear_adapters_backward(dY, X, W, A, B, ids, scales=scales)
    leaves = [t.clone().requires_grad_() for t in (X, W, A, B)]
    got = backward_under_a_late_stream(lambda: tg.linear_adapters(*leaves, strided(ids), scales=scales), dY)
    assert all(torch.equal(a, b) for a, b in zip(got[:4], want))


def test_cross_entropy():
    T, V, D = 600, 9000, 256
    g = torch.Generator(device="cuda").manual_seed(42)
    X, W = (torch.randn(s, generator=g, device="cuda").bfloat16().requires_grad_() for s in ((T, D), (V, D)))
    target = torch.randint(0, V, (T,), generator=g, device="cuda")
    one = torch.ones((), device="cuda")
    want = torch.autograd.grad(tg.linear_cross_entropy(X, W, target), (X, W), one)
    got = backward_under_a_late_stream(lambda: tg.linear_cross_entropy(X, W, strided(target)), one)
    assert all(torch.equal(a, b) for a, b in zip(got[:2], want))
