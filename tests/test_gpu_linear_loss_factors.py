"""The gradients of rows whose factors are far apart: each row's part is as
exact as if the others were not there."""

import pytest

torch = pytest.importorskip("torch")

import tiled_gemm_tgemm_amd as tg  # noqa: E402
from loss_reference import Reference  # noqa: E402
from test_gpu_linear_loss import TYPES, gpu, log  # noqa: E402,F401

pytestmark = pytest.mark.gpu


def lone_words(T, V, D, dtype, spread, seed, outlier=0):
    """The first half of the rows have a factor of 2^16 (a loss scale), the others one of about 2^(16 - spread); the
    words of the latter are none of the former's, whose probability of them is 0: exp(-100) and less.  outlier: rows of
    the second half whose states are 2^outlier times as large."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    half, words = T // 2, V // 2
    X = torch.randn((T, D), generator=g, device="cuda")
    W = torch.randn((V, D), generator=g, device="cuda") * (2.0 / D ** 0.5)
    X[:half, 0], X[half:, 0] = 16.0, 0.0
    W[:words, 0], W[words:, 0] = 0.0, -8.0
    if outlier:
        X[half::3] *= 2.0 ** outlier
        W[:, 1:] *= 2.0 ** -outlier
    y = torch.cat([torch.randint(0, words, (half,), generator=g, device="cuda"),
                   torch.randint(words, V, (T - half,), generator=g, device="cuda")])
    grad = torch.full((T,), 2.0 ** 16, device="cuda") * (1.0 + torch.rand(T, generator=g, device="cuda"))
    grad[half:] *= 2.0 ** -torch.randint(spread - 2, spread + 1, (T - half,), generator=g, device="cuda").double()
    return X.to(dtype), W.to(dtype), y, grad


def check(ref, X, grad, dX, dW):
    """The tolerance of each power of two's rows alone, added up.  In fp16 the rows share the range of dW's operand: with
    the factors f·2^e and the largest states h·2^m of the rows (f and h at least 1/2 and below 1) each is scaled by
    2^(15 + e - top), top the largest e + m.  That is exact but for a rounding of at most 2^-25 below the normal
    numbers, which meets up to 2^15 of dz and 2^(top - 30): 2^(top - 40), at most 2^-38 of the largest factor times
    state, for each row's own part of dz."""
    power = torch.frexp(grad)[1]
    off_x, off_w = 0.0, 0.0
    for p in power.unique().tolist():
        part = torch.where(power == p, grad, 0.0).double()
        _, ox, _, ow = ref.gradients(part)
        off_x, off_w = off_x + ox, off_w + ow
    want_x, _, want_w, _ = ref.gradients(grad.double())
    if X.dtype == torch.float16:
        most = (grad.double().abs() * ref.tau * X.double().abs().amax(dim=1)).max()
        p = torch.exp(ref.z - ref.lse[:, None])
        off_w = off_w + 2.0 ** -38 * most * (p + ref.wanted).sum(dim=0)[:, None]
    fits = want_w.abs() < 6e4
    ref.within("dX", torch.where(want_x.abs() < 6e4, dX, 0.0), torch.where(want_x.abs() < 6e4, want_x, 0.0), off_x)
    ref.within("dW", torch.where(fits, dW, 0.0), torch.where(fits, want_w, 0.0), off_w)


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("T,spread,outlier", [(40, 20, 0), (60, 26, 0), (300, 24, 0), (300, 30, 0), (2, 20, 0), (100, 20, 6)])
def test_words_of_rows_with_small_factors(kind, T, spread, outlier):
    log(f"factors {kind} {T} rows, 2^{spread} apart, states 2^{outlier}")
    X, W, y, grad = lone_words(T, 500, 64, TYPES[kind], spread, 41, outlier)
    loss, lse = tg.linear_cross_entropy_forward(X, W, y)
    dX, dW = tg.linear_cross_entropy_backward(grad, X, W, y, lse)
    torch.cuda.synchronize()
    check(Reference(X, W, y), X, grad, dX, dW)


@pytest.mark.parametrize("kind", TYPES)
def test_a_teachers_words_of_rows_with_small_factors(kind):
    T, V, K = 200, 700, 3
    X, W, y, grad = lone_words(T, V, 72, TYPES[kind], 22, 42)
    words = V // 2
    ids = (y[:, None] + torch.arange(K, device="cuda")) % words  # all in the row's half
    ids[T // 2:] = words + torch.arange((T - T // 2) * K, device="cuda").view(-1, K) % (V - words)
    top = torch.randn((T, K), device="cuda", generator=torch.Generator(device="cuda").manual_seed(43))
    loss, lse, student = tg.linear_distillation_forward(X, W, ids, top, temperature=2.0)
    dX, dW = tg.linear_distillation_backward(grad, X, W, ids, top, lse, student, temperature=2.0)
    torch.cuda.synchronize()
    check(Reference(X, W, ids=ids, logits=top, temperature=2.0), X, grad, dX, dW)


def test_states_that_are_zero_infinite_or_all_alike():
    """fp16 rows are scaled by their largest finite state: rows without one change nothing for the others."""
    T, V, D = 24, 300, 64
    X, W, y, grad = lone_words(T, V, D, torch.float16, 20, 44)
    want = tg.linear_cross_entropy_backward(grad, X, W, y, tg.linear_cross_entropy_forward(X, W, y)[1])[1]
    more = torch.cat([X, torch.zeros_like(X[:2])])
    y2 = torch.cat([y, torch.tensor([-100, -100], device="cuda")])
    more[-1] = float("inf")
    grad2 = torch.cat([grad, torch.tensor([float("nan"), float("inf")], device="cuda")])
    got = tg.linear_cross_entropy_backward(grad2, more, W, y2, tg.linear_cross_entropy_forward(more, W, y2)[1])[1]
    assert torch.equal(got, want)
    zero = torch.zeros_like(X)
    _, dW = tg.linear_cross_entropy_backward(grad, zero, W, y, tg.linear_cross_entropy_forward(zero, W, y)[1])
    assert not bool(dW.any())
