"""How often the 16-bit gradients are rounded, by the norm of their error: once
the results, and beyond 128 rows once the logits' gradient before them.

The model is that arithmetic in 64 bits: the logits' gradient rounded to the
type (or not), the product, its rounding.  float32's own errors are 2^-20 of a
value and move a rounding of 2^-9 or 2^-12 now and then, to the other side of
where it would have been: as far off on average, so the norms agree (2% is
allowed, 4% of the squares).  One more rounding of the logits' gradient would
add a third of the squares or more."""

import pytest

torch = pytest.importorskip("torch")

import tiled_gemm_tgemm_amd as tg  # noqa: E402
from loss_reference import Reference  # noqa: E402
from test_gpu_linear_loss import TYPES, entries, gpu, head, log, row_grads, targets  # noqa: E402,F401

pytestmark = pytest.mark.gpu


def norms(got, model, exact):
    return float((got.double() - exact).norm() / exact.norm()), float((model.double() - exact).norm() / exact.norm())


@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("T,V,D,K,temperature", [(300, 5003, 320, 33, 3.0), (777, 4001, 1000, 16, 2.0), (1500, 600, 512, 8, 1.0),
                                                 (64, 3000, 256, 8, 1.0), (128, 5000, 200, 20, 2.0)])
@pytest.mark.parametrize("distill", [False, True])
@pytest.mark.parametrize("factors", ["one", "rows"])
def test_roundings_of_a_gradient(kind, T, V, D, K, temperature, distill, factors):
    log(f"roundings {kind} {T}x{V}x{D} distill={distill} {factors}")
    dtype = TYPES[kind]
    X, W, g = head(T, V, D, dtype, 61)
    grad = torch.full((), 0.75, device="cuda") if factors == "one" else row_grads(T, g)
    if distill:
        ids, top = entries(T, V, K, dtype, g)
        ref = Reference(X, W, ids=ids, logits=top, temperature=temperature)
        loss, lse, student = tg.linear_distillation_forward(X, W, ids, top, temperature=temperature)
        dX, dW = tg.linear_distillation_backward(grad, X, W, ids, top, lse, student, temperature=temperature)
    else:
        y = targets(T, V, g)
        ref = Reference(X, W, y)
        loss, lse = tg.linear_cross_entropy_forward(X, W, y)
        dX, dW = tg.linear_cross_entropy_backward(grad, X, W, y, lse)
    torch.cuda.synchronize()
    c = torch.where(ref.counts, grad.double() * ref.tau, 0.0)[:, None]
    dz = torch.where(ref.counts[:, None], torch.exp(ref.z - ref.lse[:, None]) - ref.wanted, 0.0)
    exact = (c * dz) @ ref.W, (c * dz).t() @ ref.Xc
    if T > 128:
        # what is held: fp16's at 2^15 of a fraction; one factor for all rows comes afterwards
        held = torch.ones_like(c) if factors == "one" else torch.where(c == 0, 1.0, torch.frexp(c)[0] if kind == "fp16" else c)
        if kind == "fp16":
            held = held * 2.0 ** 15
        dz = (dz * held).to(dtype).double() / held
    model = ((c * dz) @ ref.W).to(dtype), ((c * dz).t() @ ref.Xc).to(dtype)
    once = exact[0].to(dtype), exact[1].to(dtype)
    for name, got, m, e, o in zip(("dX", "dW"), (dX, dW), model, exact, once):
        mine, its = norms(got, m, e)
        alone = norms(o, o, e)[0]
        log(f"  {name}: {mine:.3e}, model {its:.3e}, the results' rounding {alone:.3e}")
        assert mine <= 1.02 * its, name
        # two roundings of one size at most: the root of 2, or a little more where a row hangs on few entries
        assert its <= 1.6 * alone, name
