"""How far the Newton-Schulz operator's results are from float64, beyond their own
rounding, which is measured instead of bounded.

With x the exact result, x' what is rounded and r() the rounding to the
result's type: no value lies nearer to x' than r(x'), so |r(x') - x'| <= |r(x) -
x'| <= |r(x) - x| + |x' - x|, and |r(x') - x| <= |r(x) - x| + 2·|x' - x|.  Norms
of these over the norm of x: the error is at most the rounding's own and twice
the arithmetic's.  That is the float64 form's for a side of up to 64 (2^-24, the
rounding to float32 before that to 16 bits), otherwise the sum of two:

* of the products, which are summed in float32 as a chain of float32 products
  does, and of roundings that differ from value to value: 1.5 times that chain's
  error, and 2^-20 where the chain happens to be closer;
* of the planes' roundings where they are alike, as those of equal values are.
  A value is held as the nearest fp16 number and the nearest one to the rest,
  2^-11 of 2^-11 of it off at most, and the products of two rests, 2^-22 of the
  whole at most, are left out.  So X, S, S·S, the polynomial and the next X change
  by at most 2^-21 of themselves each, and the result by that times what a
  relative change common to all their values makes of it: `responses` adds
  these up over all steps, in float64.  They come to less than 800, but to 6e4
  to 1e5 with PER_STEP on a matrix of one direction, whose singular value of 1
  is the end of that set's range, where the polynomials are steep.
"""

import math

import pytest

torch = pytest.importorskip("torch")

import tiled_gemm_tgemm_amd as tg  # noqa: E402
from test_gpu_orthogonalize import MUON, TYPES, chain, error, gradient  # noqa: E402

pytestmark = pytest.mark.gpu


def responses(G, steps=5, coefficients=MUON):
    """What the result changes by for common relative changes of X, of S, of S·S, of b·S + c·S·S and of a·X before
    each step's sum and of the sum, over the changes: all of them added up."""
    change = 2.0 ** -20
    rows = [coefficients] * steps if not isinstance(coefficients[0], (tuple, list)) else coefficients
    rows = [tuple(float(torch.tensor(v, dtype=torch.float32)) for v in row) for row in rows]
    X = G.double()
    if X.shape[-2] > X.shape[-1]:
        X = X.transpose(-1, -2).contiguous()
    X = X / X.flatten(-2).norm(dim=-1)[..., None, None]
    square = lambda X: X @ X.transpose(-1, -2).contiguous()

    def go(X, rows):
        for a, b, c in rows:
            S = square(X)
            X = a * X + (b * S + c * (S @ S)) @ X
        return X

    want = go(X, rows)
    total = 0.0
    for n, (a, b, c) in enumerate(rows):
        S, more = square(X), 1 + change
        SS = S @ S
        P = b * S + c * SS
        ends = [go(more * X, rows[n:n + 1]), a * X + (b * more * S + c * more * more * SS) @ X, a * X + (b * S + c * more * SS) @ X,
                a * X + (more * P) @ X, a * more * X + P @ X, more * (a * X + P @ X)]
        total += sum(float((go(Y, rows[n + 1:]) - want).norm()) for Y in ends) / (change * float(want.norm()))
        X = a * X + P @ X
    return total


def check(G, **k):
    want = chain(G, **k)
    if min(G.shape[-2:]) <= 64:
        arithmetic = 2.0 ** -24
    else:
        arithmetic = max(1.5 * error(chain(G, dtype=torch.float32, **k), want), 2.0 ** -20) + 2.0 ** -21 * responses(G, **k)
    got = error(tg.orthogonalize(G, **k), want)
    assert got <= error(want.to(G.dtype), want) + 2 * arithmetic, got


# (entries of X, S and b·S + c·S·S stay below 20 in all of these, whatever a is)
WIDE = [(1, (100.0, -150.0, 60.0)), (1, (-70.0, 20.0, -3.0)), (2, [(40.0, -20.0, 3.0), (0.03, -0.001, 0.0)]), (1, (1e6, 0.0, 0.0))]


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16])
@pytest.mark.parametrize("shape", [(40, 300), (130, 200), (300, 130), (3, 257, 700)])
@pytest.mark.parametrize("steps,coefficients", WIDE)
def test_a_factor_of_any_size(shape, dtype, steps, coefficients):
    check(gradient(shape, dtype, 31), steps=steps, coefficients=coefficients)


# numbers that change from step to step, as minimax polynomials over the range that is left have them
PER_STEP = [(8.2872, -23.5959, 17.3004), (4.1071, -2.9478, 0.5448), (3.9487, -2.9089, 0.5518), (3.3184, -2.4885, 0.5100), (2.3007, -1.6689, 0.4188)]
# the same with singular values of up to 1.01 taken for 1
SAFE = [(a / 1.01, b / 1.01 ** 3, c / 1.01 ** 5) for a, b, c in PER_STEP]


def matrix(kind, m, n, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g, device="cuda")
    if kind.startswith("ones"):  # one direction of equal signs, as a mean that all tokens share
        return 1.0 + float(kind[5:]) * r(m, n)
    if kind == "one direction":
        return r(m, 1) * r(1, n) + 1e-3 * r(m, n)
    if kind == "a few rows":  # of an output head's words, those that were seen
        G = 0.01 * r(m, n)
        G[:max(1, m // 20)] += r(max(1, m // 20), n)
        return G
    if kind == "blocks":  # whole blocks of one value, whose roundings are alike
        signs = torch.sign(r(m // 16 + 1, n // 16 + 1))
        return signs.repeat_interleave(16, 0).repeat_interleave(16, 1)[:m, :n] + 1e-3 * r(m, n)
    if kind == "one value a row":  # an embedding's gradient: again equal values, in few places
        at = torch.randint(0, n, (m,), generator=g, device="cuda")
        return torch.nn.functional.one_hot(at, n).float() * 3 + 1e-3 * r(m, n)
    assert kind == "orthogonal"
    q = torch.linalg.qr(r(max(m, n), min(m, n)).double())[0].float()
    return (q if m >= n else q.t()).contiguous()


KINDS = ["ones+0.01", "ones+0.001", "ones+0.0001", "one direction", "a few rows", "blocks", "one value a row", "orthogonal"]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("coefficients", [MUON, PER_STEP, SAFE], ids=["one for all", "per step", "per step, safe"])
@pytest.mark.parametrize("shape", [(256, 1024), (384, 384), (70, 300), (300, 70), (40, 500)])
@pytest.mark.parametrize("kind", KINDS)
def test_matrices_of_a_dominant_direction_or_of_equal_values(kind, shape, coefficients, dtype):
    check(matrix(kind, *shape, 32).to(dtype), coefficients=coefficients)


@pytest.mark.parametrize("shape", [(65, 300), (200, 260), (257, 700), (1000, 300), (2, 320, 1100)])
@pytest.mark.parametrize("dtype", TYPES)
def test_normal_values(shape, dtype):
    check(gradient(shape, dtype, 33))


@pytest.mark.parametrize("shape,coefficients", [((8, 1024, 2048), MUON), ((2048, 1024), SAFE)])
def test_stacked_and_larger_ones(shape, coefficients):
    G = gradient(shape, torch.bfloat16, 34, rank=8, noise=0.3)
    check(G + G.new_ones(()), coefficients=coefficients)
