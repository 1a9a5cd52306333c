"""How far the Newton-Schulz operator's results are from float64, beyond their own
rounding, which is measured instead of bounded.

With x the exact result, x' what is rounded and r() the rounding to the
result's type: no value lies nearer to x' than r(x'), so |r(x') - x'| <= |r(x) -
x'| <= |r(x) - x| + |x' - x|, and |r(x') - x| <= |r(x) - x| + 2·|x' - x|.  Norms
of these over the norm of x: the error is at most the rounding's own and twice
the arithmetic's.  That is the float64 form's for a side of up to 64 (2^-24, the
rounding to float32 before that to 16 bits), otherwise, products being summed
in float32 from 22 bits, as a chain of float32 products has it: 1.5 times that
chain's error, and 2^-20 where the chain happens to be closer.
"""

import math

import pytest

torch = pytest.importorskip("torch")

import tiled_gemm_tgemm_amd as tg  # noqa: E402
from test_gpu_orthogonalize import MUON, TYPES, chain, error, gradient  # noqa: E402

pytestmark = pytest.mark.gpu


def check(G, **k):
    want = chain(G, **k)
    if min(G.shape[-2:]) <= 64:
        arithmetic = 2.0 ** -24
    else:
        arithmetic = max(1.5 * error(chain(G, dtype=torch.float32, **k), want), 2.0 ** -20)
    got = error(tg.orthogonalize(G, **k), want)
    assert got <= error(want.to(G.dtype), want) + 2 * arithmetic, got


# (entries of X, S and b·S + c·S·S stay below 20 in all of these, whatever a is)
WIDE = [(1, (100.0, -150.0, 60.0)), (1, (-70.0, 20.0, -3.0)), (2, [(40.0, -20.0, 3.0), (0.03, -0.001, 0.0)]), (1, (1e6, 0.0, 0.0))]


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16])
@pytest.mark.parametrize("shape", [(40, 300), (130, 200), (300, 130), (3, 257, 700)])
@pytest.mark.parametrize("steps,coefficients", WIDE)
def test_a_factor_of_any_size(shape, dtype, steps, coefficients):
    check(gradient(shape, dtype, 31), steps=steps, coefficients=coefficients)
