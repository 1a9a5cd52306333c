"""The Newton-Schulz operator on the GPU against the formula in float64.

Errors are norms of the difference over the norm of the exact result.  A
result rounded to its type is off by at most half a step a value, eps / 2 of it
and of the norm.  What the arithmetic adds:

* a smaller side of up to 64 runs in float64 on float32 coefficients (which the
  reference takes too): a rounding to float32 before that to 16 bits, 2^-24;
* otherwise X is held to 2^-23 of its values, so are S and Q, and products sum
  in float32, as a chain of float32 products does, whose own error against
  float64 is the yardstick: 1.5 times that, and 2^-20 where the chain happens
  to be closer than its planes' roundings (five steps of three, of 2^-23 each,
  give 2^-19 if all add up);
* bf16 results take one fp16 plane where two are not needed: S from one, 2^-11
  of a value at most and independent from value to value, which enters X times
  |b + 2·c·s| < 5: three such steps and the two single ones before them give up
  to 2^-9, half of what the result's rounding may.
"""

import math

import pytest

torch = pytest.importorskip("torch")

import tiled_gemm_tgemm_amd as tg  # noqa: E402
from tiled_gemm_tgemm_amd import _lib  # noqa: E402

pytestmark = pytest.mark.gpu
TYPES = [torch.float32, torch.bfloat16, torch.float16]
MUON = (3.4445, -4.7750, 2.0315)


def chain(G, steps=5, coefficients=MUON, eps=1e-7, dtype=torch.float64):
    rows = [coefficients] * steps if not isinstance(coefficients[0], (tuple, list)) else coefficients
    X = G.double()
    tall = X.shape[-2] > X.shape[-1]
    if tall:
        X = X.transpose(-1, -2).contiguous()
    X = (X / (X.flatten(-2).norm(dim=-1)[..., None, None] + float(torch.tensor(eps, dtype=torch.float32)))).to(dtype)
    for row in rows:
        a, b, c = (float(torch.tensor(v, dtype=torch.float32)) for v in row)
        S = X @ X.transpose(-1, -2).contiguous()
        X = a * X + (b * S + c * (S @ S)) @ X
    return X.transpose(-1, -2).contiguous() if tall else X


def error(got, want):
    n = float(want.norm())
    return float((got.double() - want).norm()) / n if n else float(got.double().norm())


def allowed(G, want, **k):
    half = torch.finfo(G.dtype).eps / 2
    if min(G.shape[-2:]) <= 64:
        return half * 1.01 + 2.0 ** -24
    plain = error(chain(G, dtype=torch.float32, **k), want)
    if G.dtype == torch.bfloat16:
        return half + 2.0 ** -9
    return half + max(1.5 * plain, 2.0 ** -20)


def gradient(shape, dtype, seed, rank=None, noise=0.01):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g, device="cuda")
    if rank is None:
        return r(*shape).to(dtype)
    b = shape[:-2]
    return (r(*b, shape[-2], rank) @ r(*b, rank, shape[-1]) / math.sqrt(rank) + noise * r(*shape)).to(dtype)


def check(G, **k):
    want = chain(G, **k)
    got = tg.orthogonalize(G, **k)
    assert got.shape == G.shape and got.dtype == G.dtype
    assert error(got, want) <= allowed(G, want, **k)
    return got


SMALL = [(1, 1), (1, 7), (9, 1), (5, 70), (70, 5), (16, 16), (17, 300), (300, 31), (33, 33), (3, 16, 1000), (2, 1000, 64),
         (4, 64, 64), (2, 1, 4097), (24, 16, 520), (3, 50, 2500)]
LARGE = [(65, 65), (65, 300), (300, 65), (128, 128), (130, 200), (2, 200, 130), (257, 700), (700, 257), (3, 96, 100), (513, 512),
         (1000, 300), (2, 320, 1100), (1100, 1100), (7, 130, 520)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("shape", SMALL + LARGE)
def test_against_float64(shape, dtype):
    check(gradient(shape, dtype, sum(shape)))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("shape", [(40, 333), (2, 200, 16), (130, 400), (600, 200)])
@pytest.mark.parametrize("noise", [0.3, 0.003])
def test_a_few_strong_directions(shape, dtype, noise):
    check(gradient(shape, dtype, 3, rank=4, noise=noise))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("shape", [(30, 200), (200, 260)])
@pytest.mark.parametrize("steps,coefficients", [(1, MUON), (2, MUON), (3, MUON), (6, MUON), (8, (1.5, -0.5, 0.0)), (5, (2.0, -1.5, 0.5)),
                                                (3, [(3.0, -3.2, 1.2), [2.5, -2.0, 0.6], (1.875, -1.25, 0.375)])])
def test_steps_and_coefficients(shape, dtype, steps, coefficients):
    check(gradient(shape, dtype, 5), steps=steps, coefficients=coefficients)


def test_singular_values_come_to_one_and_vectors_stay():
    G = gradient((150, 400), torch.float32, 8)
    u, s, v = torch.linalg.svd(G.double(), full_matrices=False)
    out = tg.orthogonalize(G).double()
    turned = u.t() @ out @ v.t()
    values = torch.diagonal(turned)
    assert float(values.min()) > 0.6 and float(values.max()) < 1.25
    assert float((turned - torch.diag(values)).norm() / values.norm()) < 2.0 ** -16


@pytest.mark.parametrize("shape", [(20, 90), (90, 20), (100, 130)])
@pytest.mark.parametrize("scale", [1e-30, 1e-9, 1e12, 1e30])
def test_the_norm_is_not_lost_at_float32s_ends(shape, scale):
    G = gradient(shape, torch.float32, 2) * scale
    check(G, eps=0.0)


@pytest.mark.parametrize("shape", [(30, 70), (130, 140)])
def test_fp16_below_its_normal_numbers(shape):
    check((gradient(shape, torch.float32, 4) * 1e-6).to(torch.float16), eps=0.0)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("shape", [(3, 20, 90), (3, 150, 90), (3, 90, 150)])
def test_zeros_infinities_and_nans_stay_in_their_matrix(shape, dtype):
    G = gradient(shape, dtype, 6)
    want = chain(G)
    for bad in (0.0, float("inf"), float("nan")):
        H = G.clone()
        if bad == 0.0:
            H[1] = 0.0
        else:
            H[1, 5, 7] = bad
        out = tg.orthogonalize(H)
        if bad == 0.0:
            assert not bool(out[1].any())
        else:
            assert bool(out[1].isnan().all())
        for i in (0, 2):
            assert error(out[i], want[i]) <= allowed(G[i], want[i])


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("shape", [(2, 33, 70), (2, 70, 33), (2, 100, 130), (2, 130, 100)])
def test_strides_and_what_lies_between(shape, dtype):
    b, m, n = shape
    room = torch.full((b + 1, m + 3, n + 5), 7.0, device="cuda", dtype=dtype)
    G = room[:b, 1:m + 1, 3:n + 3]
    G.copy_(gradient(shape, dtype, 9))
    back = torch.full((b, m + 2, n + 7), -3.0, device="cuda", dtype=dtype)
    out = back[:, 1:m + 1, 5:n + 5]
    got = tg.orthogonalize(G, out=out)
    assert got is out
    want = chain(G)
    assert error(out, want) <= allowed(G, want)
    around = torch.ones_like(back, dtype=torch.bool)
    around[:, 1:m + 1, 5:n + 5] = False
    assert bool((back[around] == -3.0).all())
    assert torch.equal(tg.orthogonalize(G.contiguous()), out)
    # one matrix for all of a stack
    same = tg.orthogonalize(G[:1].expand(3, m, n))
    assert torch.equal(same[0], same[2]) and torch.equal(same[0], out[0])


def test_refusals():
    G = gradient((100, 80), torch.float32, 1)
    with pytest.raises(ValueError):
        tg.orthogonalize(G.t())
    with pytest.raises(ValueError):
        tg.orthogonalize(G, steps=0)
    with pytest.raises(ValueError):
        tg.orthogonalize(G, out=torch.empty(80, 100, device="cuda"))
    with pytest.raises(TypeError):
        tg.orthogonalize(G, out=torch.empty(100, 80, device="cuda", dtype=torch.float16))
    with pytest.raises(TypeError):
        tg.orthogonalize(G, workspace=torch.empty(10, device="cuda"))
    for bad in (dict(out=G), dict(steps=33), dict(eps=-1.0), dict(workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))):
        with pytest.raises(tg.TgemmError):
            tg.orthogonalize(G, **bad)
    assert tg.orthogonalize(G[:0]).shape == (0, 80) and tg.orthogonalize(torch.empty(0, 4, 5, device="cuda")).shape == (0, 4, 5)


@pytest.mark.parametrize("shape", [(3, 16, 500), (200, 130), (2, 300, 700)])
def test_the_same_call_gives_the_same_bits(shape):
    G = gradient(shape, torch.bfloat16, 12)
    first = tg.orthogonalize(G)
    need = tg.tgemm_orthogonalize_workspace_size(_lib.TGEMM_BF16, shape[0] if len(shape) == 3 else 1, *shape[-2:], 5)
    junk = torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda")
    assert torch.equal(first, tg.orthogonalize(G, workspace=junk))
    assert torch.equal(first, tg.orthogonalize(G, workspace=junk))


@pytest.mark.parametrize("shape", [(3, 16, 500), (300, 130)])
def test_captured_and_replayed(shape):
    G = gradient(shape, torch.bfloat16, 13)
    H = [gradient(shape, torch.bfloat16, s) for s in (14, 15, 16)]
    want = [tg.orthogonalize(h) for h in H]
    out = torch.empty_like(G)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        tg.orthogonalize(G, out=out)
    for h, w in zip(H, want):
        G.copy_(h)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, w)
        assert torch.equal(tg.orthogonalize(h), w)


def test_on_a_stream_of_the_callers():
    shape = (400, 300)
    G = gradient(shape, torch.bfloat16, 17)
    want = tg.orthogonalize(G)
    x = torch.randn((4096, 4096), device="cuda").bfloat16()
    y = torch.empty_like(x)
    torch.mm(x, x, out=y)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        for _ in range(30):
            torch.mm(x, x, out=y)
    out = tg.orthogonalize(G, stream=side.cuda_stream)  # returns while the stream is behind
    need = tg.tgemm_orthogonalize_workspace_size(_lib.TGEMM_BF16, 1, *shape, 5)
    junk = [torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda") for _ in range(3)]
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    del junk


@pytest.mark.parametrize("shape,dtype", [((1, 4096, 2048), torch.bfloat16), ((5000, 700), torch.float32), ((16, 520, 264), torch.float16)])
def test_larger_ones(shape, dtype):
    check(gradient(shape, dtype, 21, rank=8, noise=0.3))
