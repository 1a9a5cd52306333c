"""The projection with low-rank adapters on the GPU against the formula in
float64, value by value.

A result is rounded once to its type, half a step: eps / 2 of the value.  Sums
of n products in float32 are off by n·2^-24 of the sum of their magnitudes at
most; hidden values, h = x·Aᵀ and u = dy·B, carry that on, and 2^-17 of their
own for the two bf16 numbers that 16-bit operands meet (fp16 ones are two bf16
numbers themselves: 2^-16 in all).  A float32 product is bounded by 4·n·2^-24
of the magnitudes, whichever way it takes.  Bounds are worked out from the
magnitudes of each value's own products.
"""

import math

import pytest

torch = pytest.importorskip("torch")

import tiled_gemm_tgemm_amd as tg  # noqa: E402
from tiled_gemm_tgemm_amd import _lib  # noqa: E402

pytestmark = pytest.mark.gpu
TYPES = [torch.float32, torch.bfloat16, torch.float16]


def layer(T, N, D, L, r, dtype, seed, ids="random"):
    g = torch.Generator(device="cuda").manual_seed(seed)
    n = lambda *s: torch.randn(s, generator=g, device="cuda")
    X, W = n(T, D).to(dtype), (n(N, D) / math.sqrt(D)).to(dtype)
    A, B = (n(L, r, D) / math.sqrt(D)).to(dtype), (n(L, N, r) / math.sqrt(r)).to(dtype)
    scales = torch.rand(L, generator=g, device="cuda") * 2 - 0.5
    if ids == "random":
        i = torch.randint(-1, L, (T,), generator=g, device="cuda")
    elif ids == "runs":
        i = torch.randint(-1, L, (T // 77 + 1,), generator=g, device="cuda").repeat_interleave(77)[:T].contiguous()
    else:
        i = torch.full((T,), ids, dtype=torch.int64, device="cuda")
    return X, W, A, B, i, scales, n(T, N).to(dtype)


def exact(X, W, A, B, ids, scales, dY):
    """Y, dX, dW, dA, dB and, for each, how far a value may be off before its rounding."""
    dtype = X.dtype
    (T, D), (N, _), (L, r, _) = X.shape, W.shape, A.shape
    x, w, a, b, dy = (t.detach().double() for t in (X, W, A, B, dY))
    step = 2.0 ** -24 * (4 if dtype == torch.float32 else 1)
    planes = 0.0 if dtype == torch.float32 else 2.0 ** -16
    Y, dX, dW = x @ w.t(), dy @ w, dy.t() @ x
    oY, oX, oW = (n * step * (p.abs() @ q.abs()) for n, p, q in ((D, x, w.t()), (N, dy, w), (T, dy.t(), x)))
    dA, dB, oA, oB = torch.zeros_like(a), torch.zeros_like(b), torch.zeros_like(a), torch.zeros_like(b)
    for i in range(L):
        at = torch.nonzero(ids == i)[:, 0]
        n = at.numel()
        if n == 0:
            continue
        s = float(scales[i]) if scales is not None else 1.0
        xi, di = x[at], dy[at]
        h, u = xi @ a[i].t(), di @ b[i]
        oh, ou = D * step * (xi.abs() @ a[i].abs().t()), N * step * (di.abs() @ b[i].abs())
        off = lambda o, v, m: o + (planes + m * step) * v.abs()  # and the m products that it enters
        Y[at] += s * (h @ b[i].t())
        oY[at] += abs(s) * (off(oh, h, r + 2) @ b[i].abs().t())
        dX[at] += s * (u @ a[i])
        oX[at] += abs(s) * (off(ou, u, r + 2) @ a[i].abs())
        dA[i], oA[i] = s * (u.t() @ xi), abs(s) * (off(ou, u, n + 2).t() @ xi.abs())
        dB[i], oB[i] = s * (di.t() @ h), abs(s) * (di.abs().t() @ off(oh, h, n + 2))
    return (Y, dX, dW, dA, dB), (oY, oX, oW, oA, oB)


def close(got, want, off, what=""):
    half = torch.finfo(got.dtype).eps / 2
    tiny = torch.finfo(got.dtype).smallest_normal * half * 2  # half a step below the normal numbers, and more
    least = (off + (want.abs() + off) * half) * 1.0001 + tiny
    bad = ~((got.double() - want).abs() <= least)
    assert not bool(bad.any()), (what, int(bad.sum()), float(((got.double() - want).abs() - least).max()))


def check(args, need=(True, True, True, True)):
    X, W, A, B, ids, scales, dY = args
    want, off = exact(*args)
    hidden = torch.full((X.shape[0], A.shape[1]), float("nan"), device="cuda")
    Y = tg.linear_adapters_forward(X, W, A, B, ids, scales=scales, hidden=hidden)
    close(Y, want[0], off[0], "Y")
    assert torch.equal(Y, tg.linear_adapters_forward(X, W, A, B, ids, scales=scales))
    grads = tg.linear_adapters_backward(dY, X, W, A, B, ids, hidden, scales=scales, need=need)
    for n, (g, name) in enumerate(zip(grads, ("dX", "dW", "dA", "dB"))):
        assert (g is not None) == need[n]
        if need[n]:
            close(g, want[n + 1], off[n + 1], name)
    return Y, grads


SIZES = [  # T, N, D, L, r
    (1, 16, 8, 1, 1), (1, 300, 130, 3, 4), (2, 33, 520, 2, 16), (15, 100, 64, 5, 8), (16, 4096, 257, 8, 16), (17, 129, 1000, 17, 5),
    (33, 8200, 96, 6, 16), (48, 520, 200, 32, 33), (64, 65, 63, 4, 64), (65, 64, 65, 3, 7), (100, 1000, 333, 40, 12), (129, 257, 512, 2, 100),
    (256, 640, 320, 20, 16), (300, 72, 1100, 9, 200), (777, 1000, 520, 3, 10), (1025, 192, 128, 5, 24), (1500, 320, 448, 2, 64),
]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("ids", ["random", "runs"])
@pytest.mark.parametrize("size", SIZES)
def test_against_float64(size, ids, dtype):
    check(layer(*size, dtype, sum(size), ids))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("size,ids", [((2048, 1024, 512, 2, 8), "runs"), ((4200, 328, 264, 3, 40), "runs"), ((3000, 512, 256, 30, 16), "random"),
                                      ((9000, 128, 192, 20, 8), "runs"), ((8500, 64, 64, 3, 130), "random"), ((70, 4096, 4096, 40, 16), "random")])
def test_larger_ones(size, ids, dtype):
    check(layer(*size, dtype, 5, ids))


@pytest.mark.parametrize("dtype", TYPES[1:])
@pytest.mark.parametrize("T", [1, 2, 16, 17, 32, 33, 47, 48, 49, 64])
@pytest.mark.parametrize("N,D", [(1, 64), (50, 128), (640, 192), (100, 256), (330, 832), (48, 1024), (8193, 64), (8200, 1088)])
def test_few_rows_of_whole_steps(T, N, D, dtype):
    """These go through LDS: sums of fewer steps than wavefronts, of fewer and of more than there are stages."""
    check(layer(T, N, D, 5, 24, dtype, T + N + D), (False, False, False, True))


@pytest.mark.parametrize("dtype", TYPES[1:])
@pytest.mark.parametrize("T", [7, 40])
def test_few_rows_of_wider_ones(T, dtype):
    """X and W with leading dimensions of their own, what lies between their rows not a number; Y's other columns stay."""
    X, W, A, B, ids, scales, dY = layer(T, 200, 320, 4, 8, dtype, 8)
    want, off = exact(X, W, A, B, ids, scales, dY)
    wide = lambda m, more: torch.cat([m, torch.full((m.shape[0], more), float("nan"), device="cuda", dtype=dtype)], 1)[:, : m.shape[1]]
    out = torch.full((T, 208), 3.0, device="cuda", dtype=dtype)
    Y = tg.linear_adapters_forward(wide(X, 8), wide(W, 64), A, B, ids, scales=scales, out=out[:, :200])
    close(Y, want[0], off[0])
    assert bool((out[:, 200:] == 3).all())


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T", [5, 70, 1100])
@pytest.mark.parametrize("ids", [-1, 2])
def test_no_adapter_or_one_for_all(T, ids, dtype):
    args = layer(T, 200, 136, 4, 12, dtype, 3, ids)
    Y, (dX, dW, dA, dB) = check(args)
    others = [i for i in range(4) if i != ids]
    assert not bool(dA[others].any()) and not bool(dB[others].any())  # zeros, not what the memory held


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T", [3, 90, 1300])
def test_without_scales_and_parts_of_the_gradients(T, dtype):
    X, W, A, B, ids, _, dY = layer(T, 96, 128, 3, 16, dtype, 4)
    args = (X, W, A, B, ids, None, dY)
    _, all_of = check(args)
    for bits in range(1, 15):
        need = tuple(bool(bits >> n & 1) for n in range(4))
        got = tg.linear_adapters_backward(dY, X, W, A, B, ids, need=need)  # hidden formed again
        for n in range(4):
            assert (got[n] is None) if not need[n] else torch.equal(got[n], all_of[n])
    assert tg.linear_adapters_backward(dY, X, W, A, B, ids, need=(False,) * 4) == (None,) * 4


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T", [6, 200, 1200])
def test_an_id_out_of_range_is_its_rows_alone(T, dtype):
    args = list(layer(T, 140, 96, 3, 8, dtype, 6))
    bad = torch.tensor([1, T // 2, T - 1], device="cuda")
    ids = args[4].clone()
    args[4] = ids.clone()
    args[4][bad] = -1  # what the formula is worked out for
    want, off = exact(*args)
    X, W, A, B, _, scales, dY = args
    ids[bad] = torch.tensor([3, -2, 1 << 40], device="cuda")
    good = torch.ones(T, dtype=torch.bool, device="cuda")
    good[bad] = False
    Y = tg.linear_adapters(X, W, A, B, ids, scales=scales)
    assert bool(Y[bad].isnan().all())
    close(Y[good], want[0][good], off[0][good])
    dX, dW, dA, dB = tg.linear_adapters_backward(dY, X, W, A, B, ids, scales=scales)
    assert bool(dX[bad].isnan().all())
    close(dX[good], want[1][good], off[1][good])
    for g, w, o in ((dW, want[2], off[2]), (dA, want[3], off[3]), (dB, want[4], off[4])):
        close(g, w, o)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,ids", [(20, "random"), (150, "random"), (1200, "random"), (1200, "runs"), (4500, "runs")])
def test_an_adapter_of_nans_reaches_its_own_rows_alone(T, ids, dtype):
    args = layer(T, 264, 192, 4, 16, dtype, 7, ids)
    X, W, A, B, i, scales, dY = args
    want, off = exact(*args)
    A, B = A.clone(), B.clone()
    A[1], B[1, :, 3] = float("nan"), float("inf")
    others, rows = [0, 2, 3], i != 1
    Y = tg.linear_adapters(X, W, A, B, i, scales=scales)
    close(Y[rows], want[0][rows], off[0][rows])
    assert bool(Y[~rows].isnan().all())
    dX, dW, dA, dB = tg.linear_adapters_backward(dY, X, W, A, B, i, scales=scales)
    close(dX[rows], want[1][rows], off[1][rows])
    assert bool(dX[~rows].isnan().all())
    close(dW, want[2], off[2])
    close(dA[others], want[3][others], off[3][others])
    close(dB[others], want[4][others], off[4][others])


@pytest.mark.parametrize("T", [40, 300, 1100])
def test_fp16_hidden_values_past_its_range(T):
    # x·Aᵀ is about 1e6, past fp16's 65504; B brings it back
    X, W, A, B, ids, scales, dY = layer(T, 96, 128, 2, 8, torch.float16, 8)
    A, B = (A.float() * 1e5).clamp(-6e4, 6e4).half(), (B.float() * 1e-5).half()
    check((X, W, A, B, ids, scales, dY), need=(False, True, False, False))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T", [0, 1])
def test_an_empty_batch_and_one_row(T, dtype):
    args = layer(T, 50, 40, 2, 3, dtype, 9)
    X, W, A, B, ids, scales, dY = args
    Y = tg.linear_adapters(X, W, A, B, ids, scales=scales)
    assert Y.shape == (T, 50)
    dX, dW, dA, dB = tg.linear_adapters_backward(dY, X, W, A, B, ids, scales=scales)
    if T == 0:
        assert dX.shape == (0, 40) and not bool(dW.any()) and not bool(dA.any()) and not bool(dB.any())
    else:
        check(args)


def padded(t, value, dtype, before=3, after=5, off=0):
    """The same values in the middle of larger memory, that starts `off` elements off its alignment."""
    rows, cols = t.shape[-2] + 2, t.shape[-1] + before + after
    lead = [t.shape[0] + 1] if t.dim() == 3 else []
    flat = torch.full((math.prod(lead + [rows, cols]) + off,), value, dtype=dtype, device="cuda")
    room = flat[off:].view(*lead, rows, cols)
    inner = (room[:-1] if lead else room)[..., 1:-1, before:cols - after]
    inner.copy_(t)
    return flat, inner


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("size", [(20, 100, 70, 3, 6), (150, 96, 64, 4, 16), (1200, 72, 128, 3, 20)])
@pytest.mark.parametrize("before,after,off", [(3, 5, 0), (8, 8, 0), (8, 0, 1)])
def test_strides_and_what_lies_between(size, before, after, off, dtype):
    X, W, A, B, ids, scales, dY = layer(*size, dtype, 10)
    T, N, D, L, r = size
    _, wide = check((X, W, A, B, ids, scales, dY))
    k = dict(before=before, after=after, off=off)
    Xs, Ws, As, Bs, dYs = (padded(t, float("nan"), dtype, **k)[1] for t in (X, W, A, B, dY))
    twice = torch.stack([ids, ids + 1], dim=1)[:, 0]  # not contiguous
    room, out = padded(torch.zeros(T, N, device="cuda", dtype=dtype), 9.0, dtype, **k)
    assert tg.linear_adapters_forward(Xs, Ws, As, Bs, twice, scales=scales, out=out) is out
    want, offs = exact(X, W, A, B, ids, scales, dY)
    close(out, want[0], offs[0], "Y")
    outs = [padded(torch.zeros_like(g), 9.0, dtype, **k) for g in wide]
    got = tg.linear_adapters_backward(dYs, Xs, Ws, As, Bs, twice, scales=scales, dX=outs[0][1], dW=outs[1][1], dA=outs[2][1], dB=outs[3][1])
    for g, w, o, name in zip(got, want[1:], offs[1:], ("dX", "dW", "dA", "dB")):
        close(g, w, o, name)
    for flat, inner in [(room, out), *outs]:  # nothing around them was written
        inner.fill_(9.0)
        assert bool((flat == 9.0).all())
    # one adapter's matrices for all of a stack
    stack = (A[:1].expand(L, r, D), B[:1].expand(L, N, r))
    want, offs = exact(X, W, *stack, ids, None, dY)
    close(tg.linear_adapters(X, W, *stack, ids), want[0], offs[0])


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T", [10, 200, 1500])
def test_autograd_gives_the_same(T, dtype):
    X, W, A, B, ids, scales, dY = layer(T, 128, 192, 3, 8, dtype, 11, "runs")
    want = (tg.linear_adapters_forward(X, W, A, B, ids, scales=scales), *tg.linear_adapters_backward(dY, X, W, A, B, ids, scales=scales))
    leaves = [t.clone().requires_grad_() for t in (X, W, A, B)]
    Y = tg.linear_adapters(*leaves, ids, scales=scales)
    got = torch.autograd.grad(Y, leaves, dY)
    assert torch.equal(Y.detach(), want[0]) and all(torch.equal(g, w) for g, w in zip(got, want[1:]))
    for n in range(4):  # any one of them alone
        some = [t.clone().requires_grad_(n == m) for m, t in enumerate((X, W, A, B))]
        Y = tg.linear_adapters(*some, ids, scales=scales)
        Y.backward(dY)
        assert torch.equal(some[n].grad, want[n + 1]) and all(t.grad is None for m, t in enumerate(some) if m != n)
    # a gradient that is one number for all, and one that lies the other way
    Y = tg.linear_adapters(*leaves, ids, scales=scales)
    one = torch.autograd.grad(Y.float().sum(), leaves[2])[0]
    assert torch.equal(one, tg.linear_adapters_backward(torch.ones_like(dY), X, W, A, B, ids, scales=scales)[2])
    Y = tg.linear_adapters(*leaves, ids, scales=scales)
    assert torch.equal(torch.autograd.grad(Y, leaves[3], dY.t().contiguous().t())[0], want[4])
    with torch.no_grad():
        assert not tg.linear_adapters(*leaves, ids, scales=scales).requires_grad
    # twice through one graph, and not after a leaf has changed
    Y = tg.linear_adapters(*leaves, ids, scales=scales)
    first = torch.autograd.grad(Y, leaves, dY, retain_graph=True)
    assert all(torch.equal(a, b) for a, b in zip(first, torch.autograd.grad(Y, leaves, dY, retain_graph=True)))
    with torch.no_grad():
        leaves[2].add_(1.0)
    with pytest.raises(RuntimeError):
        torch.autograd.grad(Y, leaves, dY)


@pytest.mark.parametrize("T", [12, 100, 1100])
def test_gradients_against_differences(T):
    # the result is linear in each argument alone, so a difference of any width is exact but for roundings: those of
    # 2·T·N results of about 2 in float32, weighted with dY, against a sum of about sqrt(T·N)
    X, W, A, B, ids, scales, dY = layer(T, 130, 70, 3, 9, torch.float32, 12)
    grads = tg.linear_adapters_backward(dY, X, W, A, B, ids, scales=scales)
    g = torch.Generator(device="cuda").manual_seed(1)
    for n, t in enumerate((X, W, A, B)):
        V = torch.randn(t.shape, generator=g, device="cuda")
        some = [X, W, A, B]
        ends = []
        for sign in (0.5, -0.5):
            some[n] = t + sign * V
            ends.append(tg.linear_adapters(*some, ids, scales=scales).double())
        change = float(((ends[0] - ends[1]) * dY.double()).sum())
        slope = float((grads[n].double() * V.double()).sum())
        assert abs(change - slope) <= 2.0 ** -14 * math.sqrt(T * 130) * 8


@pytest.mark.parametrize("T", [30, 200, 1500])
def test_captured_and_replayed(T):
    captured((T, 128, 192, 3, 8), torch.bfloat16)


@pytest.mark.parametrize("sizes", [(50, 100, 90, 3, 8), (300, 200, 1000, 20, 6), (2100, 1000, 520, 3, 10)])
def test_captured_and_replayed_in_float32(sizes):
    """Few rows, the float32 product in parts, and the planes' product."""
    captured(sizes, torch.float32)


def captured(sizes, dtype):
    T, N, _, _, r = sizes
    args = layer(*sizes, dtype, 13)
    X, W, A, B, ids, scales, dY = args
    hidden = torch.empty(T, r, device="cuda")
    out = torch.empty(T, N, device="cuda", dtype=dtype)
    grads = [torch.empty_like(t) for t in (X, W, A, B)]

    def step():
        tg.linear_adapters_forward(X, W, A, B, ids, scales=scales, out=out, hidden=hidden)
        tg.linear_adapters_backward(dY, X, W, A, B, ids, hidden, scales=scales, dX=grads[0], dW=grads[1], dA=grads[2], dB=grads[3])

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seed in (14, 15, 16):
        for t, v in zip((X, W, A, B, ids, scales, dY), layer(*sizes, dtype, seed, "runs" if seed == 15 else "random")):
            t.copy_(v)
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (out, *grads)]
        step()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, (out, *grads)))


@pytest.mark.parametrize("T", [30, 500, 1500])
def test_on_a_stream_of_the_callers(T):
    args = layer(T, 256, 192, 3, 8, torch.bfloat16, 17)
    X, W, A, B, ids, scales, dY = args
    want = (tg.linear_adapters_forward(X, W, A, B, ids, scales=scales), *tg.linear_adapters_backward(dY, X, W, A, B, ids, scales=scales))
    x = torch.randn((4096, 4096), device="cuda").bfloat16()
    y = torch.empty_like(x)
    torch.mm(x, x, out=y)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        for _ in range(30):
            torch.mm(x, x, out=y)
    twice = torch.stack([ids, ids], dim=1)[:, 0]  # a copy that the call makes of it, too
    got = (tg.linear_adapters_forward(X, W, A, B, twice, scales=scales, stream=side.cuda_stream),
           *tg.linear_adapters_backward(dY, X, W, A, B, twice, scales=scales, stream=side.cuda_stream))
    need = max(tg.tgemm_linear_adapters_workspace_size(_lib.TGEMM_BF16, T, 256, 192, X.data_ptr(), 192, W.data_ptr(), 192, 3, 8, dY.data_ptr(), 256, n)
               for n in (0, 15))
    junk = [torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda") for n in (need, need, T * 8, T * 8, 1024)]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    del junk


def test_autograd_on_a_side_stream():
    args = layer(400, 256, 192, 3, 8, torch.bfloat16, 18)
    X, W, A, B, ids, scales, dY = args
    want = tg.linear_adapters_backward(dY, X, W, A, B, ids, scales=scales)
    leaves = [t.clone().requires_grad_() for t in (X, W, A, B)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        Y = tg.linear_adapters(*leaves, ids, scales=scales)
    torch.cuda.current_stream().wait_stream(side)
    got = torch.autograd.grad(Y, leaves, dY)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_refusals():
    X, W, A, B, ids, scales, dY = layer(20, 48, 64, 2, 4, torch.bfloat16, 19)
    for bad in (dict(W=W.float()), dict(A=A.half()), dict(B=B[0]), dict(ids=ids.int()), dict(ids=ids[:-1]), dict(X=X.cpu()), dict(A=A.cpu()),
                dict(ids=ids.cpu())):
        with pytest.raises((TypeError, ValueError)):
            tg.linear_adapters(*dict(dict(X=X, W=W, A=A, B=B, ids=ids), **bad).values())
    for bad in (dict(W=W[:, :-1]), dict(A=A[:, :, :-1]), dict(B=B[:, :-1]), dict(B=B[:1]), dict(X=X.t().contiguous().t()), dict(A=A[:0]),
                dict(B=B.transpose(1, 2).contiguous().transpose(1, 2))):
        with pytest.raises(ValueError):
            tg.linear_adapters(*dict(dict(X=X, W=W, A=A, B=B, ids=ids), **bad).values())
    for bad in (dict(scales=scales.half()), dict(scales=scales[:1]), dict(scales=2.0)):
        with pytest.raises((TypeError, ValueError)):
            tg.linear_adapters(X, W, A, B, ids, **bad)
    with pytest.raises((TypeError, ValueError)):
        tg.linear_adapters_forward(X, W, A, B, ids, hidden=torch.empty(20, 5, device="cuda"))
    with pytest.raises(ValueError):
        tg.linear_adapters_forward(X, W, A, B, ids, out=torch.empty(20, 49, device="cuda", dtype=X.dtype))
    with pytest.raises(ValueError):
        tg.linear_adapters_backward(dY[:-1], X, W, A, B, ids)
    with pytest.raises(tg.TgemmError):
        tg.linear_adapters_forward(X, W, A, B, ids, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(tg.TgemmError):  # results over an input
        tg.linear_adapters_backward(dY, X, W, A, B, ids, dX=X)
