"""The losses on an output head's product against their formulas in 64 bits
(tests/loss_reference.py, which derives the tolerances), on the GPU."""

import pytest

torch = pytest.importorskip("torch")

import tiled_gemm_tgemm_amd as tg  # noqa: E402
from loss_reference import Reference  # noqa: E402
from tiled_gemm_tgemm_amd import _lib  # noqa: E402

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}

# T, V, D: single rows and words, sizes that no tile or step divides, whole
# tiles, and enough rows or words for several tiles each way
SIZES = [(1, 1, 1), (1, 257, 64), (2, 31, 7), (5, 300, 40), (20, 129, 1000), (33, 1000, 128), (64, 512, 64),
         (65, 513, 72), (130, 777, 200), (257, 2049, 64), (256, 1024, 256), (300, 5003, 320), (1, 20011, 192),
         (700, 130, 65), (2100, 100, 64), (1500, 600, 512),
         (16, 4001, 136), (17, 130, 520), (32, 1000, 8), (3, 70, 384)]


@pytest.fixture(scope="module", autouse=True)
def gpu():
    assert torch.cuda.is_available(), "GPU tests need an MI355X"
    tg.library()
    yield


def log(msg):
    print(msg, flush=True)


def generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def matrix(rows, cols, dtype, g, scale=1.0, pad=0, shift=0):
    """rows×cols normal values; rows `pad` elements apart beyond cols, the first `shift` elements into its storage."""
    room = torch.full((rows * (cols + pad) + shift + 8,), float("nan"), dtype=dtype, device="cuda")
    m = room[shift:shift + rows * (cols + pad)].view(rows, cols + pad)[:, :cols]
    m.copy_(torch.randn((rows, cols), generator=g, device="cuda") * scale)
    return m


def head(T, V, D, dtype, seed, pad=0, shift=0):
    g = generator(seed)
    return matrix(T, D, dtype, g, pad=pad, shift=shift), matrix(V, D, dtype, g, 2.0 / D ** 0.5, pad=pad, shift=shift), g


def targets(T, V, g, ignored=0.15):
    t = torch.randint(0, V, (T,), generator=g, device="cuda")
    if T > 4:
        t[torch.rand(T, generator=g, device="cuda") < ignored] = -100
        t[0] = 0
        t[1] = V - 1
        t[2] = -100
    return t


def entries(T, V, K, dtype, g):
    """A teacher's entries: ids with repetitions, absent ones (with any id), rows without one."""
    ids = torch.randint(0, V, (T, K), generator=g, device="cuda")
    logits = (torch.randn((T, K), generator=g, device="cuda") * 3).to(dtype)
    if T > 4:
        if K > 1:
            ids[0, 1] = ids[0, 0]
            gone = torch.rand((T, K), generator=g, device="cuda") < 0.2
            gone[0] = False
            logits[gone] = float("-inf")
            ids[gone] = torch.where(torch.rand((T, K), generator=g, device="cuda") < 0.5, -7, V + 5)[gone]
            logits[3] = torch.finfo(dtype).min
            ids[3] = torch.arange(K, device="cuda") % V
        logits[4] = float("-inf")
    return ids, logits


def row_grads(T, g):
    return torch.randn(T, generator=g, device="cuda") * 0.1


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("T,V,D", SIZES)
def test_cross_entropy(kind, T, V, D):
    log(f"cross entropy {kind} {T}x{V}x{D}")
    X, W, g = head(T, V, D, TYPES[kind], 1)
    y, grad = targets(T, V, g), row_grads(T, g)
    loss, lse = tg.linear_cross_entropy_forward(X, W, y)
    torch.cuda.synchronize()
    ref = Reference(X, W, y)
    ref.check_rows(loss, lse)
    dX, dW = tg.linear_cross_entropy_backward(grad, X, W, y, lse)
    torch.cuda.synchronize()
    assert dX.dtype == dW.dtype == X.dtype
    ref.check_gradients(grad.double(), dX, dW)


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("T,V,D,K,temperature", [(1, 5, 3, 1, 1.0), (6, 40, 64, 40, 2.0), (20, 1000, 128, 7, 1.0),
                                                 (130, 777, 200, 33, 3.0), (257, 2049, 64, 64, 0.5),
                                                 (300, 5003, 320, 100, 2.0), (8, 4000, 64, 1024, 1.5),
                                                 (5, 262144, 8, 90, 1.0), (40, 262145, 8, 33, 2.0),
                                                 (9, 600007, 16, 200, 1.0), (20, 16383, 24, 50, 1.0),
                                                 (7, 16384, 200, 128, 2.0)])
def test_distillation(kind, T, V, D, K, temperature):
    log(f"distillation {kind} {T}x{V}x{D} K={K} temperature={temperature}")
    X, W, g = head(T, V, D, TYPES[kind], 2)
    ids, logits = entries(T, V, K, TYPES[kind], g)
    grad = row_grads(T, g)
    loss, lse, student = tg.linear_distillation_forward(X, W, ids, logits, temperature=temperature)
    torch.cuda.synchronize()
    ref = Reference(X, W, ids=ids, logits=logits, temperature=temperature)
    ref.check_rows(loss, lse, student)
    dX, dW = tg.linear_distillation_backward(grad, X, W, ids, logits, lse, student, temperature=temperature)
    torch.cuda.synchronize()
    ref.check_gradients(grad.double(), dX, dW)


# rows apart and bases off 16 bytes: the copies that the matrix cores need
@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("D,pad,shift", [(64, 8, 0), (64, 3, 0), (128, 0, 1), (128, 8, 8), (100, 28, 4), (65, 0, 0)])
def test_strides_and_alignment(kind, D, pad, shift):
    T, V = 70, 333
    log(f"strides {kind} D={D} pad={pad} shift={shift}")
    dtype = TYPES[kind]
    X, W, g = head(T, V, D, dtype, 3, pad, shift)
    y, grad = targets(T, V, g), row_grads(T, g)
    loss, lse = tg.linear_cross_entropy_forward(X, W, y)
    room_x = torch.full((T, D + pad + shift), 7.0, dtype=dtype, device="cuda")
    room_w = torch.full((V, D + pad + shift), 7.0, dtype=dtype, device="cuda")
    dX, dW = room_x[:, shift:shift + D], room_w[:, shift:shift + D]
    tg.linear_cross_entropy_backward(grad, X, W, y, lse, dX=dX, dW=dW)
    torch.cuda.synchronize()
    ref = Reference(X, W, y)
    ref.check_rows(loss, lse)
    ref.check_gradients(grad.double(), dX, dW)
    for room in (room_x, room_w):  # nothing beside the gradients is written
        assert bool((room[:, :shift] == 7).all()) and bool((room[:, shift + D:] == 7).all())


# a few rows are read as they are stored, wherever that is
@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("T", [1, 7, 20, 32])
@pytest.mark.parametrize("D,pad,shift", [(1, 0, 0), (7, 2, 1), (33, 0, 0), (64, 1, 1), (100, 3, 5), (257, 0, 3), (1003, 2, 0)])
def test_few_rows_anywhere(kind, T, D, pad, shift):
    log(f"few rows {kind} T={T} D={D} pad={pad} shift={shift}")
    X, W, g = head(T, 150, D, TYPES[kind], 13, pad, shift)
    y, grad = targets(T, 150, g), row_grads(T, g)
    loss, lse = tg.linear_cross_entropy_forward(X, W, y)
    ref = Reference(X, W, y)
    ref.check_rows(loss, lse)
    room_x = torch.full((T, D + pad + shift), 7.0, dtype=X.dtype, device="cuda")
    room_w = torch.full((150, D + pad + shift), 7.0, dtype=X.dtype, device="cuda")
    dX, dW = room_x[:, shift:shift + D], room_w[:, shift:shift + D]
    tg.linear_cross_entropy_backward(grad, X, W, y, lse, dX=dX, dW=dW)
    torch.cuda.synchronize()
    ref.check_gradients(grad.double(), dX, dW)
    for room in (room_x, room_w):
        assert bool((room[:, :shift] == 7).all()) and bool((room[:, shift + D:] == 7).all())


@pytest.mark.parametrize("kind", ["bf16", "fp32"])
def test_vocabulary_in_pieces(kind):
    T, V, D = (8192, 20003, 64) if kind == "bf16" else (4096, 13001, 64)
    log(f"pieces {kind}")
    X, W, g = head(T, V, D, TYPES[kind], 4)
    y, grad = targets(T, V, g), row_grads(T, g)
    loss, lse = tg.linear_cross_entropy_forward(X, W, y)
    dX, dW = tg.linear_cross_entropy_backward(grad, X, W, y, lse)
    torch.cuda.synchronize()
    ref = Reference(X, W, y)
    ref.check_rows(loss, lse)
    ref.check_gradients(grad.double(), dX, dW)
    ids, logits = entries(T, V, 9, TYPES[kind], g)
    loss, lse, student = tg.linear_distillation_forward(X, W, ids, logits)
    dX, dW = tg.linear_distillation_backward(grad, X, W, ids, logits, lse, student)
    torch.cuda.synchronize()
    ref = Reference(X, W, ids=ids, logits=logits)
    ref.check_rows(loss, lse, student)
    ref.check_gradients(grad.double(), dX, dW)


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("filler", ["nan", "inf"])
def test_rows_that_do_not_count_may_hold_anything(kind, filler):
    T, V, D = 70, 300, 96
    X, W, g = head(T, V, D, TYPES[kind], 5)
    y, grad = targets(T, V, g), row_grads(T, g)
    X[y == -100] = float(filler)
    grad[y == -100] = float(filler)
    loss, lse = tg.linear_cross_entropy_forward(X, W, y)
    dX, dW = tg.linear_cross_entropy_backward(grad, X, W, y, lse)
    torch.cuda.synchronize()
    clean = torch.where((y != -100)[:, None], X, 0.0)
    ref = Reference(clean, W, y)
    ref.check_rows(loss, lse)
    ref.check_gradients(torch.where(y != -100, grad, 0.0).double(), dX, dW)


@pytest.mark.parametrize("kind", TYPES)
def test_no_row_counts(kind):
    T, V, D = 9, 100, 64
    X, W, g = head(T, V, D, TYPES[kind], 6)
    y = torch.full((T,), -100, device="cuda")
    X.requires_grad_()
    W.requires_grad_()
    loss = tg.linear_cross_entropy(X, W, y)
    dX, dW = torch.autograd.grad(loss, (X, W))
    assert float(loss.detach()) == 0 and not bool(dX.any()) and not bool(dW.any())
    ids, logits = entries(T, V, 4, TYPES[kind], g)
    logits.fill_(float("-inf"))
    loss = tg.linear_distillation(X, W, ids, logits)
    dX, dW = torch.autograd.grad(loss, (X, W))
    assert float(loss.detach()) == 0 and not bool(dX.any()) and not bool(dW.any())


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("bad", [-1, 300, 2 ** 40, -2 ** 62])
def test_an_index_out_of_range_gives_nan(kind, bad):
    T, V, D = 40, 300, 64
    X, W, g = head(T, V, D, TYPES[kind], 7)
    y, grad = targets(T, V, g), row_grads(T, g)
    y[7] = bad
    loss, lse = tg.linear_cross_entropy_forward(X, W, y)
    dX, dW = tg.linear_cross_entropy_backward(grad, X, W, y, lse)
    nan = torch.isnan(loss)
    assert nan.nonzero()[:, 0].tolist() == [7]
    assert torch.isnan(dX).all(dim=1).nonzero()[:, 0].tolist() == [7] and int(torch.isnan(dX).sum()) == D
    assert bool(torch.isnan(dW).all())
    ids, logits = entries(T, V, 5, TYPES[kind], g)
    ids[9, 2], logits[9, 2] = bad, 0.0
    loss, lse, student = tg.linear_distillation_forward(X, W, ids, logits)
    dX, dW = tg.linear_distillation_backward(grad, X, W, ids, logits, lse, student)
    assert torch.isnan(loss).nonzero()[:, 0].tolist() == [9]
    assert torch.isnan(dX).all(dim=1).nonzero()[:, 0].tolist() == [9] and int(torch.isnan(dX).sum()) == D
    assert bool(torch.isnan(dW).all())


def test_an_empty_batch():
    W = torch.ones((50, 64), device="cuda")
    X = torch.empty((0, 64), device="cuda")
    y = torch.empty((0,), dtype=torch.int64, device="cuda")
    loss, lse = tg.linear_cross_entropy_forward(X, W, y)
    assert loss.shape == lse.shape == (0,)
    dW = torch.full_like(W, 3.0)
    dX, _ = tg.linear_cross_entropy_backward(torch.empty(0, device="cuda"), X, W, y, lse, dW=dW)
    assert dX.shape == (0, 64) and not bool(dW.any())
    W.requires_grad_()
    mean = tg.linear_cross_entropy(X, W, y)
    (dW,) = torch.autograd.grad(mean, (W,))
    assert float(mean) == 0 and not bool(dW.any())


# uneven factors of the rows: fp16 scales each row by its own power of two
@pytest.mark.parametrize("kind", TYPES)
def test_row_factors_of_many_sizes(kind):
    T, V, D = 60, 500, 64
    X, W, g = head(T, V, D, TYPES[kind], 8)
    y = targets(T, V, g)
    grad = torch.ldexp(row_grads(T, g), torch.randint(-24, 3, (T,), generator=g, device="cuda"))
    grad[11] = 0.0
    loss, lse = tg.linear_cross_entropy_forward(X, W, y)
    dX, dW = tg.linear_cross_entropy_backward(grad, X, W, y, lse)
    torch.cuda.synchronize()
    Reference(X, W, y).check_gradients(grad.double(), dX, dW)


@pytest.mark.parametrize("kind", TYPES)
def test_only_what_is_needed(kind):
    T, V, D = 100, 400, 128
    X, W, g = head(T, V, D, TYPES[kind], 9)
    y, grad = targets(T, V, g), row_grads(T, g)
    loss, lse = tg.linear_cross_entropy_forward(X, W, y)
    both = tg.linear_cross_entropy_backward(grad, X, W, y, lse)
    dX, none = tg.linear_cross_entropy_backward(grad, X, W, y, lse, need=(True, False))
    assert none is None and torch.equal(dX, both[0])
    none, dW = tg.linear_cross_entropy_backward(grad, X, W, y, lse, need=(False, True))
    assert none is None and torch.equal(dW, both[1])
    one = torch.full((), 0.5, device="cuda")
    a = tg.linear_cross_entropy_backward(one, X, W, y, lse)
    b = tg.linear_cross_entropy_backward(one.expand(T).contiguous(), X, W, y, lse)
    assert all(torch.equal(p, q) for p, q in zip(a, b))


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("reduction", ["mean", "sum", "none"])
def test_differentiable(kind, reduction):
    T, V, D = 90, 600, 128
    X, W, g = head(T, V, D, TYPES[kind], 10)
    y = targets(T, V, g)
    ids, logits = entries(T, V, 12, TYPES[kind], g)
    X.requires_grad_()
    W.requires_grad_()
    for loss, ref in ((tg.linear_cross_entropy(X, W, y, reduction=reduction), Reference(X.detach(), W.detach(), y)),
                      (tg.linear_distillation(X, W, ids, logits, temperature=2.0, reduction=reduction),
                       Reference(X.detach(), W.detach(), ids=ids, logits=logits, temperature=2.0))):
        n = int(ref.counts.sum())
        assert loss.dtype == torch.float32 and loss.shape == ((T,) if reduction == "none" else ())
        up = torch.randn(loss.shape, generator=g, device="cuda")
        grad = up.double() * (1.0 / n if reduction == "mean" else 1.0)
        want = ref.loss if reduction == "none" else ref.loss.sum() / (n if reduction == "mean" else 1)
        off = ref.loss_off * ref.counts
        off = off if reduction == "none" else off.sum() / (n if reduction == "mean" else 1) + 2 ** -23 * want.abs()
        assert bool(((loss.double() - want).abs() <= off).all())
        dX, dW = torch.autograd.grad(loss, (X, W), up)
        # the factor of a row is rounded twice on its way
        ref.check_gradients((grad * torch.ones(T, device="cuda")).double(), dX, dW)


def test_gradient_against_differences():
    T, V, D = 12, 50, 8
    X, W, g = head(T, V, D, torch.float32, 11)
    y = targets(T, V, g)
    ids, logits = entries(T, V, 6, torch.float32, g)
    X.requires_grad_()
    W.requires_grad_()
    for name, f, ref in (
            ("ce", lambda: tg.linear_cross_entropy(X, W, y),
             lambda x, w: Reference(x, w, y)),
            ("kd", lambda: tg.linear_distillation(X, W, ids, logits, temperature=1.5),
             lambda x, w: Reference(x, w, ids=ids, logits=logits, temperature=1.5))):
        dX, dW = torch.autograd.grad(f(), (X, W))
        x, w = X.detach().double(), W.detach().double()
        for _ in range(4):
            ux = torch.randn((T, D), generator=g, device="cuda").double()
            uw = torch.randn((V, D), generator=g, device="cuda").double()

            def at(h):
                r = ref(x + h * ux, w + h * uw)
                return float(r.loss.sum() / r.counts.sum())
            h = 1e-5
            slope = (at(h) - at(-h)) / (2 * h)
            got = float((dX.double() * ux).sum() + (dW.double() * uw).sum())
            # float32 gradients (2^-20 of the sum of magnitudes) and the third derivative's h²
            room = float((dX.double() * ux).abs().sum() + (dW.double() * uw).abs().sum())
            assert abs(slope - got) <= 2.0 ** -20 * room + 1e-7, (name, slope, got)


@pytest.mark.parametrize("kind", TYPES)
def test_the_same_call_gives_the_same_bits(kind):
    X, W, g = head(300, 3000, 256, TYPES[kind], 12)
    y, grad = targets(300, 3000, g), row_grads(300, g)
    first = None
    for _ in range(3):
        loss, lse = tg.linear_cross_entropy_forward(X, W, y)
        out = (loss, lse, *tg.linear_cross_entropy_backward(grad, X, W, y, lse))
        if first is None:
            first = out
        assert all(torch.equal(a, b) for a, b in zip(first, out))


def test_workspaces_of_the_caller():
    T, V, D = 100, 700, 72
    X, W, g = head(T, V, D, torch.bfloat16, 13)
    y, grad = targets(T, V, g), row_grads(T, g)
    want = tg.linear_cross_entropy_forward(X, W, y)
    want += tg.linear_cross_entropy_backward(grad, X, W, y, want[1])
    args = (_lib.TGEMM_BF16, T, V, D, X.data_ptr(), D, W.data_ptr(), D, 0)
    for backward in (0, 1):
        need = tg.tgemm_linear_loss_workspace_size(*args, backward)
        room = torch.full((need + 4096,), 0xFF, dtype=torch.uint8, device="cuda")  # its contents do not matter: NaN
        ws = room[:need]
        if backward:
            got = tg.linear_cross_entropy_backward(grad, X, W, y, want[1], workspace=ws)
            assert all(torch.equal(a, b) for a, b in zip(got, want[2:]))
        else:
            got = tg.linear_cross_entropy_forward(X, W, y, workspace=ws)
            assert all(torch.equal(a, b) for a, b in zip(got, want[:2]))
        assert bool((room[need:] == 0xFF).all())
        with pytest.raises(tg.TgemmError):
            tg.linear_cross_entropy_backward(grad, X, W, y, want[1], workspace=ws[:64])


@pytest.mark.parametrize("kind", TYPES)
def test_captured_and_replayed(kind):
    """Forward and backward of both losses in one graph, replayed on new inputs with eager work between."""
    T, V, D, K = 96, 1000, 128, 8
    X, W, g = head(T, V, D, TYPES[kind], 14)
    y, (ids, logits), grad = targets(T, V, g), entries(T, V, K, TYPES[kind], g), row_grads(T, g)

    def step():
        loss, lse = tg.linear_cross_entropy_forward(X, W, y)
        a = tg.linear_cross_entropy_backward(grad, X, W, y, lse)
        kd, lse2, student = tg.linear_distillation_forward(X, W, ids, logits, temperature=2.0)
        b = tg.linear_distillation_backward(grad, X, W, ids, logits, lse2, student, temperature=2.0)
        return (loss, lse, *a, kd, lse2, student, *b)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for seed in range(4):
        g = generator(100 + seed)
        X.copy_(torch.randn((T, D), generator=g, device="cuda"))
        y.copy_(targets(T, V, g))
        ids.copy_(torch.randint(0, V, (T, K), generator=g, device="cuda"))
        graph.replay()
        torch.cuda.synchronize()
        want = step()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want)), f"replay {seed}"


def test_on_another_stream():
    T, V, D = 200, 3000, 256
    X, W, g = head(T, V, D, torch.bfloat16, 15)
    y, grad = targets(T, V, g), row_grads(T, g)
    want = tg.linear_cross_entropy_forward(X, W, y)
    want += tg.linear_cross_entropy_backward(grad, X, W, y, want[1])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    loss, lse = tg.linear_cross_entropy_forward(X, W, y, stream=side.cuda_stream)
    junk = [torch.full((1 << 16,), float("nan"), device="cuda") for _ in range(8)]  # takes memory released meanwhile
    dX, dW = tg.linear_cross_entropy_backward(grad, X, W, y, lse, stream=side.cuda_stream)
    del junk
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip((loss, lse, dX, dW), want))
    with torch.cuda.stream(side):
        got = tg.linear_cross_entropy_forward(X, W, y)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got[0], want[0])


@pytest.mark.parametrize("kind,teacher", [("bf16", "fp32"), ("fp32", "bf16"), ("fp16", "fp32"), ("bf16", "fp16")])
def test_a_teacher_of_another_type(kind, teacher):
    T, V, D, K = 70, 900, 128, 17
    X, W, g = head(T, V, D, TYPES[kind], 17)
    ids, logits = entries(T, V, 2 * K, TYPES[teacher], g)
    ids, logits = ids[:, :K], logits[:, 3:K + 3]  # rows apart
    logits[(ids < 0) | (ids >= V)] = float("-inf")
    grad = row_grads(T, g)
    loss, lse, student = tg.linear_distillation_forward(X, W, ids, logits, temperature=2.5)
    dX, dW = tg.linear_distillation_backward(grad, X, W, ids, logits, lse, student, temperature=2.5)
    torch.cuda.synchronize()
    ref = Reference(X, W, ids=ids, logits=logits, temperature=2.5)
    ref.check_rows(loss, lse, student)
    ref.check_gradients(grad.double(), dX, dW)


@pytest.mark.parametrize("kind", TYPES)
def test_strided_targets_and_factors(kind):
    """A target and factors that are every second element of others, on another stream."""
    T, V, D = 90, 500, 64
    X, W, g = head(T, V, D, TYPES[kind], 18)
    y2, grad2 = targets(2 * T, V, g), row_grads(2 * T, g)
    y, grad = y2[::2], grad2[::2]
    want = tg.linear_cross_entropy_forward(X, W, y.clone())
    want += tg.linear_cross_entropy_backward(grad.clone(), X, W, y.clone(), want[1])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    loss, lse = tg.linear_cross_entropy_forward(X, W, y, stream=side.cuda_stream)
    got = (loss, lse, *tg.linear_cross_entropy_backward(grad, X, W, y, lse, stream=side.cuda_stream))
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_two_streams_at_once():
    T, V, D = 300, 4000, 256
    X, W, g = head(T, V, D, torch.bfloat16, 19)
    y = [targets(T, V, g) for _ in range(2)]
    grad = row_grads(T, g)
    want = []
    for t in y:
        loss, lse = tg.linear_cross_entropy_forward(X, W, t)
        want.append((loss, lse, *tg.linear_cross_entropy_backward(grad, X, W, t, lse)))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(3):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                loss, lse = tg.linear_cross_entropy_forward(X, W, y[i])
                got[i].append((loss, lse, *tg.linear_cross_entropy_backward(grad, X, W, y[i], lse)))
    torch.cuda.synchronize()
    for i in range(2):
        for out in got[i]:
            assert all(torch.equal(a, b) for a, b in zip(out, want[i]))


@pytest.mark.parametrize("kind", ["bf16", "fp32"])
def test_saved_tensors_may_be_stored_elsewhere(kind):
    """torch's hooks on what the backward pass keeps: rows that were apart come back together."""
    T, V, D = 40, 300, 64
    X, W, g = head(T, V, D, TYPES[kind], 20, pad=16)
    y = targets(T, V, g)
    X.requires_grad_()
    W.requires_grad_()
    want = torch.autograd.grad(tg.linear_cross_entropy(X, W, y), (X, W))
    with torch.autograd.graph.saved_tensors_hooks(lambda t: t.cpu(), lambda t: t.cuda()):
        loss = tg.linear_cross_entropy(X, W, y)
    loss_before = float(loss.detach())
    got = torch.autograd.grad(loss, (X, W), retain_graph=True)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    again = torch.autograd.grad(loss, (X, W))
    assert all(torch.equal(a, b) for a, b in zip(again, want)) and float(loss.detach()) == loss_before


def test_a_loss_may_be_changed_in_place():
    T, V, D = 40, 300, 64
    X, W, g = head(T, V, D, torch.bfloat16, 21)
    y = targets(T, V, g)
    X.requires_grad_()
    W.requires_grad_()
    for reduction in ("mean", "sum", "none"):
        loss = tg.linear_cross_entropy(X, W, y, reduction=reduction)
        half = tg.linear_cross_entropy(X, W, y, reduction=reduction) * 0.5
        loss *= 0.5
        a = torch.autograd.grad(loss.sum(), (X, W))
        b = torch.autograd.grad(half.sum(), (X, W))
        assert all(torch.equal(p, q) for p, q in zip(a, b))


def test_trained_together():
    """A student's steps on both losses with one weight: the gradients of their sum, accumulated over two parts of a
    batch, against the formulas."""
    T, V, D, K = 64, 500, 64, 10
    X, W, g = head(T, V, D, torch.float32, 16)
    y, (ids, logits) = targets(T, V, g), entries(T, V, K, torch.float32, g)
    weight = torch.nn.Parameter(W.clone())
    hidden = torch.nn.Parameter(X.clone())
    opt = torch.optim.SGD([weight, hidden], lr=0.1)
    for _ in range(3):
        opt.zero_grad()
        want_x, want_w = torch.zeros_like(hidden, dtype=torch.float64), torch.zeros_like(weight, dtype=torch.float64)
        off_w = torch.zeros_like(want_w)
        for part in (slice(0, 40), slice(40, T)):
            x = hidden[part]
            loss = (0.3 * tg.linear_cross_entropy(x, weight, y[part], reduction="sum")
                    + 0.7 * tg.linear_distillation(x, weight, ids[part], logits[part], temperature=2.0, reduction="sum"))
            loss.backward()
            for f, r in ((0.3, Reference(x.detach(), weight.detach(), y[part])),
                         (0.7, Reference(x.detach(), weight.detach(), ids=ids[part], logits=logits[part], temperature=2.0))):
                gx, ox, gw, ow = r.gradients(torch.full((x.shape[0],), f, dtype=torch.float64, device="cuda"))
                want_x[part] += gx
                want_w += gw
                off_w += ow + 2.0 ** -22 * gw.abs()
        assert bool(((weight.grad.double() - want_w).abs() <= off_w).all())
        assert float((hidden.grad.double() - want_x).norm() / want_x.norm()) < 2.0 ** -16
        opt.step()


# the products kept for the backward pass: by the tiles of each size, by the few rows' kernel, in rows that start
# anywhere, with nothing written between them
@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("T,V,D,pad", [(1, 1, 1, 0), (5, 301, 40, 2), (20, 1000, 72, 0), (33, 1001, 128, 1), (64, 30000, 64, 0),
                                       (130, 777, 200, 3), (300, 5003, 65, 0), (700, 4099, 320, 5)])
def test_kept_logits(kind, T, V, D, pad):
    log(f"kept {kind} {T}x{V}x{D} pad={pad}")
    X, W, g = head(T, V, D, TYPES[kind], 14)
    y, grad = targets(T, V, g), row_grads(T, g)
    room = torch.full((T, V + pad), 7.0, device="cuda")
    Z = room[:, :V]
    for distill in (False, True):
        if distill:
            ids, top = entries(T, V, min(V, 9), TYPES[kind], g)
            loss, lse, student = tg.linear_distillation_forward(X, W, ids, top, temperature=2.0, logits=Z)
            ref = Reference(X, W, ids=ids, logits=top, temperature=2.0)
            ref.check_rows(loss, lse, student)
            dX, dW = tg.linear_distillation_backward(grad, X, W, ids, top, lse, student, temperature=2.0, logits=Z)
        else:
            loss, lse = tg.linear_cross_entropy_forward(X, W, y, logits=Z)
            ref = Reference(X, W, y)
            ref.check_rows(loss, lse)
            dX, dW = tg.linear_cross_entropy_backward(grad, X, W, y, lse, logits=Z)
        torch.cuda.synchronize()
        # the reference's tolerance counts the products of rows that count (the others are cleared in it)
        assert bool(((Z.double() - ref.z * ref.tau).abs() <= ref.z_off * ref.tau)[ref.counts].all())
        assert bool((room[:, V:] == 7).all())
        ref.check_gradients(grad.double(), dX, dW)
        if not distill:  # for one of the gradients only
            only = tg.linear_cross_entropy_backward(grad, X, W, y, lse, logits=Z, need=(False, True))
            assert only[0] is None and torch.equal(only[1], dW)
            only = tg.linear_cross_entropy_backward(grad, X, W, y, lse, logits=Z, need=(True, False))
            assert only[1] is None and torch.equal(only[0], dX)


@pytest.mark.parametrize("kind", ["bf16", "fp32"])
def test_kept_logits_in_pieces(kind):
    T, V, D = (8192, 20003, 64) if kind == "bf16" else (4096, 13001, 64)
    log(f"kept in pieces {kind}")
    X, W, g = head(T, V, D, TYPES[kind], 15)
    y, grad = targets(T, V, g), row_grads(T, g)
    Z = torch.empty((T, V), device="cuda")
    loss, lse = tg.linear_cross_entropy_forward(X, W, y, logits=Z)
    kept = tg.linear_cross_entropy_backward(grad, X, W, y, lse, logits=Z)
    again = tg.linear_cross_entropy_backward(grad, X, W, y, lse)
    torch.cuda.synchronize()
    # the same products, the same arithmetic on them
    assert torch.equal(kept[0], again[0]) and torch.equal(kept[1], again[1])


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("T,V,D", [(12, 900, 64), (200, 900, 256), (40, 300, 1032)])
def test_differentiable_with_kept_logits(kind, T, V, D):
    log(f"differentiable, kept {kind} {T}x{V}x{D}")
    X, W, g = head(T, V, D, TYPES[kind], 16)
    X, W = X.contiguous().requires_grad_(), W.contiguous().requires_grad_()
    y = targets(T, V, g)
    X.data[2] = float("nan")  # a row that does not count
    ref = Reference(X.detach(), W.detach(), y)
    one = torch.full((T,), 1.0 / int(ref.counts.sum()), dtype=torch.float64, device="cuda")
    for keep in (True, False, None):
        loss = tg.linear_cross_entropy(X, W, y, keep_logits=keep)
        first = torch.autograd.grad(loss, (X, W), retain_graph=True)
        second = torch.autograd.grad(loss, (X, W))
        torch.cuda.synchronize()
        ref.check_gradients(one, *first)
        assert torch.equal(first[0], second[0]) and torch.equal(first[1], second[1])
    ids, top = entries(T, V, 7, TYPES[kind], g)
    X.data[2] = 0.5
    ref = Reference(X.detach(), W.detach(), ids=ids, logits=top, temperature=1.5)
    for keep in (True, False):
        loss = tg.linear_distillation(X, W, ids, top, temperature=1.5, reduction="sum", keep_logits=keep)
        ref.check_gradients(torch.ones(T, dtype=torch.float64, device="cuda"), *torch.autograd.grad(loss, (X, W)))


def test_kept_logits_and_an_index_out_of_range():
    X, W, g = head(40, 100, 64, torch.bfloat16, 17)
    y = torch.randint(0, 100, (40,), generator=g, device="cuda")
    y[7] = 100
    Z = torch.empty((40, 100), device="cuda")
    loss, lse = tg.linear_cross_entropy_forward(X, W, y, logits=Z)
    dX, dW = tg.linear_cross_entropy_backward(torch.ones(40, device="cuda"), X, W, y, lse, logits=Z)
    torch.cuda.synchronize()
    bad = torch.arange(40, device="cuda") == 7
    assert bool(torch.isnan(loss[bad]).all()) and bool(torch.isnan(dX[bad]).all()) and bool(torch.isnan(dW).all())
    assert bool(torch.isfinite(loss[~bad]).all()) and bool(torch.isfinite(dX[~bad]).all())


def test_a_step_with_kept_logits_captured_and_replayed():
    log("kept, captured")
    T, V, D = 150, 2000, 1024
    X, W, g = head(T, V, D, torch.bfloat16, 18)
    y, grad = targets(T, V, g), row_grads(T, g)
    Z = torch.empty((T, V), device="cuda")
    loss, lse = torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
    dX, dW = torch.empty_like(X), torch.empty_like(W)

    def step():
        tg.linear_cross_entropy_forward(X, W, y, loss=loss, lse=lse, logits=Z)
        tg.linear_cross_entropy_backward(grad, X, W, y, lse, logits=Z, dX=dX, dW=dW)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for n in range(3):
        X.copy_(torch.randn((T, D), generator=g, device="cuda"))
        step()
        torch.cuda.synchronize()
        want = [t.clone() for t in (loss, lse, dX, dW)]
        for t in (loss, lse, dX, dW, Z):
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for have, t in zip((loss, lse, dX, dW), want):
            assert torch.equal(have, t)


def peak(call):
    torch.cuda.synchronize()
    before = torch.cuda.memory_allocated()
    torch.cuda.reset_peak_memory_stats()
    call()
    torch.cuda.synchronize()
    return torch.cuda.max_memory_allocated() - before


def test_logits_are_held_only_where_a_gradient_can_come():
    log("what is held")
    T, V, D = 1000, 20000, 1024
    X, W, g = head(T, V, D, torch.bfloat16, 19)
    X, W = X.contiguous().requires_grad_(), W.contiguous().requires_grad_()
    y = targets(T, V, g)
    ids, top = entries(T, V, 4, torch.bfloat16, g)
    logits = 4 * T * V
    for call in (lambda **k: tg.linear_cross_entropy(X, W, y, **k), lambda **k: tg.linear_distillation(X, W, ids, top, **k)):
        assert peak(lambda: call()) > logits
        assert peak(lambda: call(keep_logits=False)) < logits // 4
        with torch.no_grad():
            for keep in (None, True):
                assert peak(lambda: call(keep_logits=keep)) < logits // 4


def test_a_step_holds_a_small_part_of_large_logits():
    log("peak of a step")
    T, V, D = 8192, 131072, 64
    X, W, g = head(T, V, D, torch.bfloat16, 20)
    X, W = X.contiguous().requires_grad_(), W.contiguous().requires_grad_()
    y = targets(T, V, g)
    # a piece of the logits' gradient (256 MiB and a row's padding), sums in float32, statistics
    assert peak(lambda: torch.autograd.grad(tg.linear_cross_entropy(X, W, y), (X, W))) < 4 * T * V // 8


@pytest.mark.parametrize("keep", [False, True])
def test_differentiable_on_a_side_stream(keep):
    log(f"side stream, kept {keep}")
    T, V, D = 200, 3000, 256
    X, W, g = head(T, V, D, torch.bfloat16, 21)
    X, W = X.contiguous().requires_grad_(), W.contiguous().requires_grad_()
    y = targets(T, V, g)
    want = torch.autograd.grad(tg.linear_cross_entropy(X, W, y, keep_logits=keep), (X, W))
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        with torch.cuda.stream(side):
            loss = tg.linear_cross_entropy(X, W, y, keep_logits=keep)
        junk = [torch.full((T, V), 3.0, device="cuda") for _ in range(4)]  # would land on memory handed back too soon
        have = torch.autograd.grad(loss, (X, W))  # torch runs it on `side`, and this stream waits for it
        torch.cuda.synchronize()
        assert torch.equal(have[0], want[0]) and torch.equal(have[1], want[1])
        del junk
