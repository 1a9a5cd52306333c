"""The loss operators on streams of the caller's that are behind: the calls
return before their kernels start, and what they allocated stays theirs."""

import pytest

torch = pytest.importorskip("torch")

import tiled_gemm_tgemm_amd as tg  # noqa: E402
from test_gpu_linear_loss import entries, gpu, head, row_grads, targets  # noqa: E402,F401
from tiled_gemm_tgemm_amd import _lib  # noqa: E402

pytestmark = pytest.mark.gpu

T, V, D, K = 600, 9000, 256, 8


def later(*streams):
    """Some 20 ms of products on each stream, before what is queued next; the current stream goes on."""
    x = torch.randn((8192, 8192), device="cuda").to(torch.bfloat16)
    out = [torch.empty_like(x) for _ in streams]
    torch.mm(x, x, out=out[0])  # what the library sets up on its first use
    torch.cuda.synchronize()
    for s, o in zip(streams, out):
        with torch.cuda.stream(s):
            for _ in range(25):
                torch.mm(x, x, out=o)
    return x, out


def take(X, W, k, backward):
    """Allocates what such a call's workspace takes on the current stream, some times over, and writes to it."""
    need = tg.tgemm_linear_loss_workspace_size(_lib.TGEMM_BF16, T, V, D, X.data_ptr(), D, W.data_ptr(), D, k, backward)
    return [torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda") for _ in range(3)]


@pytest.mark.parametrize("distill", [False, True])
def test_a_workspace_is_not_handed_out_before_its_kernels_ran(distill):
    X, W, g = head(T, V, D, torch.bfloat16, 31)
    y, (ids, top), grad = targets(T, V, g), entries(T, V, K, torch.bfloat16, g), row_grads(T, g)

    def forward(**k):
        return tg.linear_distillation_forward(X, W, ids, top, **k) if distill else tg.linear_cross_entropy_forward(X, W, y, **k)

    def backward(rows, **k):
        if distill:
            return tg.linear_distillation_backward(grad, X, W, ids, top, *rows[1:], **k)
        return tg.linear_cross_entropy_backward(grad, X, W, y, rows[1], **k)

    want = forward()
    want += backward(want)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    held = later(side)
    rows = forward(stream=side.cuda_stream)
    junk = take(X, W, K if distill else 0, 0)
    del junk
    got = rows + backward(rows, stream=side.cuda_stream)
    junk = take(X, W, K if distill else 0, 1)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    del junk, held


def test_two_late_streams_of_one_thread():
    X, W, g = head(T, V, D, torch.bfloat16, 32)
    ys, grad = [targets(T, V, g) for _ in range(2)], row_grads(T, g)
    want = []
    for y in ys:
        loss, lse = tg.linear_cross_entropy_forward(X, W, y)
        want.append((loss, lse, *tg.linear_cross_entropy_backward(grad, X, W, y, lse)))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    held = later(*streams)
    rows = [tg.linear_cross_entropy_forward(X, W, y, stream=s.cuda_stream) for y, s in zip(ys, streams)]
    got = [(*r, *tg.linear_cross_entropy_backward(grad, X, W, y, r[1], stream=s.cuda_stream))
           for r, y, s in zip(rows, ys, streams)]
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert all(torch.equal(p, q) for p, q in zip(a, b))
    del held


@pytest.mark.parametrize("keep", [False, True])
def test_a_node_called_under_a_late_stream(keep):
    X, W, g = head(T, V, D, torch.bfloat16, 33)
    X, W = X.contiguous().requires_grad_(), W.contiguous().requires_grad_()
    y = targets(T, V, g)
    loss = tg.linear_cross_entropy(X, W, y, keep_logits=keep)
    one = torch.ones((), device="cuda")
    want = torch.autograd.grad(loss, (X, W), one, retain_graph=True)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    held = later(side)
    with torch.cuda.stream(side):
        got = loss.grad_fn.apply(one)[:2]
    junk = take(X, W, 0, 1)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    del junk, held


@pytest.mark.parametrize("distill", [False, True])
@pytest.mark.parametrize("reduction,keep", [("mean", True), ("mean", False), ("none", None)])
def test_a_differentiable_step_captured_and_replayed(distill, reduction, keep):
    """Both passes in one graph, on inputs that change between its replays, with eager steps between them."""
    X, W, g = head(T, V, D, torch.bfloat16, 34)
    y, (ids, top) = targets(T, V, g), entries(T, V, K, torch.bfloat16, g)
    up = torch.rand((T,) if reduction == "none" else (), generator=g, device="cuda")

    def step(x, w):
        loss = (tg.linear_distillation(x, w, ids, top, reduction=reduction, keep_logits=keep) if distill
                else tg.linear_cross_entropy(x, w, y, reduction=reduction, keep_logits=keep))
        return (loss.detach(), *torch.autograd.grad(loss, (x, w), up))

    def leaves():  # of each step's own
        return X.detach().requires_grad_(), W.detach().requires_grad_()

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(*leaves())
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    x, w = leaves()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(x, w)
    for seed in range(3):
        X.copy_(torch.randn((T, D), generator=g, device="cuda"))
        want = [t.clone() for t in step(*leaves())]
        for t in out:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want)), f"replay {seed}"


def test_steps_of_several_threads_at_once():
    """Threads share torch's current stream by default, and torch's backward thread."""
    import concurrent.futures

    X, W, g = head(T, V, D, torch.bfloat16, 35)
    ys, (ids, top) = [targets(T, V, g) for _ in range(4)], entries(T, V, K, torch.bfloat16, g)

    def step(y, distill):
        x, w = X.detach().requires_grad_(), W.detach().requires_grad_()
        loss = tg.linear_distillation(x, w, ids, top) if distill else tg.linear_cross_entropy(x, w, y)
        first = torch.autograd.grad(loss, (x, w), retain_graph=True)
        return (loss.detach(), *first, *torch.autograd.grad(loss, (x, w)))

    calls = [(y, distill) for y in ys for distill in (False, True)]
    want = [step(*c) for c in calls]
    torch.cuda.synchronize()
    with concurrent.futures.ThreadPoolExecutor(4) as pool:
        for _ in range(5):
            got = list(pool.map(lambda c: step(*c), calls))
            torch.cuda.synchronize()
            for a, b in zip(got, want):
                assert all(torch.equal(p, q) for p, q in zip(a, b))


def test_two_threads_through_one_graph():
    import concurrent.futures

    X, W, g = head(T, V, D, torch.bfloat16, 36)
    x, w = X.detach().requires_grad_(), W.detach().requires_grad_()
    y = targets(T, V, g)
    loss = tg.linear_cross_entropy(x, w, y)
    want = torch.autograd.grad(loss, (x, w), retain_graph=True)
    with concurrent.futures.ThreadPoolExecutor(4) as pool:
        for got in pool.map(lambda n: torch.autograd.grad(loss, (x, w), retain_graph=True), range(24)):
            assert all(torch.equal(p, q) for p, q in zip(got, want))
