"""The operators together, as fine-tuning uses them: a projection with adapters
of several tasks in one batch, an output head's loss on it, the gradients of the
adapters, and their orthogonalised updates."""

import math
import threading

import pytest

torch = pytest.importorskip("torch")

import tiled_gemm_tgemm_amd as tg  # noqa: E402
from test_gpu_orthogonalize import chain, error  # noqa: E402

pytestmark = pytest.mark.gpu


def model(T, D, N, V, L, r, dtype, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    n = lambda *s: torch.randn(s, generator=g, device="cuda")
    X, W = n(T, D).to(dtype), (n(N, D) / math.sqrt(D)).to(dtype)
    A, B = (n(L, r, D) / math.sqrt(D)).to(dtype), (n(L, N, r) * 0.1).to(dtype)
    head = (n(V, N) / math.sqrt(N)).to(dtype)
    ids = torch.randint(-1, L, (T // 40 + 1,), generator=g, device="cuda").repeat_interleave(40)[:T].contiguous()
    return X, W, A, B, ids, torch.rand(L, generator=g, device="cuda") + 0.5, head, torch.randint(0, V, (T,), generator=g, device="cuda")


def step(X, W, A, B, ids, scales, head, target):
    hidden = tg.linear_adapters(X, W, A, B, ids, scales=scales)
    loss = tg.linear_cross_entropy(hidden, head, target)
    dA, dB = torch.autograd.grad(loss, (A, B))
    return loss.detach(), dA, dB, tg.orthogonalize(dA), tg.orthogonalize(dB)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("sizes", [(50, 96, 128, 300, 3, 4), (600, 256, 192, 1000, 4, 16), (1300, 200, 264, 777, 2, 80)])
def test_a_step(sizes, dtype):
    X, W, A, B, ids, scales, head, target = model(*sizes, dtype, 1)
    A.requires_grad_(), B.requires_grad_()
    loss, dA, dB, uA, uB = step(X, W, A, B, ids, scales, head, target)
    a, b = A.detach().double().requires_grad_(), B.detach().double().requires_grad_()
    y = X.double() @ W.double().t()
    for i in range(A.shape[0]):
        mine = (ids == i).double()[:, None] * float(scales[i])
        y = y + mine * ((X.double() @ a[i].t()) @ b[i].t())
    # the hidden states between the two are rounded to the type
    want = torch.nn.functional.cross_entropy(y @ head.double().t(), target)
    ga, gb = torch.autograd.grad(want, (a, b))
    half = torch.finfo(dtype).eps / 2
    # the loss: of a mean over T rows of log-sums, each off by what the rounded states do to a row's logits
    assert abs(float(loss) - float(want.detach())) <= 8 * half * float(y.detach().norm(dim=1).max()) / math.sqrt(y.shape[1]) + 2.0 ** -18
    # gradients: roundings of the states, of the logits' gradient, of the states' gradient and their own, and what the
    # first of these turns the second by (as much again, as a logit's error is its probability's relative one)
    for got, exact in ((dA, ga), (dB, gb)):
        assert error(got, exact) <= 8 * half + 2.0 ** -18
    # the updates of the gradients as they came out
    for got, grad in ((uA, dA), (uB, dB)):
        ref = chain(grad)
        for i in range(len(grad)):
            assert error(got[i], ref[i]) <= (half + 2.0 ** -9 if dtype == torch.bfloat16 else 2.0 ** -15)


def test_some_steps_and_a_captured_one():
    X, W, A, B, ids, scales, head, target = model(400, 128, 192, 500, 3, 8, torch.bfloat16, 2)
    A.requires_grad_(), B.requires_grad_()
    for _ in range(3):  # as a program does before it captures
        loss, dA, dB, uA, uB = step(X, W, A, B, ids, scales, head, target)
        with torch.no_grad():
            A -= 0.01 * uA
            B -= 0.01 * uB
    del loss, dA, dB, uA, uB
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(2):
            step(X, W, A, B, ids, scales, head, target)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(X, W, A, B, ids, scales, head, target)
    for seed in (3, 4, 5):
        fresh = model(400, 128, 192, 500, 3, 8, torch.bfloat16, seed)
        with torch.no_grad():
            for t, v in zip((X, W, A, B, ids, scales, head, target), fresh):
                t.copy_(v)
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in out]
        want = step(X, W, A, B, ids, scales, head, target)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        del want


def test_steps_from_several_threads():
    cases = [model(300 + 60 * i, 128, 192, 500, 3, 8, torch.bfloat16, 10 + i) for i in range(4)]
    for c in cases:
        c[2].requires_grad_(), c[3].requires_grad_()
    want = [step(*c) for c in cases]
    torch.cuda.synchronize()
    got = [[] for _ in cases]

    def work(i):
        stream = torch.cuda.Stream()
        with torch.cuda.stream(stream):
            for _ in range(5):
                got[i].append(step(*cases[i]))
        stream.synchronize()

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(cases))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    for w, runs in zip(want, got):
        assert len(runs) == 5
        for run in runs:
            assert all(torch.equal(a, b) for a, b in zip(run, w))
