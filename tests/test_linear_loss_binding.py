"""The loss operators' torch calls without a GPU: tensors of the host stand in
for the device's, and the library's entry points are replaced by ones that
look at what they are handed: the stream, and whether the memory behind every
address is still somebody's."""

import types

import pytest

torch = pytest.importorskip("torch")

import tiled_gemm_tgemm_amd as tg  # noqa: E402
from tiled_gemm_tgemm_amd import _lib  # noqa: E402

T, V, D, K = 6, 11, 8, 3
REAL_EMPTY = torch.empty
ROOM = 1 << 12


class Host:
    """What the calls see instead of the library and the GPU."""

    def __init__(self):
        self.stream = 1 << 44
        self.memory = []  # (memory, address, reference to who has it) of everything allocated
        self.calls = []   # (entry, arguments)
        self.allocating = []  # called at the next allocations, one each

    def empty(self, shape, dtype=torch.float32, device=None):
        """As torch.empty."""
        if self.allocating:
            self.allocating.pop(0)()
        return self.room(shape, dtype)

    def room(self, shape, dtype):
        from torch.multiprocessing.reductions import StorageWeakRef

        shape = torch.Size([shape] if isinstance(shape, int) else shape)
        t = REAL_EMPTY((0,), dtype=dtype)
        if shape.numel():
            memory = bytearray(shape.numel() * dtype.itemsize + 64)  # stays: no address comes twice
            room = torch.frombuffer(memory, dtype=dtype, count=shape.numel()).untyped_storage()
            self.memory.append((memory, room.data_ptr(), StorageWeakRef(room)))
            t.set_(room, 0, shape)
        return t if t.shape == shape else t.view(shape)

    def copy(self, t):
        return self.room(t.shape, t.dtype).copy_(t.detach())

    def at(self, address):
        """Who has, or had, this address, or None."""
        for memory, lo, ref in self.memory:
            if lo <= address < lo + len(memory):
                return ref
        return None

    def entry(self, name, args):
        for a in args:
            ref = self.at(a) if isinstance(a, int) else None
            assert ref is None or not ref.expired(), f"{name} is handed memory that was released"
        assert self.at(args[-3]) is not None, f"{name}: the workspace is not a known one"
        self.calls.append((name, args))
        return 0

    def __getattr__(self, name):
        if name == "tgemm_linear_loss_workspace_size":
            return lambda *args: ROOM
        if name.startswith("tgemm_linear_"):
            return lambda *args: self.entry(name, args)
        raise AttributeError(name)


@pytest.fixture
def host(monkeypatch):
    h = Host()
    monkeypatch.setattr(_lib, "library", lambda: h)
    monkeypatch.setattr(torch, "empty", h.empty)
    monkeypatch.setattr(torch.Tensor, "is_cuda", property(lambda t: True), raising=False)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: None)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: types.SimpleNamespace(cuda_stream=h.stream))
    monkeypatch.setattr(tg, "_hold_for_stream", lambda stream, device, *tensors: None)
    return h


def head():
    g = torch.Generator().manual_seed(1)
    return torch.randn(T, D, generator=g), torch.randn(V, D, generator=g)


Y = torch.arange(T) % V
IDS = (torch.arange(T * K) % V).view(T, K)
TOP = torch.arange(T * K, dtype=torch.float32).view(T, K)


def losses():
    """The differentiable calls on X and W."""
    return {"ce": lambda X, W, **k: tg.linear_cross_entropy(X, W, Y, **k),
            "kd": lambda X, W, **k: tg.linear_distillation(X, W, IDS, TOP, **k)}


@pytest.mark.parametrize("stream", [None, 1 << 45])
def test_memory_is_held_until_the_kernels_are_queued(host, stream):
    X, W = head()
    loss, lse = tg.linear_cross_entropy_forward(X, W, Y, stream=stream)
    tg.linear_cross_entropy_backward(loss, X, W, Y, lse, stream=stream)
    # a target that the call copies
    tg.linear_cross_entropy_forward(X, W, Y.repeat_interleave(2)[::2], stream=stream)
    loss, lse, student = tg.linear_distillation_forward(X, W, IDS, TOP, stream=stream)
    tg.linear_distillation_backward(loss, X, W, IDS, TOP, lse, student, stream=stream)
    assert len(host.calls) == 5
    assert all(args[-1] == (host.stream if stream is None else stream) for _, args in host.calls)


@pytest.mark.parametrize("op", ["ce", "kd"])
@pytest.mark.parametrize("keep", [False, True])
def test_differentiable_calls_hold_their_memory_until_then(host, op, keep):
    X, W = (t.requires_grad_() for t in head())
    loss = losses()[op](X, W, keep_logits=keep)
    torch.autograd.grad(loss, (X, W))
    assert [name for name, _ in host.calls] == [f"tgemm_linear_{op}_forward", f"tgemm_linear_{op}_backward"]


def test_a_workspace_is_released_after_the_call(host):
    X, W = (t.requires_grad_() for t in head())
    loss = losses()["ce"](X, W)
    torch.autograd.grad(loss, (X, W), retain_graph=True)
    assert all(host.at(args[-3]).expired() for _, args in host.calls)


@pytest.mark.parametrize("op", ["ce", "kd"])
@pytest.mark.parametrize("turn", [0, 1, 2])
def test_backward_passes_through_one_node_do_not_meet(host, op, turn):
    """Another pass comes in where the first one allocates its `turn`-th tensor, as another thread's may, and each has
    saved tensors of its own, as hooks make them."""
    X, W = (t.requires_grad_() for t in head())
    with torch.autograd.graph.saved_tensors_hooks(lambda t: t, lambda t: host.copy(t)):
        loss = losses()[op](X, W)
    host.allocating = [lambda: None] * turn + [lambda: torch.autograd.grad(loss, (X, W), retain_graph=True)]
    torch.autograd.grad(loss, (X, W), retain_graph=True)
    assert [name for name, _ in host.calls] == [f"tgemm_linear_{op}_forward"] + 2 * [f"tgemm_linear_{op}_backward"]
    inner, outer = host.calls[1][1], host.calls[2][1]
    assert inner[4] != outer[4] and inner[6] != outer[6] and inner[-3] != outer[-3]


def test_a_saved_tensor_that_changed_its_size_is_refused(host):
    X, W = (t.requires_grad_() for t in head())
    for change in (lambda t: t[:2], lambda t: t.double()):
        with torch.autograd.graph.saved_tensors_hooks(lambda t: t, lambda t: change(t.detach()) if t.dim() == 2 else t):
            loss = losses()["ce"](X, W, keep_logits=False)
        with pytest.raises((TypeError, ValueError)):
            torch.autograd.grad(loss, (X, W))
    assert all(name.endswith("forward") for name, _ in host.calls)


@pytest.mark.parametrize("op", ["ce", "kd"])
@pytest.mark.parametrize("keep", [False, True])
def test_a_node_called_under_another_stream_runs_there(host, op, keep, monkeypatch):
    recorded = []
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: recorded.append((t.data_ptr(), s.cuda_stream)),
                        raising=False)
    X, W = (t.requires_grad_() for t in head())
    loss = losses()[op](X, W, keep_logits=keep)
    first = host.stream
    torch.autograd.grad(loss, (X, W), retain_graph=True)
    assert host.calls[-1][1][-1] == first and not recorded
    host.stream = 1 << 46
    loss.grad_fn.apply(torch.ones(()))
    name, args = host.calls[-1]
    assert name.endswith("backward") and args[-1] == host.stream
    # what the forward pass allocated on its own stream is known to be in use on this one
    assert len(recorded) == 2 + keep + (op == "kd") and {s for _, s in recorded} == {host.stream}
    torch.autograd.grad(loss, (X, W))
    assert len(host.calls) == 4


@pytest.mark.parametrize("op", ["ce", "kd"])
@pytest.mark.parametrize("reduction,size", [("mean", 12), ("sum", 12), ("none", 4 * T)])
def test_a_loss_that_is_kept_holds_no_more_than_itself(host, op, reduction, size):
    X, W = (t.requires_grad_() for t in head())
    loss = losses()[op](X, W, reduction=reduction)
    assert loss.shape == ((T,) if reduction == "none" else ()) and not loss._is_view()
    assert loss.detach().untyped_storage().nbytes() <= size
    torch.autograd.grad(loss.sum(), (X, W))
    forward, backward = (args for _, args in host.calls)
    # lse is the forward call's, and only a mean's gradient has its third number as a factor
    assert backward[15 if op == "kd" else 10] == forward[16 if op == "kd" else 11]
    assert backward[21 if op == "kd" else 15] == (forward[-4] + 8 if reduction == "mean" else 0)


@pytest.mark.parametrize("op", ["ce", "kd"])
@pytest.mark.parametrize("kind,other", [(torch.bfloat16, torch.float32), (torch.float32, torch.float16),
                                        (torch.float16, torch.bfloat16)])
def test_operands_of_two_types_are_refused(host, op, kind, other):
    X, W = head()
    with torch.autocast("cpu", dtype=torch.bfloat16):
        for autograd in (False, True):
            x, w = X.to(kind).requires_grad_(autograd), W.to(other).requires_grad_(autograd)
            with pytest.raises(TypeError, match=f"W must be {kind}"):
                losses()[op](x, w)
    with pytest.raises(TypeError, match=f"W must be {kind}"):
        tg.linear_cross_entropy_forward(X.to(kind), W.to(other), Y)
    assert not host.calls
    w = W.to(other).requires_grad_()
    loss = losses()[op](X.to(kind), w.to(kind))  # as the module says
    (dW,) = torch.autograd.grad(loss, (w,))
    assert dW.dtype == other and len(host.calls) == 2


@pytest.mark.parametrize("name", ["ce_forward", "ce_backward", "kd_forward", "kd_backward"])
def test_arguments_reach_their_place_in_the_c_call(name, monkeypatch):
    """Each by its name in the header; those that come last here, and only those, stand elsewhere there."""
    import inspect
    import os
    import re

    with open(os.path.join(os.path.dirname(os.path.dirname(__file__)), "include", "tgemm.h")) as f:
        declared = re.search(rf"tgemm_linear_{name}\((.*?)\);", f.read(), re.S).group(1)
    order = [re.search(r"(\w+)$", p.strip()).group(1) for p in declared.split(",")]
    seen = []
    monkeypatch.setattr(_lib, "library", lambda: types.SimpleNamespace(
        **{f"tgemm_linear_{name}": lambda *args: seen.append(args) or 0}))
    call = getattr(tg, f"tgemm_linear_{name}")
    here = list(inspect.signature(call).parameters)
    call(**{p: f"<{p}>" for p in here})
    assert seen == [tuple(f"<{p}>" for p in order)]
    assert here[-2:] == ["logits", "ldz"] and here[:-2] == [p for p in order if p not in ("logits", "ldz")]


@pytest.mark.parametrize("op", ["ce", "kd"])
@pytest.mark.parametrize("reduction", ["mean", "sum", "none"])
def test_without_autograd_nothing_is_kept(host, op, reduction):
    X, W = (t.requires_grad_() for t in head())
    for without in (torch.no_grad, torch.inference_mode):
        with without():
            loss = losses()[op](X, W, reduction=reduction, keep_logits=True)
            loss += 1.0
        assert not loss.requires_grad and loss.shape == ((T,) if reduction == "none" else ())
    assert all(args[18 if op == "kd" else 12] == 0 for _, args in host.calls)
    del loss
    assert all(ref.expired() for _, _, ref in host.memory)
