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
ROOM = 1 << 12


class Host:
    """What the calls see instead of the library and the GPU."""

    def __init__(self):
        self.stream = 1 << 44
        self.memory = []  # (address, bytes, reference) of everything allocated, in order
        self.calls = []   # (entry, arguments)
        self.entered = []  # called at the next entries, one each

    def watch(self, t):
        from torch.multiprocessing.reductions import StorageWeakRef

        room = t.untyped_storage()
        if room.nbytes():
            self.memory.append((room.data_ptr(), room.nbytes(), StorageWeakRef(room)))
        return t

    def at(self, address):
        """The last allocation that has this address, or None."""
        for lo, size, ref in reversed(self.memory):
            if lo <= address < lo + size:
                return ref
        return None

    def entry(self, name, args):
        if self.entered:
            self.entered.pop(0)()
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
    empty = torch.empty
    monkeypatch.setattr(_lib, "library", lambda: h)
    monkeypatch.setattr(torch, "empty", lambda *a, **k: h.watch(empty(*a, **k)))
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
