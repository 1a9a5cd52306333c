"""The adapters' torch calls without a GPU, as test_linear_loss_binding has the
losses': tensors of the host stand in for the device's, and the library's entry
points are replaced by ones that look at what they are handed."""

import types

import pytest

torch = pytest.importorskip("torch")

import tiled_gemm_tgemm_amd as tg  # noqa: E402
from test_linear_loss_binding import Host  # noqa: E402
from tiled_gemm_tgemm_amd import _lib  # noqa: E402

T, N, D, L, R = 6, 11, 8, 3, 2
IDS, HIDDEN = 16, 20  # where a forward call's arguments have them


class Library(Host):
    def __getattr__(self, name):
        if name == "tgemm_linear_adapters_workspace_size":
            return lambda *args: 1 << 12
        return super().__getattr__(name)


@pytest.fixture
def host(monkeypatch):
    h = Library()
    contiguous = torch.Tensor.contiguous
    monkeypatch.setattr(_lib, "library", lambda: h)
    monkeypatch.setattr(torch, "empty", h.empty)
    monkeypatch.setattr(torch.Tensor, "contiguous", lambda t: t if t.is_contiguous() else h.copy(contiguous(t)))
    monkeypatch.setattr(torch.Tensor, "is_cuda", property(lambda t: True), raising=False)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: None)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: types.SimpleNamespace(cuda_stream=h.stream))
    monkeypatch.setattr(tg, "_hold_for_stream", lambda stream, device, *tensors: None)
    return h


def layer():
    g = torch.Generator().manual_seed(1)
    n = lambda *s: torch.randn(s, generator=g)
    return n(T, D), n(N, D), n(L, R, D), n(L, N, R), torch.arange(T) % (L + 1) - 1


@pytest.mark.parametrize("strided", [False, True])
def test_a_node_called_under_another_stream_runs_there(host, strided, monkeypatch):
    recorded = []
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: recorded.append((t.data_ptr(), s.cuda_stream)), raising=False)
    X, W, A, B, ids = layer()
    if strided:
        ids = ids.repeat_interleave(2)[::2]
    Y = tg.linear_adapters(X, W, A.requires_grad_(), B.requires_grad_(), ids)
    forward = host.calls[-1][1]
    assert (forward[IDS] == ids.data_ptr()) != strided and forward[HIDDEN]
    first = host.stream
    torch.autograd.grad(Y, (A, B), torch.ones(T, N), retain_graph=True)
    assert host.calls[-1][1][-1] == first and not recorded
    host.stream = 1 << 46
    Y.grad_fn.apply(torch.ones(T, N))
    name, args = host.calls[-1]
    assert name.endswith("backward") and args[-1] == host.stream and args[IDS] == forward[IDS]
    # what the forward pass allocated on its own stream is known to be in use on this one, and nothing of the caller's
    own = [forward[HIDDEN]] + [forward[IDS]] * strided
    assert sorted(recorded) == sorted((at, host.stream) for at in own)


@pytest.mark.parametrize("which", range(5))
@pytest.mark.parametrize("others", [False, True])
def test_a_forward_mode_derivative_is_not_dropped(host, which, others):
    """Of any of the arguments, where no backward pass comes and where one does."""
    from torch.autograd import forward_ad

    X, W, A, B, ids = layer()
    if others:
        X.requires_grad_()
    args = [X, W, A, B, torch.ones(L)]
    with forward_ad.dual_level():
        assert tg.linear_adapters(X, W, A, B, ids).shape == (T, N)  # none of them has one
        args[which] = forward_ad.make_dual(args[which], torch.ones_like(args[which]))
        calls = len(host.calls)
        for autograd in (torch.enable_grad, torch.no_grad):
            with autograd(), pytest.raises(NotImplementedError):
                tg.linear_adapters(*args[:4], ids, scales=args[4])
        assert len(host.calls) == calls
    with pytest.raises((NotImplementedError, RuntimeError)):
        torch.func.jvp(lambda t: tg.linear_adapters(*args[:which], t, *args[which + 1:4], ids, scales=None) if which < 4
                       else tg.linear_adapters(*args[:4], ids, scales=t), (torch.ones_like(args[which]),), (torch.ones_like(args[which]),))


@pytest.mark.parametrize("others", [False, True])
def test_scales_that_require_a_gradient_are_refused(host, others):
    X, W, A, B, ids = layer()
    if others:
        A.requires_grad_()
    scales = torch.ones(L, requires_grad=True)
    with pytest.raises(NotImplementedError, match="scales"):
        tg.linear_adapters(X, W, A, B, ids, scales=scales)
    assert not host.calls
    assert tg.linear_adapters(X, W, A, B, ids, scales=scales.detach()).requires_grad == others
    with torch.no_grad():
        assert not tg.linear_adapters(X, W, A, B, ids, scales=scales).requires_grad


@pytest.mark.parametrize("change", [lambda t: t[:2], lambda t: t.double(), lambda t: t.repeat_interleave(2)[::2]])
def test_saved_ids_and_scales_that_changed_are_refused(host, change):
    """As hooks may hand them back: the kernels would read past their ends, or other values."""
    X, W, A, B, ids = layer()
    for which in (torch.int64, torch.float32):
        with torch.autograd.graph.saved_tensors_hooks(lambda t: t, lambda t: change(t.detach()) if t.dim() == 1 and t.dtype == which else t):
            Y = tg.linear_adapters(X, W, A.requires_grad_(), B.requires_grad_(), ids, scales=torch.ones(L))
        with pytest.raises((TypeError, ValueError)):
            torch.autograd.grad(Y, (A, B), torch.ones(T, N))
    assert all(name.endswith("forward") for name, _ in host.calls)
