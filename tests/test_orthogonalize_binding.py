"""The torch call of the Newton-Schulz operator without a GPU: tensors of the host
stand in for the device's, and the library's entry points note what they are
handed."""

import contextlib
import types

import pytest

torch = pytest.importorskip("torch")

import tiled_gemm_tgemm_amd as tg  # noqa: E402
from tiled_gemm_tgemm_amd import _lib  # noqa: E402


@pytest.fixture
def calls(monkeypatch):
    seen = []
    library = types.SimpleNamespace(tgemm_orthogonalize=lambda *args: seen.append(args) or 0,
                                    tgemm_orthogonalize_workspace_size=lambda *args: 64)
    monkeypatch.setattr(_lib, "library", lambda: library)
    monkeypatch.setattr(torch.Tensor, "is_cuda", property(lambda t: True), raising=False)
    monkeypatch.setattr(torch.cuda, "device", lambda device: contextlib.nullcontext())
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: types.SimpleNamespace(cuda_stream=1 << 44))
    return seen


def test_a_gradient_is_not_lost(calls):
    G = torch.randn(4, 6, requires_grad=True)
    out = tg.orthogonalize(G)
    assert out.requires_grad and out.shape == G.shape and len(calls) == 1 and calls[0][4] == G.data_ptr()
    with pytest.raises(NotImplementedError, match="orthogonalize"):
        out.sum().backward()
    with pytest.raises(NotImplementedError, match="orthogonalize"):
        torch.autograd.grad((G * 2 + tg.orthogonalize(G * 3)).sum(), G)
    assert G.grad is None
    # nothing may be written into a tensor that a backward pass is to come through
    with pytest.raises(RuntimeError, match="out"):
        tg.orthogonalize(G, out=torch.empty(4, 6))
    # as an optimiser calls it
    with torch.no_grad():
        room = torch.empty(4, 6)
        assert not tg.orthogonalize(G).requires_grad and tg.orthogonalize(G, out=room) is room
    assert not tg.orthogonalize(G.detach()).requires_grad


def test_a_forward_mode_derivative_is_not_dropped(calls):
    from torch.autograd import forward_ad

    G = torch.randn(4, 6)
    with forward_ad.dual_level():
        assert tg.orthogonalize(G).shape == (4, 6)
        for t in (G, G.clone().requires_grad_()):
            with pytest.raises(NotImplementedError):
                tg.orthogonalize(forward_ad.make_dual(t, torch.ones(4, 6)))
    assert len(calls) == 1
