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


def numbers(args):
    return list(args[8]) if args[7] else []


@pytest.mark.parametrize("rows", [
    ([1.0, 2.0, 3.0], [4.0, 5.0, 6.0]),                      # a tuple of lists
    [[1.0, 2.0, 3.0], (4.0, 5.0, 6.0)],
    ((1, 2, 3), torch.tensor([4.0, 5.0, 6.0])),
    torch.tensor([[1.0, 2.0, 3.0], [4.0, 5.0, 6.0]]),
    ((torch.tensor(1.0), torch.tensor(2.0), 3), (4, 5, torch.tensor(6.0))),
    iter([iter([1.0, 2.0, 3.0]), iter([4.0, 5.0, 6.0])]),
])
def test_a_row_of_coefficients_for_each_step(calls, rows):
    tg.orthogonalize(torch.randn(4, 6), steps=2, coefficients=rows)
    assert numbers(calls[0]) == [1, 2, 3, 4, 5, 6]


@pytest.mark.parametrize("row", [(1, 2.0, 3), [1.0, 2.0, 3.0], torch.tensor([1.0, 2.0, 3.0]),
                                 (torch.tensor(1.0), torch.tensor(2.0), torch.tensor(3.0)), iter([1.0, 2.0, 3.0])])
def test_coefficients_for_all_steps(calls, row):
    tg.orthogonalize(torch.randn(4, 6), steps=2, coefficients=row)
    assert numbers(calls[0]) == [1, 2, 3, 1, 2, 3]


def test_coefficients_are_what_they_are_at_the_call(calls):
    t = torch.tensor(1.0)
    for value in (1.0, 7.0):
        t.fill_(value)
        tg.orthogonalize(torch.randn(4, 6), steps=1, coefficients=(t, 2.0, 3.0))
    assert [numbers(c) for c in calls] == [[1, 2, 3], [7, 2, 3]]


@pytest.mark.parametrize("bad", [(), (1.0, 2.0), (1.0, 2.0, 3.0, 4.0), ((1.0, 2.0, 3.0),), ([1.0, 2.0], [3.0, 4.0]),
                                 ((1.0, 2.0, 3.0), 4.0), ((1.0, 2.0, 3.0), (1.0, 2.0, 3.0), (1.0, 2.0, 3.0))])
def test_other_coefficients_are_refused(calls, bad):
    with pytest.raises(ValueError, match="coefficients must be three numbers"):
        tg.orthogonalize(torch.randn(4, 6), steps=2, coefficients=bad)
    assert not calls


def test_what_is_no_number_is_refused(calls):
    for bad in ("123", ("a", 2.0, 3.0), (None, 2.0, 3.0)):
        with pytest.raises((TypeError, ValueError)):
            tg.orthogonalize(torch.randn(4, 6), coefficients=bad)
    assert not calls
