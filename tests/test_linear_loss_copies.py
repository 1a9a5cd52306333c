"""What the losses' differentiable calls keep for the backward pass besides the
results: a copy of targets that are not contiguous (tensors of the host stand
in for the device's, as in test_linear_loss_binding)."""

import pytest

torch = pytest.importorskip("torch")

import tiled_gemm_tgemm_amd as tg  # noqa: E402
from test_linear_loss_binding import Y, head, host  # noqa: E402,F401

TARGET = 8  # where the calls' arguments have it


@pytest.mark.parametrize("strided", [False, True])
def test_a_copy_of_the_targets_is_held_for_another_stream(host, strided, monkeypatch):  # noqa: F811
    recorded = []
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: recorded.append((t.data_ptr(), s.cuda_stream)), raising=False)
    contiguous = torch.Tensor.contiguous
    monkeypatch.setattr(torch.Tensor, "contiguous", lambda t: t if t.is_contiguous() else host.copy(contiguous(t)))
    X, W = (t.requires_grad_() for t in head())
    target = Y.repeat_interleave(2)[::2] if strided else Y
    loss = tg.linear_cross_entropy(X, W, target, keep_logits=False)
    copied = host.calls[-1][1][TARGET]
    assert (copied == target.data_ptr()) != strided
    host.stream = 1 << 46
    loss.grad_fn.apply(torch.ones(()))
    name, args = host.calls[-1]
    assert name.endswith("backward") and args[TARGET] == copied
    # lse, the summary and the copy, and nothing of the caller's
    assert len(recorded) == 2 + strided and {s for _, s in recorded} == {host.stream}
    assert (copied in [at for at, _ in recorded]) == strided
