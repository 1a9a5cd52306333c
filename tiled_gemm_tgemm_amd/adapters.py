"""A projection X·Wᵀ with low-rank adapters of many requests beside it, for torch tensors.

X (T×D) holds a row a token, W (N×D) the shared weight, A (L×r×D) and B (L×N×r)
the adapters, ids (T, int64) each token's adapter, -1 for none, and scales (L,
float32) their factors:

    y_t = x_t·Wᵀ + scales_i·(x_t·A_iᵀ)·B_iᵀ,  i = ids_t

X, W, A and B have one type, float32, bfloat16 or float16, which the result and
the gradients have too; others, and mixed ones, raise TypeError (torch.autocast
does not reach these calls).

* ``linear_adapters`` is differentiable in X, W, A and B;
* ``linear_adapters_forward`` and ``linear_adapters_backward`` are the same calls
  without torch's autograd, for programs that keep their own buffers or capture
  them into a graph.

All are queued on `stream` (default: torch's current stream of X's device) and
return without waiting.  include/tgemm.h states the arithmetic.
"""

from __future__ import annotations

import functools

from . import _lib
from ._lib import TgemmError
from .linear_loss import _floats, _ids, _no_tangents, _ptr, _rows, _types


def _stacked(t, name, shape, device, dtype):
    """(leading dimension, stride) of a stack of row-major matrices."""
    import torch

    if not isinstance(t, torch.Tensor) or t.dim() != 3 or t.dtype != dtype:
        raise TypeError(f"{name} must be a 3-D {dtype} torch tensor")
    if t.device != device:
        raise TypeError(f"{name} must live on {device}")
    if tuple(t.shape) != shape:
        raise ValueError(f"{name} must be {'x'.join(map(str, shape))}")
    count, rows, cols = shape
    if t.is_contiguous():
        return cols, rows * cols
    apart, down, across = t.stride()
    if cols > 1 and across != 1 or rows > 1 and down < cols:
        raise ValueError(f"{name} must hold row-major matrices")
    return (down if rows > 1 else cols), (apart if count > 1 else rows * cols)


class _Call:
    """The arguments shared by the calls, and what they allocate."""

    def __init__(self, X, W, A, B, ids, scales, stream):
        import torch

        ldx = _rows(X, "X")
        self.device, self.dtype = X.device, X.dtype
        ldw = _rows(W, "W", device=self.device, like=self.dtype)
        (self.T, self.D), (self.N, inner) = X.shape, W.shape
        if inner != self.D:
            raise ValueError(f"inner sizes differ: X is {tuple(X.shape)}, W is {tuple(W.shape)}")
        if self.N < 1 or self.D < 1:
            raise ValueError("W must have a row and a column")
        if not isinstance(A, torch.Tensor) or A.dim() != 3:
            raise TypeError(f"A must be a 3-D {self.dtype} torch tensor")
        self.L, self.r = A.shape[:2]
        if self.L < 1 or self.r < 1:
            raise ValueError("there must be an adapter, of a rank")
        lda, stride_a = _stacked(A, "A", (self.L, self.r, self.D), self.device, self.dtype)
        ldb, stride_b = _stacked(B, "B", (self.L, self.N, self.r), self.device, self.dtype)
        self.made = []
        ids = _ids(ids, "ids", (self.T,), self.device)
        if not ids.is_contiguous():
            ids = ids.contiguous()
            self.made.append(ids)
        if scales is not None:
            _floats(scales, "scales", (self.L,), self.device)
        self.elsewhere = stream is not None
        self.stream = stream if self.elsewhere else torch.cuda.current_stream(self.device).cuda_stream
        self.head = (_types()[self.dtype], self.T, self.N, self.D, X.data_ptr(), ldx, W.data_ptr(), ldw)
        self.adapters = (self.L, self.r, A.data_ptr(), lda, stride_a, B.data_ptr(), ldb, stride_b, ids.data_ptr(),
                         _ptr(scales))

    def again(self, X, W, A, B, ids, scales, *kept):
        """The call of a backward pass: the same tensors, wherever and however they are stored by now, on the stream
        that is torch's current one (its engine makes that the forward pass's; a node that is called by hand runs where
        its caller is).  It is the pass's own: others may go through the same node meanwhile.  kept: what the forward
        pass allocated."""
        import torch

        c = _Call.__new__(_Call)
        c.__dict__.update(self.__dict__)
        current = torch.cuda.current_stream(c.device)
        if current.cuda_stream != c.stream:
            c.stream = current.cuda_stream
            for t in kept:
                if t is not None:
                    t.record_stream(current)
        if not _ids(ids, "ids", (c.T,), c.device).is_contiguous():
            raise ValueError("ids must be contiguous")
        if scales is not None:
            _floats(scales, "scales", (c.L,), c.device)
        ldx = _rows(X, "X", (c.T, c.D), c.device, c.dtype)
        c.head = (*c.head[:4], X.data_ptr(), ldx, W.data_ptr(), _rows(W, "W", (c.N, c.D), c.device, c.dtype))
        c.adapters = (c.L, c.r, A.data_ptr(), *_stacked(A, "A", (c.L, c.r, c.D), c.device, c.dtype), B.data_ptr(),
                      *_stacked(B, "B", (c.L, c.N, c.r), c.device, c.dtype), ids.data_ptr(), _ptr(scales))
        c.made = []
        return c

    def new(self, shape, dtype=None):
        import torch

        t = torch.empty(shape, dtype=dtype or self.dtype, device=self.device)
        self.made.append(t)
        return t

    def matrix(self, t, name, shape):
        """A result of rows: the tensor, its address and leading dimension."""
        if t is None:
            t = self.new(shape)
            return t, (t.data_ptr(), shape[1])
        ld = _rows(t, name, shape, self.device, self.dtype)
        return t, (t.data_ptr(), ld)

    def stack(self, t, name, shape):
        if t is None:
            t = self.new(shape)
            return t, (t.data_ptr(), shape[2], shape[1] * shape[2])
        return t, (t.data_ptr(), *_stacked(t, name, shape, self.device, self.dtype))

    def hidden(self, t):
        if t is None:
            return 0
        return _floats(t, "hidden", (self.T, self.r), self.device).data_ptr()

    def room(self, workspace, *gradients):
        import torch

        if workspace is None:
            need = _lib.library().tgemm_linear_adapters_workspace_size(*self.head, self.L, self.r, *(gradients or (0, 0, 0)))
            workspace = torch.empty(need or 1, dtype=torch.uint8, device=self.device)
            self.made.append(workspace)
            return workspace.data_ptr(), need or 1
        if not isinstance(workspace, torch.Tensor) or workspace.dtype != torch.uint8:
            raise TypeError("workspace must be a CUDA uint8 tensor")
        if workspace.device != self.device or not workspace.is_contiguous():
            raise TypeError(f"workspace must be contiguous and live on {self.device}")
        return workspace.data_ptr(), workspace.numel()

    def queue(self, entry, *args):
        import torch

        if self.elsewhere:
            from . import _hold_for_stream

            _hold_for_stream(self.stream, self.device, *self.made)
        entry_point = getattr(_lib.library(), entry)
        try:
            if torch.cuda.current_device() == self.device.index:
                st = entry_point(*self.head, *self.adapters, *args, self.stream)
            else:
                with torch.cuda.device(self.device):
                    st = entry_point(*self.head, *self.adapters, *args, self.stream)
        finally:
            # only now: what is released after the launches is handed out again behind them
            self.made.clear()
        if st != _lib.TGEMM_SUCCESS:
            raise TgemmError(st, entry)


def linear_adapters_forward(X, W, A, B, ids, *, scales=None, out=None, hidden=None, workspace=None, stream=None):
    """Y (tgemm_linear_adapters_forward); ids outside [-1, L) give rows of NaN.  out: a row-major tensor to write to;
    hidden: a float32 tensor of T×r to leave x_t·A_iᵀ in, for the backward call (not kept if omitted); workspace: a
    CUDA uint8 tensor of at least tgemm_linear_adapters_workspace_size bytes (allocated if omitted; two calls in flight
    at once need two)."""
    c = _Call(X, W, A, B, ids, scales, stream)
    Y, out = c.matrix(out, "out", (c.T, c.N))
    c.queue("tgemm_linear_adapters_forward", *out, c.hidden(hidden), *c.room(workspace))
    return Y


def _backward(c, dY, hidden, results, need, workspace):
    """results: dX, dW, dA, dB to write to, or None to have them allocated."""
    lddy = _rows(dY, "dY", (c.T, c.N), c.device, c.dtype)
    shapes = ((c.T, c.D), (c.N, c.D), (c.L, c.r, c.D), (c.L, c.N, c.r))
    out, args = [], []
    for t, name, shape, wanted in zip(results, ("dX", "dW", "dA", "dB"), shapes, need):
        if wanted:
            t, at = (c.matrix if len(shape) == 2 else c.stack)(t, name, shape)
        else:
            t, at = None, (0, shape[1]) if len(shape) == 2 else (0, shape[2], shape[1] * shape[2])
        out.append(t)
        args += at
    bits = sum(1 << n for n in range(4) if need[n])
    if bits:
        c.queue("tgemm_linear_adapters_backward", c.hidden(hidden), dY.data_ptr(), lddy, *args,
                *c.room(workspace, dY.data_ptr(), lddy, bits))
    return tuple(out)


def linear_adapters_backward(dY, X, W, A, B, ids, hidden=None, *, scales=None, dX=None, dW=None, dA=None, dB=None,
                             need=(True, True, True, True), workspace=None, stream=None):
    """(dX, dW, dA, dB) for the gradient dY of the result (tgemm_linear_adapters_backward); hidden as
    linear_adapters_forward left it (formed again without).  dX ... dB: tensors to write to; need: which of the four
    are computed (None is returned for the others).  An adapter without tokens gets zeros."""
    c = _Call(X, W, A, B, ids, scales, stream)
    return _backward(c, dY, hidden, (dX, dW, dA, dB), need, workspace)


@functools.lru_cache(maxsize=None)
def _function():
    """The differentiable form.  One backward pass per forward pass through it; there is no second derivative."""
    import torch
    from torch.autograd.function import once_differentiable

    class Adapters(torch.autograd.Function):
        @staticmethod
        def forward(ctx, X, W, A, B, ids, scales):
            # (a copy that the call makes of ids stands in for it in the backward pass)
            c = _Call(X, W, A, B, ids, scales, None)
            ctx.copied = bool(c.made)
            if ctx.copied:
                ids = c.made[0]
            Y = torch.empty((c.T, c.N), dtype=c.dtype, device=c.device)
            hidden = torch.empty((c.T, c.r), dtype=torch.float32, device=c.device) if ctx.needs_input_grad[3] else None
            c.queue("tgemm_linear_adapters_forward", Y.data_ptr(), c.N, _ptr(hidden), *c.room(None))
            ctx.save_for_backward(X, W, A, B, ids, scales, hidden)
            ctx.call = c
            return Y

        @staticmethod
        @once_differentiable
        def backward(ctx, dY):
            X, W, A, B, ids, scales, hidden = ctx.saved_tensors
            c = ctx.call.again(X, W, A, B, ids, scales, hidden, ids if ctx.copied else None)
            if not dY.is_contiguous():
                dY = dY.contiguous()
            return (*_backward(c, dY, hidden, (None,) * 4, ctx.needs_input_grad[:4], None), None, None)

    return Adapters


def linear_adapters(X, W, A, B, ids, *, scales=None):
    """The projection X·Wᵀ with each token's adapter beside it, differentiable in X, W, A and B (in those of them that
    require a gradient).  Without a gradient to compute it is linear_adapters_forward.  There is no gradient of scales
    and no forward-mode derivative: where autograd would want either, NotImplementedError is raised."""
    import torch

    _no_tangents("linear_adapters", X, W, A, B, scales)
    if torch.is_grad_enabled():
        if isinstance(scales, torch.Tensor) and scales.requires_grad:
            raise NotImplementedError("linear_adapters has no gradient of scales: pass scales.detach()")
        if any(isinstance(t, torch.Tensor) and t.requires_grad for t in (X, W, A, B)):
            return _function().apply(X, W, A, B, ids, scales)
    return linear_adapters_forward(X, W, A, B, ids, scales=scales)
