"""Losses on an output head's product X·Wᵀ, for torch tensors, without the product.

X (T×D) holds the tokens' hidden states and W (V×D) the head's weight, both
float32, bfloat16 or float16 on one GPU, row-major with any leading dimension.
Both have the same type, and gradients have it too: float32 weights beside
16-bit states (torch.autocast does not reach these calls) raise TypeError;
`W.to(X.dtype)` there, or `X.to(W.dtype)`, is differentiable.

* ``linear_cross_entropy`` and ``linear_distillation`` are differentiable in X
  and W and reduce over the rows;
* ``..._forward`` gives the losses of the rows and what the backward pass
  needs, ``..._backward`` the gradients of sum_t grad_loss_t·loss_t: the same
  calls without torch's autograd, for programs that keep their own buffers or
  capture them into a graph.

All are queued on `stream` (default: torch's current stream of X's device) and
return without waiting.  include/tgemm.h states the arithmetic.
"""

from __future__ import annotations

import functools

from . import _lib
from ._lib import TgemmError

REDUCTIONS = ("mean", "sum", "none")

# Unless told otherwise the differentiable calls form the logits again in the backward pass, and hold them (float32)
# only where all of them take no more than the 256 MiB that a piece of their gradient is meant to take, and that
# is faster.  Writing and reading them costs about as much as forming them again does at an inner size (a sixth of it
# for float32 operands, which take six products) that depends on where they stay meanwhile: (bytes, inner size), one
# line that both meet is enough.  A step with them held, of its time with them formed again (cross entropy bf16;
# distillation up to 0.03 more, float32 at a sixth of the inner size up to 0.12 less), at inner sizes of 64, 256, 512,
# 768, 1024 and 2048:
#     1 MiB (33×8192)       0.93  0.91  0.88  0.86  0.84  0.79
#     8 MiB (128×16384)     0.96  0.93  0.90  0.90  0.89  0.86
#    32 MiB (512×16384)     1.07  1.02  0.98  0.96  0.93  0.88
#    59 MiB (777×20011)     1.06  1.00  0.95  0.92  0.88  0.86
#    80 MiB (1024×20480)    1.13  1.04  0.98  0.94  0.91  0.89
#    98 MiB (512×50001)     1.14  1.07  1.01  0.99  0.94  0.87
#   128 MiB (2048×16384)    1.17  1.11  1.04  0.99  0.98  0.90
#   183 MiB (1500×32000)    1.42  1.26  1.17  1.06  0.99  0.90
#   250 MiB (2048×32000)    1.55  1.41  1.20  1.05  0.99  0.91
# Larger ones, for those who ask for it: 4096×32768 (512 MiB) with 2048 0.89, with 4096 0.83.
KEPT = ((4 << 20, 0), (96 << 20, 512), (256 << 20, 1024))


@functools.lru_cache(maxsize=None)
def _types():
    import torch

    return {torch.float32: _lib.TGEMM_F32, torch.bfloat16: _lib.TGEMM_BF16, torch.float16: _lib.TGEMM_F16}


def _dtype(t):
    return _types().get(t.dtype)


def _rows(t, name, shape=None, device=None, like=None):
    """The leading dimension of a row-major matrix of a supported type."""
    import torch

    if not isinstance(t, torch.Tensor) or t.dim() != 2 or t.dtype not in _types():
        raise TypeError(f"{name} must be a 2-D float32, bfloat16 or float16 torch tensor")
    if not t.is_cuda or (device is not None and t.device != device):
        raise TypeError(f"{name} must live on {'a GPU' if device is None else device}")
    if like is not None and t.dtype != like:
        raise TypeError(f"{name} must be {like}")
    if shape is not None and tuple(t.shape) != shape:
        raise ValueError(f"{name} must be {shape[0]}x{shape[1]}")
    rows, cols = t.shape
    if rows > 1 and t.is_contiguous():
        return cols or 1
    down, across = t.stride()
    if cols > 1 and rows > 0 and across != 1 or rows > 1 and down < cols:
        raise ValueError(f"{name} must be row-major")
    return max(down, cols, 1) if rows > 1 else max(cols, 1)


def _ids(t, name, shape, device):
    import torch

    if not isinstance(t, torch.Tensor) or t.dtype != torch.int64 or tuple(t.shape) != shape:
        raise TypeError(f"{name} must be an int64 torch tensor of {'x'.join(map(str, shape))}")
    if t.device != device:
        raise TypeError(f"{name} must live on {device}")
    return t


def _floats(t, name, shape, device):
    import torch

    if not isinstance(t, torch.Tensor) or t.dtype != torch.float32 or tuple(t.shape) != shape:
        raise TypeError(f"{name} must be a float32 torch tensor of {'x'.join(map(str, shape))}")
    if t.device != device or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous and live on {device}")
    return t


class _Call:
    """The arguments shared by the four calls, and what they allocate."""

    def __init__(self, X, W, stream):
        import torch

        ldx = _rows(X, "X")
        device, dtype = X.device, X.dtype
        ldw = _rows(W, "W", device=device, like=dtype)
        (T, D), (V, inner) = X.shape, W.shape
        if D != inner:
            raise ValueError(f"inner sizes differ: X is {tuple(X.shape)}, W is {tuple(W.shape)}")
        if V < 1 or D < 1:
            raise ValueError("W must have a row and a column")
        self.device, self.dtype, self.T, self.V, self.D = device, dtype, T, V, D
        self.head = (_types()[dtype], T, V, D, X.data_ptr(), ldx, W.data_ptr(), ldw)
        self.elsewhere = stream is not None
        self.stream = stream if self.elsewhere else torch.cuda.current_stream(device).cuda_stream
        self.made = []

    def again(self, X, W, *kept):
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
        ldx = _rows(X, "X", (c.T, c.D), c.device, c.dtype)
        c.head = (*c.head[:4], X.data_ptr(), ldx, W.data_ptr(), _rows(W, "W", (c.V, c.D), c.device, c.dtype))
        c.made = []
        return c

    def teacher(self, ids, logits, temperature):
        import torch

        if not isinstance(ids, torch.Tensor) or ids.dim() != 2 or ids.shape[0] != self.T or ids.shape[1] < 1:
            raise TypeError(f"teacher_ids must be an int64 torch tensor of {self.T} rows")
        self.K = ids.shape[1]
        ids = _ids(ids, "teacher_ids", (self.T, self.K), self.device)
        if self.T and (self.K > 1 and ids.stride(1) != 1 or self.T > 1 and ids.stride(0) < self.K):
            raise ValueError("teacher_ids must be row-major")
        ld = _rows(logits, "teacher_logits", (self.T, self.K), self.device)
        ld_ids = max(ids.stride(0), self.K) if self.T > 1 else self.K
        return (self.K, ids.data_ptr(), ld_ids, _dtype(logits), logits.data_ptr(), ld, float(temperature))

    def target(self, t):
        t = _ids(t, "target", (self.T,), self.device)
        if not t.is_contiguous():
            t = t.contiguous()
            self.made.append(t)
        return t

    def new(self, shape, dtype):
        import torch

        t = torch.empty(shape, dtype=dtype, device=self.device)
        self.made.append(t)
        return t

    def floats(self, t, name, shape):
        import torch

        return self.new(shape, torch.float32) if t is None else _floats(t, name, shape, self.device)

    def logits(self, t):
        """The address and leading dimension of the logits' room, or none."""
        import torch

        return (0, 0) if t is None else (t.data_ptr(), _rows(t, "logits", (self.T, self.V), self.device, torch.float32))

    def keep(self, keep):
        """Room for the logits between the two passes of a differentiable call; None to have them formed again."""
        import torch

        if keep is None:
            size, inner = 4 * self.T * self.V, self.D * (6 if self.dtype == torch.float32 else 1)
            keep = any(size <= room and inner >= least for room, least in KEPT)
        return torch.empty((self.T, self.V), dtype=torch.float32, device=self.device) if keep else None

    def gradient(self, t, name, shape):
        if t is None:
            return self.new(shape, self.dtype), shape[1]
        return t, _rows(t, name, shape, self.device, self.dtype)

    def room(self, workspace, k, backward):
        import torch

        if workspace is None:
            need = _lib.library().tgemm_linear_loss_workspace_size(*self.head, k, backward)
            workspace = torch.empty(need or 1, dtype=torch.uint8, device=self.device)
            self.made.append(workspace)
            return workspace.data_ptr(), need or 1
        if not isinstance(workspace, torch.Tensor) or workspace.dtype != torch.uint8:
            raise TypeError("workspace must be a CUDA uint8 tensor")
        elif workspace.device != self.device or not workspace.is_contiguous():
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
                st = entry_point(*self.head, *args, self.stream)
            else:
                with torch.cuda.device(self.device):
                    st = entry_point(*self.head, *args, self.stream)
        finally:
            # only now: what is released after the launches is handed out again behind them.  The call is kept for the
            # backward pass, its workspace not.
            self.made.clear()
        if st != _lib.TGEMM_SUCCESS:
            raise TgemmError(st, entry)

    def results(self, reduction):
        """What a differentiable forward pass writes to: the tensor that is returned, what is kept for the backward
        pass (lse first, and the summary, whose third number is the mean's factor), and the addresses of loss, lse and
        summary.  The returned tensor shares no memory with what grows with the rows."""
        import torch

        if reduction == "none":
            loss = torch.empty((self.T,), dtype=torch.float32, device=self.device)
            lse = torch.empty((self.T,), dtype=torch.float32, device=self.device)
            return loss, (lse, None), (loss.data_ptr(), lse.data_ptr(), 0)
        rows = torch.empty((2 * self.T,), dtype=torch.float32, device=self.device)
        summary = torch.empty((3,), dtype=torch.float32, device=self.device)
        # `data`: not a view of the summary to torch, so a caller may change it in place
        loss = summary.as_strided((), (), 1 if reduction == "mean" else 0).data
        at = rows.data_ptr()
        return loss, (rows, summary if reduction == "mean" else None), (at + 4 * self.T, at, summary.data_ptr())


def _ptr(t):
    return 0 if t is None else t.data_ptr()


def linear_cross_entropy_forward(X, W, target, *, ignore_index=-100, loss=None, lse=None, logits=None, workspace=None,
                                 stream=None):
    """(loss, lse) of the rows (tgemm_linear_ce_forward): lse_t = log sum_v exp(x_t·w_v), loss_t = lse_t - x_t·w_y
    with y = target_t (int64), 0 where y is ignore_index and NaN where y is outside the vocabulary otherwise.  loss
    and lse: float32 tensors of T to write to; logits: a row-major float32 tensor of T×V to leave the logits in, for
    the backward call (not written if omitted); workspace: a CUDA uint8 tensor of at least
    tgemm_linear_loss_workspace_size bytes (allocated if omitted; two calls in flight at once need two)."""
    c = _Call(X, W, stream)
    target = c.target(target)
    loss, lse = c.floats(loss, "loss", (c.T,)), c.floats(lse, "lse", (c.T,))
    c.queue("tgemm_linear_ce_forward", target.data_ptr(), int(ignore_index), loss.data_ptr(), lse.data_ptr(),
            *c.logits(logits), 0, *c.room(workspace, 0, 0))
    return loss, lse


def _gradients(c, dX, dW, need):
    dX, lddx = c.gradient(dX, "dX", (c.T, c.D)) if need[0] else (None, c.D)
    dW, lddw = c.gradient(dW, "dW", (c.V, c.D)) if need[1] else (None, c.D)
    return dX, dW, (_ptr(dX), lddx, _ptr(dW), lddw)


def _grad_loss(c, grad):
    """grad_loss: one value a row, or one for all."""
    import torch

    if not isinstance(grad, torch.Tensor) or grad.dtype != torch.float32 or tuple(grad.shape) not in ((c.T,), ()):
        raise TypeError(f"grad_loss must be a float32 torch tensor of {c.T}, or of no dimension")
    if grad.device != c.device:
        raise TypeError(f"grad_loss must live on {c.device}")
    return grad.data_ptr(), grad.stride(0) if grad.dim() and c.T > 1 else 0


def linear_cross_entropy_backward(grad_loss, X, W, target, lse, *, ignore_index=-100, logits=None, dX=None, dW=None,
                                  need=(True, True), workspace=None, stream=None):
    """(dX, dW) = the gradients of sum_t grad_loss_t·loss_t (tgemm_linear_ce_backward).  grad_loss: float32, one
    value a row or one of no dimension for all; lse, and logits if it left them, as linear_cross_entropy_forward gave
    them (without logits they are formed again).  dX, dW: row-major tensors to write to; need: which of the two are computed (None is returned for the other)."""
    c = _Call(X, W, stream)
    target = c.target(target)
    lse = _floats(lse, "lse", (c.T,), c.device)
    dX, dW, outs = _gradients(c, dX, dW, need)
    c.queue("tgemm_linear_ce_backward", target.data_ptr(), int(ignore_index), lse.data_ptr(), *c.logits(logits),
            *_grad_loss(c, grad_loss), 0, *outs, *c.room(workspace, 0, 1))
    return dX, dW


def linear_distillation_forward(X, W, teacher_ids, teacher_logits, *, temperature=1.0, loss=None, lse=None,
                                student=None, logits=None, workspace=None, stream=None):
    """(loss, lse, student) of the rows (tgemm_linear_kd_forward) for a teacher's top logits: teacher_ids (T×K,
    int64) the words and teacher_logits (T×K, float32, bfloat16 or float16) their logits; an entry with the logit
    -inf is absent.  With q the softmax of a row's logits / temperature over its entries and z the student's logits
    / temperature, loss_t = temperature²·sum_k q_k·(log q_k - (z_k - lse_t)), 0 for a row without entries and NaN
    where an entry's id is outside the vocabulary.  student: z at the teacher's ids (0 where absent).  logits: as
    linear_cross_entropy_forward's, before the division by the temperature."""
    c = _Call(X, W, stream)
    teacher = c.teacher(teacher_ids, teacher_logits, temperature)
    loss, lse = c.floats(loss, "loss", (c.T,)), c.floats(lse, "lse", (c.T,))
    student = c.floats(student, "student", (c.T, c.K))
    c.queue("tgemm_linear_kd_forward", *teacher, loss.data_ptr(), lse.data_ptr(), student.data_ptr(),
            *c.logits(logits), 0, *c.room(workspace, c.K, 0))
    return loss, lse, student


def linear_distillation_backward(grad_loss, X, W, teacher_ids, teacher_logits, lse, student, *, temperature=1.0,
                                 logits=None, dX=None, dW=None, need=(True, True), workspace=None, stream=None):
    """(dX, dW) = the gradients of sum_t grad_loss_t·loss_t (tgemm_linear_kd_backward); lse, student and, if it left
    them, logits as linear_distillation_forward gave them, the rest as linear_cross_entropy_backward."""
    c = _Call(X, W, stream)
    teacher = c.teacher(teacher_ids, teacher_logits, temperature)
    lse = _floats(lse, "lse", (c.T,), c.device)
    student = _floats(student, "student", (c.T, c.K), c.device)
    dX, dW, outs = _gradients(c, dX, dW, need)
    c.queue("tgemm_linear_kd_backward", *teacher, lse.data_ptr(), student.data_ptr(), *c.logits(logits),
            *_grad_loss(c, grad_loss), 0, *outs, *c.room(workspace, c.K, 1))
    return dX, dW


@functools.lru_cache(maxsize=None)
def _functions():
    """The differentiable forms.  One backward pass per forward pass through each; there is no second derivative."""
    import torch
    from torch.autograd.function import once_differentiable

    def gradients(ctx, grad, c, summary):
        """What _gradients and _grad_loss give, for what torch hands over."""
        need_x, need_w = ctx.needs_input_grad[:2]
        dX = torch.empty((c.T, c.D), dtype=c.dtype, device=c.device) if need_x else None
        dW = torch.empty((c.V, c.D), dtype=c.dtype, device=c.device) if need_w else None
        return dX, dW, (grad.data_ptr(), grad.stride(0) if c.T > 1 and grad.dim() else 0,
                        0 if summary is None else summary.data_ptr() + 8, _ptr(dX), c.D, _ptr(dW), c.D)

    class CrossEntropy(torch.autograd.Function):
        @staticmethod
        def forward(ctx, X, W, target, ignore_index, reduction, keep):
            c = _Call(X, W, None)
            target = c.target(target)
            loss, kept, at = c.results(reduction)
            logits = c.keep(keep) if any(ctx.needs_input_grad) else None
            c.queue("tgemm_linear_ce_forward", target.data_ptr(), int(ignore_index), *at[:2], *c.logits(logits), at[2],
                    *c.room(None, 0, 0))
            ctx.save_for_backward(X, W, target, *kept, logits)
            ctx.call, ctx.ignore_index = c, int(ignore_index)
            return loss

        @staticmethod
        @once_differentiable
        def backward(ctx, grad):
            X, W, target, lse, summary, logits = ctx.saved_tensors
            c = ctx.call.again(X, W, lse, summary, logits)
            dX, dW, rest = gradients(ctx, grad, c, summary)
            c.queue("tgemm_linear_ce_backward", target.data_ptr(), ctx.ignore_index, lse.data_ptr(), *c.logits(logits),
                    *rest, *c.room(None, 0, 1))
            return dX, dW, None, None, None, None

    class Distillation(torch.autograd.Function):
        @staticmethod
        def forward(ctx, X, W, teacher_ids, teacher_logits, temperature, reduction, keep):
            c = _Call(X, W, None)
            teacher = c.teacher(teacher_ids, teacher_logits, temperature)
            loss, kept, at = c.results(reduction)
            student = torch.empty((c.T, c.K), dtype=torch.float32, device=c.device)
            logits = c.keep(keep) if any(ctx.needs_input_grad) else None
            c.queue("tgemm_linear_kd_forward", *teacher, *at[:2], student.data_ptr(), *c.logits(logits), at[2],
                    *c.room(None, c.K, 0))
            ctx.save_for_backward(X, W, teacher_ids, teacher_logits, *kept, student, logits)
            ctx.call, ctx.temperature = c, temperature
            return loss

        @staticmethod
        @once_differentiable
        def backward(ctx, grad):
            X, W, ids, top, lse, summary, student, logits = ctx.saved_tensors
            c = ctx.call.again(X, W, lse, summary, student, logits)
            dX, dW, rest = gradients(ctx, grad, c, summary)
            c.queue("tgemm_linear_kd_backward", *c.teacher(ids, top, ctx.temperature), lse.data_ptr(), student.data_ptr(),
                    *c.logits(logits), *rest, *c.room(None, c.K, 1))
            return dX, dW, None, None, None, None, None

    return CrossEntropy, Distillation


def _choices(reduction, keep_logits):
    """The two, checked; nothing is kept where no backward pass can come (autograd is off within a Function)."""
    import torch

    if reduction not in REDUCTIONS:
        raise ValueError(f"reduction must be one of {REDUCTIONS}")
    if keep_logits not in (None, True, False):
        raise ValueError("keep_logits must be None, True or False")
    return reduction, keep_logits if torch.is_grad_enabled() else False


def linear_cross_entropy(X, W, target, *, ignore_index=-100, reduction="mean", keep_logits=None):
    """The softmax cross entropy of the logits X·Wᵀ against `target`, differentiable in X and W.  reduction: "mean"
    over the rows whose target is not ignore_index (0 if there is none), "sum", or "none" for the losses of the rows.
    Losses are float32; gradients have the type of X and W.  keep_logits: False: the logits are held nowhere and formed
    again in the backward pass; True: they are held until then (T×V float32), which is faster by up to a fifth where
    the inner size is large; None: held where that is faster and takes no more than 256 MiB.  Without a gradient to
    compute they are never held."""
    return _functions()[0].apply(X, W, target, ignore_index, *_choices(reduction, keep_logits))


def linear_distillation(X, W, teacher_ids, teacher_logits, *, temperature=1.0, reduction="mean", keep_logits=None):
    """The distillation loss of the logits X·Wᵀ against a teacher's top logits (linear_distillation_forward),
    differentiable in X and W (the teacher's logits get no gradient).  reduction: "mean" over the rows that have an
    entry (0 if none has), "sum" or "none"; keep_logits as linear_cross_entropy's."""
    return _functions()[1].apply(X, W, teacher_ids, teacher_logits, temperature, *_choices(reduction, keep_logits))
