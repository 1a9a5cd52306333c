"""Updates made orthogonal by Newton-Schulz products, for torch tensors.

``orthogonalize`` takes a matrix, or a stack of matrices of one shape (the
adapters of a model, the weights of its blocks), and gives what the Muon
optimiser applies in place of it.  It is queued on `stream` (default: torch's
current stream of G's device) and returns without waiting.  include/tgemm.h
states the arithmetic.
"""

from __future__ import annotations

import ctypes
import functools

from . import _lib
from ._lib import TgemmError
from .linear_loss import _no_tangents, _types

MUON = (3.4445, -4.7750, 2.0315)


def _floats_of(v):
    """A number as a float, rows of them as tuples: what is kept by its values, whatever they come in."""
    if type(v) is tuple and set(map(type, v)) == {float}:
        return v
    if hasattr(v, "__iter__") and getattr(v, "ndim", 1) and not isinstance(v, str):  # (an array of no dimension is a number)
        return tuple(_floats_of(e) for e in v)
    return float(v)


@functools.lru_cache(maxsize=64)
def _coefficients(coefficients, steps):
    """3·steps floats; coefficients: floats, or tuples of them."""
    rows = coefficients if coefficients and isinstance(coefficients[0], tuple) else (coefficients,) * steps
    if len(rows) != steps or any(not isinstance(r, tuple) or len(r) != 3 for r in rows):
        raise ValueError("coefficients must be three numbers, or as many rows of three as there are steps")
    return (ctypes.c_float * (3 * steps))(*(float(c) for r in rows for c in r))


def _stack(t, name):
    """(batch, rows, columns, leading dimension, stride) of a row-major matrix or a stack of them."""
    import torch

    if not isinstance(t, torch.Tensor) or t.dim() not in (2, 3) or t.dtype not in _types():
        raise TypeError(f"{name} must be a 2-D or 3-D float32, bfloat16 or float16 torch tensor")
    if not t.is_cuda:
        raise TypeError(f"{name} must live on a GPU")
    rows, cols = t.shape[-2:]
    batch = t.shape[0] if t.dim() == 3 else 1
    down, across = t.stride()[-2:]
    if t.numel() and (cols > 1 and across != 1 or rows > 1 and down < cols):
        raise ValueError(f"{name} must be row-major")
    ld = max(down, cols, 1) if rows > 1 else max(cols, 1)
    return batch, rows, cols, ld, t.stride(0) if batch > 1 and t.numel() else 0


@functools.lru_cache(maxsize=None)
def _function():
    """The call as a node of a graph, which no backward pass gets through."""
    import torch

    class Orthogonalize(torch.autograd.Function):
        @staticmethod
        def forward(ctx, G, steps, coefficients, eps, workspace, stream):
            return _run(G, steps, coefficients, eps, None, workspace, stream)

        @staticmethod
        def backward(ctx, grad):
            raise NotImplementedError("orthogonalize has no derivative: call it on G.detach() or under torch.no_grad()")

    return Orthogonalize


def orthogonalize(G, *, steps=5, coefficients=MUON, eps=1e-7, out=None, workspace=None, stream=None):
    """X_steps of X_0 = G / (|G| + eps) and X <- a·X + (b·S + c·S·S)·X with S = X·Xᵀ (of the transpose where G has more
    rows than columns): G with its singular values brought near 1 (tgemm_orthogonalize).  G: a row-major matrix or a
    stack of them (3-D), float32, bfloat16 or float16; the result has its type.  coefficients: (a, b, c), or a row of
    three for each step.  out: a tensor like G to write to, not G itself; workspace: a CUDA uint8 tensor of at least
    tgemm_orthogonalize_workspace_size bytes (allocated if omitted; two calls in flight at once need two).  Not
    differentiable: a backward pass through the result raises NotImplementedError."""
    import torch

    _no_tangents("orthogonalize", G)
    if torch.is_grad_enabled() and isinstance(G, torch.Tensor) and G.requires_grad:
        if out is not None:
            raise RuntimeError("orthogonalize has no derivative, so a G that requires a gradient is not written to out: "
                               "call it on G.detach() or under torch.no_grad()")
        return _function().apply(G, steps, coefficients, eps, workspace, stream)
    return _run(G, steps, coefficients, eps, out, workspace, stream)


def _run(G, steps, coefficients, eps, out, workspace, stream):
    import torch

    batch, rows, cols, ldg, stride_g = _stack(G, "G")
    steps = int(steps)
    if steps < 1:
        raise ValueError("steps must be at least 1")
    numbers = _coefficients(_floats_of(coefficients), steps)
    device, made = G.device, []
    if out is None:
        out = torch.empty(G.shape, dtype=G.dtype, device=device)
        made.append(out)
        ldo, stride_out = max(cols, 1), rows * cols
    else:
        _, _, _, ldo, stride_out = _stack(out, "out")
        if out.shape != G.shape:
            raise ValueError(f"out must be {'x'.join(map(str, G.shape))}")
        if out.dtype != G.dtype or out.device != device:
            raise TypeError(f"out must be {G.dtype} and live on {device}")
    dtype = _types()[G.dtype]
    if workspace is None:
        need = _lib.library().tgemm_orthogonalize_workspace_size(dtype, batch, rows, cols, steps)
        workspace = torch.empty(need or 1, dtype=torch.uint8, device=device)
        made.append(workspace)
    elif not isinstance(workspace, torch.Tensor) or workspace.dtype != torch.uint8:
        raise TypeError("workspace must be a CUDA uint8 tensor")
    elif workspace.device != device or not workspace.is_contiguous():
        raise TypeError(f"workspace must be contiguous and live on {device}")
    if stream is None:
        stream = torch.cuda.current_stream(device).cuda_stream
    else:
        from . import _hold_for_stream

        _hold_for_stream(stream, device, *made)
    with torch.cuda.device(device):
        st = _lib.library().tgemm_orthogonalize(dtype, batch, rows, cols, G.data_ptr(), ldg, stride_g, steps, numbers,
                                                float(eps), out.data_ptr(), ldo, stride_out, workspace.data_ptr(),
                                                workspace.numel(), stream)
    if st != _lib.TGEMM_SUCCESS:
        raise TgemmError(st, "tgemm_orthogonalize")
    return out
