"""ctypes binding of libtgemm.so: the C entry points under the same names.

Argument marshalling only — every step of the product runs in the HIP
kernels of libtgemm.so.  If the library has not been built this module
raises; there is no other code path.
"""

from __future__ import annotations

import ctypes
import os

HERE = os.path.dirname(os.path.abspath(__file__))
LIBRARY = os.path.join(HERE, "libtgemm.so")

# tgemm_status_t values (include/tgemm.h)
TGEMM_SUCCESS = 0
TGEMM_ERROR_INVALID_VALUE = 1
TGEMM_ERROR_NOT_SUPPORTED = 2
TGEMM_ERROR_HIP = 3
# size of the fixed device scratch behind tgemm_sgemm_splitk_noalloc (include/tgemm.h)
TGEMM_SPLITK_NOALLOC_BYTES = 32 << 20

# every function the header declares, with (restype, argtypes)
_i64 = ctypes.c_int64
_ptr = ctypes.c_void_p
_GEMM = [_i64, _i64, _i64, _ptr, _i64, _ptr, _i64, _ptr, _i64]
TGEMM_OP_N = 0
TGEMM_OP_T = 1
# tgemm_transpose_kernel_t values
TGEMM_TRANSPOSE_BLOCKED = 0
TGEMM_TRANSPOSE_NAIVE = 1
TGEMM_TRANSPOSE_TILED = 2
TGEMM_TRANSPOSE_TILED_PADDED = 3
# tgemm_dtype_t values
TGEMM_F32 = 0
TGEMM_BF16 = 1
TGEMM_F16 = 2

_HEAD = [ctypes.c_int, _i64, _i64, _i64, _ptr, _i64, _ptr, _i64]  # dtype, T, V, D, X, ldx, W, ldw
_TEACHER = [_i64, _ptr, _i64, ctypes.c_int, _ptr, _i64, ctypes.c_float]
_GRADS = [_ptr, _i64, _ptr, _ptr, _i64, _ptr, _i64]  # grad_loss, grad_step, grad_weight, dX, lddx, dW, lddw
_KEPT = [_ptr, _i64]  # logits, ldz
_ADAPTERS = [_i64, _i64] + [_ptr, _i64, _i64] * 2 + [_ptr, _ptr]  # count, rank, A, lda, stride_a, B, ldb, stride_b, ids, scales
_ROOM = [_ptr, ctypes.c_size_t, _ptr]  # workspace, its bytes, stream

SIGNATURES = {
    "tgemm_sgemm": (ctypes.c_int, _GEMM + [_ptr]),
    "tgemm_sgemm_ex": (ctypes.c_int, [ctypes.c_int, ctypes.c_int] + _GEMM + [_ptr]),
    "tgemm_sgemm_mfma_ex": (ctypes.c_int, [ctypes.c_int, ctypes.c_int] + _GEMM + [ctypes.c_int, _ptr]),
    "tgemm_sgemm_variant_for_ex": (ctypes.c_int, [ctypes.c_int, ctypes.c_int] + _GEMM),
    "tgemm_sgemm_mfma": (ctypes.c_int, _GEMM + [ctypes.c_int, _ptr]),
    "tgemm_mfma_variant_count": (ctypes.c_int, []),
    "tgemm_mfma_variant_name": (ctypes.c_char_p, [ctypes.c_int]),
    "tgemm_sgemm_variant_for": (ctypes.c_int, _GEMM),
    "tgemm_sgemm_naive": (ctypes.c_int, _GEMM + [_ptr]),
    "tgemm_sgemm_lds": (ctypes.c_int, _GEMM + [ctypes.c_int, ctypes.c_int, _ptr]),
    "tgemm_sgemm_simt": (ctypes.c_int, _GEMM + [_ptr]),
    "tgemm_transpose": (ctypes.c_int, [_i64, _i64, _ptr, _i64, _ptr, _i64, ctypes.c_int, _ptr]),
    "tgemm_sgemm_host": (ctypes.c_int, _GEMM + [_ptr, _i64, _i64, _ptr, _ptr, _ptr]),
    "tgemm_sgemm_host_workspace_size": (_i64, [_i64, _i64, _i64, _i64]),
    "tgemm_sgemm_splitk": (ctypes.c_int, _GEMM + [ctypes.c_int, _ptr, ctypes.c_size_t, _ptr]),
    "tgemm_sgemm_splitk_ex": (ctypes.c_int, [ctypes.c_int, ctypes.c_int] + _GEMM
                              + [ctypes.c_int, _ptr, ctypes.c_size_t, _ptr]),
    "tgemm_sgemm_splitk_noalloc": (ctypes.c_int, [ctypes.c_int, ctypes.c_int] + _GEMM + [ctypes.c_int, _ptr]),
    "tgemm_sgemm_splitk_workspace_size": (ctypes.c_size_t, [_i64, _i64, _i64, ctypes.c_int]),
    "tgemm_sgemm_splitk_choose": (ctypes.c_int, [_i64, _i64, _i64]),
    "tgemm_linear_loss_workspace_size": (ctypes.c_size_t, _HEAD + [_i64, ctypes.c_int]),
    "tgemm_linear_ce_forward": (ctypes.c_int, _HEAD + [_ptr, _i64] + [_ptr] * 2 + _KEPT + [_ptr] + _ROOM),
    "tgemm_linear_ce_backward": (ctypes.c_int, _HEAD + [_ptr, _i64, _ptr] + _KEPT + _GRADS + _ROOM),
    "tgemm_linear_kd_forward": (ctypes.c_int, _HEAD + _TEACHER + [_ptr] * 3 + _KEPT + [_ptr] + _ROOM),
    "tgemm_linear_kd_backward": (ctypes.c_int, _HEAD + _TEACHER + [_ptr] * 2 + _KEPT + _GRADS + _ROOM),
    "tgemm_linear_adapters_forward": (ctypes.c_int, _HEAD + _ADAPTERS + [_ptr, _i64, _ptr] + _ROOM),
    "tgemm_linear_adapters_backward": (ctypes.c_int, _HEAD + _ADAPTERS + [_ptr, _ptr, _i64] + [_ptr, _i64] * 2
                                       + [_ptr, _i64, _i64] * 2 + _ROOM),
    "tgemm_linear_adapters_workspace_size": (ctypes.c_size_t, _HEAD + [_i64, _i64, _ptr, _i64, ctypes.c_int]),
    "tgemm_orthogonalize": (ctypes.c_int, [ctypes.c_int, _i64, _i64, _i64, _ptr, _i64, _i64, ctypes.c_int, _ptr,
                                           ctypes.c_float, _ptr, _i64, _i64] + _ROOM),
    "tgemm_orthogonalize_workspace_size": (ctypes.c_size_t, [ctypes.c_int, _i64, _i64, _i64, ctypes.c_int]),
    "tgemm_status_string": (ctypes.c_char_p, [ctypes.c_int]),
    "tgemm_version": (ctypes.c_int, []),
}

_lib = None


class TgemmError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {tgemm_status_string(status)} (status {status})")


def library():
    """The loaded libtgemm.so (loads it on first use; raises if not built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIBRARY):
            raise RuntimeError(
                f"{LIBRARY} is not built; run `python -m tiled_gemm_tgemm_amd.build`")
        lib = ctypes.CDLL(LIBRARY)
        for name, (restype, argtypes) in SIGNATURES.items():
            fn = getattr(lib, name)
            fn.restype = restype
            fn.argtypes = argtypes
        _lib = lib
    return _lib


# ---- the C entry points, same names and argument order ---------------------
# (but the loss operators' `logits` and `ldz`: optional here, they come last)

def tgemm_sgemm(M, N, K, A, lda, B, ldb, C, ldc, stream=None) -> int:
    return library().tgemm_sgemm(M, N, K, A, lda, B, ldb, C, ldc, stream)


def tgemm_sgemm_ex(op_a, op_b, M, N, K, A, lda, B, ldb, C, ldc, stream=None) -> int:
    return library().tgemm_sgemm_ex(op_a, op_b, M, N, K, A, lda, B, ldb, C, ldc, stream)


def tgemm_sgemm_mfma_ex(op_a, op_b, M, N, K, A, lda, B, ldb, C, ldc, variant, stream=None) -> int:
    return library().tgemm_sgemm_mfma_ex(op_a, op_b, M, N, K, A, lda, B, ldb, C, ldc, variant, stream)


def tgemm_sgemm_variant_for_ex(op_a, op_b, M, N, K, A, lda, B, ldb, C, ldc) -> int:
    return library().tgemm_sgemm_variant_for_ex(op_a, op_b, M, N, K, A, lda, B, ldb, C, ldc)


def tgemm_sgemm_mfma(M, N, K, A, lda, B, ldb, C, ldc, variant, stream=None) -> int:
    return library().tgemm_sgemm_mfma(M, N, K, A, lda, B, ldb, C, ldc, variant, stream)


def tgemm_sgemm_naive(M, N, K, A, lda, B, ldb, C, ldc, stream=None) -> int:
    return library().tgemm_sgemm_naive(M, N, K, A, lda, B, ldb, C, ldc, stream)


def tgemm_sgemm_lds(M, N, K, A, lda, B, ldb, C, ldc, tile, pad, stream=None) -> int:
    return library().tgemm_sgemm_lds(M, N, K, A, lda, B, ldb, C, ldc, tile, pad, stream)


def tgemm_sgemm_simt(M, N, K, A, lda, B, ldb, C, ldc, stream=None) -> int:
    return library().tgemm_sgemm_simt(M, N, K, A, lda, B, ldb, C, ldc, stream)


def tgemm_transpose(M, N, A, lda, B, ldb, kernel=TGEMM_TRANSPOSE_BLOCKED, stream=None) -> int:
    return library().tgemm_transpose(M, N, A, lda, B, ldb, kernel, stream)


def tgemm_sgemm_host(M, N, K, A, lda, B, ldb, C, ldc, workspace, workspace_bytes, panel_rows,
                     compute=None, copy_in=None, copy_out=None) -> int:
    return library().tgemm_sgemm_host(M, N, K, A, lda, B, ldb, C, ldc, workspace, workspace_bytes,
                                      panel_rows, compute, copy_in, copy_out)


def tgemm_sgemm_host_workspace_size(M, N, K, panel_rows=0) -> int:
    return library().tgemm_sgemm_host_workspace_size(M, N, K, panel_rows)


def tgemm_sgemm_splitk(M, N, K, A, lda, B, ldb, C, ldc, splits, workspace, workspace_bytes,
                       stream=None) -> int:
    return library().tgemm_sgemm_splitk(M, N, K, A, lda, B, ldb, C, ldc, splits, workspace,
                                        workspace_bytes, stream)


def tgemm_sgemm_splitk_ex(op_a, op_b, M, N, K, A, lda, B, ldb, C, ldc, splits, workspace, workspace_bytes,
                          stream=None) -> int:
    return library().tgemm_sgemm_splitk_ex(op_a, op_b, M, N, K, A, lda, B, ldb, C, ldc, splits, workspace,
                                           workspace_bytes, stream)


def tgemm_sgemm_splitk_noalloc(op_a, op_b, M, N, K, A, lda, B, ldb, C, ldc, splits, stream=None) -> int:
    return library().tgemm_sgemm_splitk_noalloc(op_a, op_b, M, N, K, A, lda, B, ldb, C, ldc, splits, stream)


def tgemm_sgemm_splitk_workspace_size(M, N, K, splits) -> int:
    return library().tgemm_sgemm_splitk_workspace_size(M, N, K, splits)


def tgemm_sgemm_splitk_choose(M, N, K) -> int:
    return library().tgemm_sgemm_splitk_choose(M, N, K)


def tgemm_linear_loss_workspace_size(dtype, T, V, D, X, ldx, W, ldw, teacher_k=0, backward_pass=0) -> int:
    return library().tgemm_linear_loss_workspace_size(dtype, T, V, D, X, ldx, W, ldw, teacher_k, backward_pass)


def tgemm_linear_ce_forward(dtype, T, V, D, X, ldx, W, ldw, target, ignore_index, loss, lse, summary, workspace,
                            workspace_bytes, stream=None, logits=0, ldz=0) -> int:
    return library().tgemm_linear_ce_forward(dtype, T, V, D, X, ldx, W, ldw, target, ignore_index, loss, lse, logits,
                                             ldz, summary, workspace, workspace_bytes, stream)


def tgemm_linear_ce_backward(dtype, T, V, D, X, ldx, W, ldw, target, ignore_index, lse, grad_loss, grad_step,
                             grad_weight, dX, lddx, dW, lddw, workspace, workspace_bytes, stream=None, logits=0,
                             ldz=0) -> int:
    return library().tgemm_linear_ce_backward(dtype, T, V, D, X, ldx, W, ldw, target, ignore_index, lse, logits, ldz,
                                              grad_loss, grad_step, grad_weight, dX, lddx, dW, lddw, workspace,
                                              workspace_bytes, stream)


def tgemm_linear_kd_forward(dtype, T, V, D, X, ldx, W, ldw, K, teacher_ids, ld_ids, teacher_dtype, teacher_logits,
                            ld_logits, temperature, loss, lse, student, summary, workspace, workspace_bytes,
                            stream=None, logits=0, ldz=0) -> int:
    return library().tgemm_linear_kd_forward(dtype, T, V, D, X, ldx, W, ldw, K, teacher_ids, ld_ids, teacher_dtype,
                                             teacher_logits, ld_logits, temperature, loss, lse, student, logits, ldz,
                                             summary, workspace, workspace_bytes, stream)


def tgemm_linear_kd_backward(dtype, T, V, D, X, ldx, W, ldw, K, teacher_ids, ld_ids, teacher_dtype, teacher_logits,
                             ld_logits, temperature, lse, student, grad_loss, grad_step, grad_weight, dX, lddx, dW,
                             lddw, workspace, workspace_bytes, stream=None, logits=0, ldz=0) -> int:
    return library().tgemm_linear_kd_backward(dtype, T, V, D, X, ldx, W, ldw, K, teacher_ids, ld_ids, teacher_dtype,
                                              teacher_logits, ld_logits, temperature, lse, student, logits, ldz,
                                              grad_loss, grad_step, grad_weight, dX, lddx, dW, lddw, workspace,
                                              workspace_bytes, stream)


def tgemm_linear_adapters_forward(dtype, T, N, D, X, ldx, W, ldw, count, rank, A, lda, stride_a, B, ldb, stride_b, ids,
                                  scales, Y, ldy, hidden, workspace, workspace_bytes, stream=None) -> int:
    return library().tgemm_linear_adapters_forward(dtype, T, N, D, X, ldx, W, ldw, count, rank, A, lda, stride_a, B, ldb,
                                                   stride_b, ids, scales, Y, ldy, hidden, workspace, workspace_bytes,
                                                   stream)


def tgemm_linear_adapters_backward(dtype, T, N, D, X, ldx, W, ldw, count, rank, A, lda, stride_a, B, ldb, stride_b, ids,
                                   scales, hidden, dY, lddy, dX, lddx, dW, lddw, dA, ldda, stride_da, dB, lddb,
                                   stride_db, workspace, workspace_bytes, stream=None) -> int:
    return library().tgemm_linear_adapters_backward(dtype, T, N, D, X, ldx, W, ldw, count, rank, A, lda, stride_a, B,
                                                    ldb, stride_b, ids, scales, hidden, dY, lddy, dX, lddx, dW, lddw,
                                                    dA, ldda, stride_da, dB, lddb, stride_db, workspace,
                                                    workspace_bytes, stream)


def tgemm_linear_adapters_workspace_size(dtype, T, N, D, X, ldx, W, ldw, count, rank, dY=0, lddy=0, need=0) -> int:
    return library().tgemm_linear_adapters_workspace_size(dtype, T, N, D, X, ldx, W, ldw, count, rank, dY, lddy, need)


def tgemm_orthogonalize(dtype, batch, M, N, G, ldg, stride_g, steps, coefficients, eps, out, ldo, stride_out, workspace,
                        workspace_bytes, stream=None) -> int:
    """coefficients: the address of 3·steps floats in host memory, or a ctypes array of them."""
    return library().tgemm_orthogonalize(dtype, batch, M, N, G, ldg, stride_g, steps, coefficients, eps, out, ldo,
                                         stride_out, workspace, workspace_bytes, stream)


def tgemm_orthogonalize_workspace_size(dtype, batch, M, N, steps) -> int:
    return library().tgemm_orthogonalize_workspace_size(dtype, batch, M, N, steps)


def tgemm_mfma_variant_count() -> int:
    return library().tgemm_mfma_variant_count()


def tgemm_mfma_variant_name(variant: int):
    name = library().tgemm_mfma_variant_name(variant)
    return name.decode() if name is not None else None


def tgemm_sgemm_variant_for(M, N, K, A, lda, B, ldb, C, ldc) -> int:
    return library().tgemm_sgemm_variant_for(M, N, K, A, lda, B, ldb, C, ldc)


def tgemm_status_string(status: int) -> str:
    return library().tgemm_status_string(status).decode()


def tgemm_version() -> int:
    return library().tgemm_version()
