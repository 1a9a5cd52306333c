/*
 * libtgemm — single-precision C = A·B on one AMD Instinct MI355X (gfx950), and,
 * declared last, two losses on such a product of an output head, a projection
 * with low-rank adapters beside it, and updates made orthogonal.
 *
 * The operation is the dense product of page 1 ("[Multi-Core & GPU
 * Programming] CUDA - Matrix Multiplication", section [Matrix
 * Multiplication]): every output is the sum over k of one row of the left
 * matrix times one column of the right one.  The pages call the matrices
 * M, N, P and the size Width; here they are A (M×K), B (K×N) and C (M×N),
 * and M, N, K are sizes.
 *
 * Conventions shared by every compute entry point below
 * ------------------------------------------------------
 * Layout      Row-major float32 with leading dimensions counted in elements:
 *             A(i,k) = A[i*lda + k], B(k,j) = B[k*ldb + j], C(i,j) = C[i*ldc + j]
 *             (page 1, section [Coalescing], indexes M as M[row*width + k]).
 *             Requires lda >= max(1,K), ldb >= max(1,N), ldc >= max(1,N).
 * Semantics   C(i,j) = sum_{k<K} A(i,k)·B(k,j).  C is overwritten, never read
 *             (page 1 keeps the sum in a register and writes the output once,
 *             at the end).  K = 0 sets C to +0.0; M = 0 or N = 0 is a no-op.
 * Memory      A, B and C are device pointers (hipMalloc, or a torch CUDA
 *             tensor's storage) owned by the caller.  The library allocates
 *             nothing and keeps no per-call state.  C must not overlap A or B.
 * Streams     Work is queued on `stream` (NULL = the default stream) and the
 *             call returns without waiting; results are ready once the
 *             stream has been synchronised (page 3, "CUDA.3 Writing CUDA SIMT
 *             Kernels", Global Memory: kernels hand results back only through
 *             device memory).
 * Errors      Argument problems are reported before anything is queued, and C
 *             is then left untouched.  TGEMM_ERROR_HIP means the launch itself
 *             failed.  A fault inside a kernel shows up at the caller's next
 *             stream synchronisation, as for any asynchronous HIP work.
 *             Nothing is printed and no C++ exception crosses this interface.
 * Sizes       M, N, K up to 2^31 - 2^16 (TGEMM_ERROR_NOT_SUPPORTED above);
 *             element offsets are 64-bit.
 * Threads     All entry points are re-entrant and may be called concurrently
 *             on different streams.
 * Rounding    The tiled MFMA kernels sum in an order of their own; for real
 *             inputs the result lies within 4·K·2^-24·sum_k|A(i,k)·B(k,j)| of
 *             the exact one, and integer-valued inputs whose partial sums stay
 *             below 2^24 in magnitude give the exact result.  The two
 *             one-product-per-step kernels (naive, LDS-tiled) add the products
 *             one fused multiply-add at a time in ascending k.
 */
#ifndef TGEMM_H
#define TGEMM_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Same definition as the HIP runtime's, so either header may come first. */
typedef struct ihipStream_t *hipStream_t;

/* How an operand is stored (BLAS's "op"): as is, or transposed. */
typedef enum tgemm_op {
    TGEMM_OP_N = 0, /* op(X) = X */
    TGEMM_OP_T = 1  /* op(X) = Xᵀ */
} tgemm_op_t;

/* Element types of the operators on 16-bit tiles: losses, adapters, orthogonalised updates. */
typedef enum tgemm_dtype {
    TGEMM_F32 = 0,
    TGEMM_BF16 = 1,
    TGEMM_F16 = 2
} tgemm_dtype_t;

typedef enum tgemm_status {
    TGEMM_SUCCESS = 0,
    TGEMM_ERROR_INVALID_VALUE = 1, /* bad size, leading dimension, pointer or overlap, or an
                                      operand that would run past the end of the address space */
    TGEMM_ERROR_NOT_SUPPORTED = 2, /* a size above 2^31-2^16, or an unknown kernel choice */
    TGEMM_ERROR_HIP = 3            /* the HIP runtime refused the launch */
} tgemm_status_t;

/*
 * C = A·B with the tiled matrix-core kernel: the product of page 1 computed
 * tile by tile as in page 1's section [Shared Memory] and page 2 ("Lec 29 ·
 * GPU Architecture (2)") §1.2 — tiles of A and B staged through on-chip
 * memory in phases, one barrier per phase, sums kept in registers — with
 * the tile shape chosen from M, N, K and the alignment of A, B and C.
 * Arguments and errors: see the conventions above.
 */
tgemm_status_t tgemm_sgemm(int64_t M, int64_t N, int64_t K,
                           const float *A, int64_t lda,
                           const float *B, int64_t ldb,
                           float *C, int64_t ldc, hipStream_t stream);

/*
 * C = op(A)·op(B), op(A) M×K and op(B) K×N, with the tiled matrix-core kernel.
 * op_a = TGEMM_OP_T: A is stored K×M row-major (op(A) = Aᵀ), op(A)(i,k) =
 * A[k*lda + i], lda >= max(1,M); otherwise as tgemm_sgemm.  op_b = TGEMM_OP_T:
 * B is stored N×K, op(B)(k,j) = B[j*ldb + k], ldb >= max(1,K).  Each operand
 * is read along the dimension it is contiguous in and kept that way on chip,
 * the fragments taking whichever order the matrix cores need (page 1,
 * section [Coalescing], "Corner Turning").  Other values of op_a / op_b:
 * TGEMM_ERROR_NOT_SUPPORTED.  Transposed operands need leading dimensions
 * below 2^21 (the 64-bit-pointer configuration takes operands as stored
 * only): otherwise TGEMM_ERROR_NOT_SUPPORTED.  tgemm_sgemm(...) is
 * tgemm_sgemm_ex(TGEMM_OP_N, TGEMM_OP_N, ...).
 */
tgemm_status_t tgemm_sgemm_ex(tgemm_op_t op_a, tgemm_op_t op_b, int64_t M, int64_t N, int64_t K,
                              const float *A, int64_t lda,
                              const float *B, int64_t ldb,
                              float *C, int64_t ldc, hipStream_t stream);

/*
 * C = A·B (row-major operands, as tgemm_sgemm; transposed ones through
 * tgemm_sgemm_splitk_ex below) with the k range split
 * across work-groups: the sum over k of page 1's section [Matrix
 * Multiplication] taken in up to `splits` contiguous slices that run side by
 * side, each slice's partial product written to its own M×N block of
 * `workspace`, and a second pass adding the blocks into C in slice order.
 * For shapes with too few output tiles to fill the GPU and a long K (e.g.
 * 512×512×16384).  Results do not depend on timing; the summation order
 * differs from tgemm_sgemm's, within the same error bound, and integer
 * inputs whose sums stay below 2^24 give the same exact results.
 *   splits: 1 ... 64; 1 runs tgemm_sgemm (workspace unused, may be NULL).
 *     The library may run fewer slices than asked (each slice is a whole
 *     number of its tile configuration's K steps), never more.
 *   workspace: device memory owned by the caller, 16-byte aligned, at least
 *     tgemm_sgemm_splitk_workspace_size(M, N, K, splits) bytes, overlapping
 *     none of A, B, C; its contents on return are unspecified.  The call
 *     allocates nothing.  Two calls in flight at once need two workspaces.
 * Errors as tgemm_sgemm; also TGEMM_ERROR_INVALID_VALUE for splits outside
 * 1 ... 64, a missing, misaligned, overlapping or too small workspace.
 */
tgemm_status_t tgemm_sgemm_splitk(int64_t M, int64_t N, int64_t K,
                                  const float *A, int64_t lda,
                                  const float *B, int64_t ldb,
                                  float *C, int64_t ldc, int splits,
                                  void *workspace, size_t workspace_bytes, hipStream_t stream);

/*
 * tgemm_sgemm_splitk with operands stored transposed, as tgemm_sgemm_ex
 * (op_a / op_b = TGEMM_OP_T: A stored K×M, B stored N×K); the same
 * workspace.  tgemm_sgemm_splitk(...) is tgemm_sgemm_splitk_ex(TGEMM_OP_N,
 * TGEMM_OP_N, ...).
 */
tgemm_status_t tgemm_sgemm_splitk_ex(tgemm_op_t op_a, tgemm_op_t op_b, int64_t M, int64_t N, int64_t K,
                                     const float *A, int64_t lda,
                                     const float *B, int64_t ldb,
                                     float *C, int64_t ldc, int splits,
                                     void *workspace, size_t workspace_bytes, hipStream_t stream);

/* Bytes of the fixed device scratch behind tgemm_sgemm_splitk_noalloc. */
#define TGEMM_SPLITK_NOALLOC_BYTES ((size_t)32 << 20)

/*
 * tgemm_sgemm_splitk_ex for callers that cannot allocate device memory: code
 * under HIP graph capture, tight serving loops, harnesses that forbid
 * hipMalloc.  The same product with the same kernels and slices, so the same
 * results bit for bit, but the slices' partial products live in a fixed
 * scratch array of TGEMM_SPLITK_NOALLOC_BYTES (32 MiB) that the library holds
 * on each GPU it runs on until the process ends, not in a caller's
 * workspace.  The call allocates nothing: no hipMalloc, hipFree or
 * allocating library routine.  Every call on one GPU shares that GPU's
 * array, which keeps the last call's contents (nothing in it needs to start
 * at zero): calls whose work overlaps in time on one GPU (two streams, two
 * threads) race and give wrong results, so serialise them.  Argument
 * meaning, layout, ownership and errors as tgemm_sgemm_splitk_ex, with
 * TGEMM_ERROR_NOT_SUPPORTED when tgemm_sgemm_splitk_workspace_size(M, N, K,
 * splits) exceeds TGEMM_SPLITK_NOALLOC_BYTES (e.g. 1024×1024 with more than 8
 * splits), and TGEMM_ERROR_HIP if the array's device address cannot be
 * obtained on the current device.
 */
tgemm_status_t tgemm_sgemm_splitk_noalloc(tgemm_op_t op_a, tgemm_op_t op_b, int64_t M, int64_t N, int64_t K,
                                          const float *A, int64_t lda,
                                          const float *B, int64_t ldb,
                                          float *C, int64_t ldc, int splits, hipStream_t stream);

/* Workspace bytes tgemm_sgemm_splitk needs: splits·M·N·4; 0 when splits <= 1,
 * splits > 64, a size is not positive or above 2^31-2^16, or the product does
 * not fit in a size_t. */
size_t tgemm_sgemm_splitk_workspace_size(int64_t M, int64_t N, int64_t K, int splits);

/* The split count (1, 2, 4, ..., 64) the library's cost model expects to be
 * fastest for M, N, K with 16-byte-aligned row-major operands; 1 means no
 * split (then tgemm_sgemm is the call to make).  Host-only: no GPU work. */
int tgemm_sgemm_splitk_choose(int64_t M, int64_t N, int64_t K);

/*
 * Same product with an explicitly chosen matrix-core tile configuration,
 * 0 <= variant < tgemm_mfma_variant_count().  Variants with 16-byte loads
 * ("vec4") need A and B 16-byte aligned, lda, ldb and the stored row lengths
 * of A and B (K and N here) multiples of 4; buffer-load variants need their
 * 32-bit offsets to span the leading dimensions; otherwise, and for an
 * unknown variant, TGEMM_ERROR_NOT_SUPPORTED.
 */
tgemm_status_t tgemm_sgemm_mfma(int64_t M, int64_t N, int64_t K,
                                const float *A, int64_t lda,
                                const float *B, int64_t ldb,
                                float *C, int64_t ldc, int variant, hipStream_t stream);

/* tgemm_sgemm_mfma with operand orders, as tgemm_sgemm_ex. */
tgemm_status_t tgemm_sgemm_mfma_ex(tgemm_op_t op_a, tgemm_op_t op_b, int64_t M, int64_t N, int64_t K,
                                   const float *A, int64_t lda,
                                   const float *B, int64_t ldb,
                                   float *C, int64_t ldc, int variant, hipStream_t stream);

/* Number of matrix-core tile configurations. */
int tgemm_mfma_variant_count(void);

/*
 * Static description of a variant, e.g. "m256n128k16_w2x2_vec4" (macro tile
 * 256×128, depth 16 per phase, 2×2 wavefronts, 16-byte loads),
 * "m32n32k32_w1x1s8_vec4" (32×32 tile staged through LDS, K split over 8
 * single-wavefront slices), "..._nn" (operands as stored only: TGEMM_OP_T is
 * refused; "m160n128k32_w1x4_vec4_nn" also writes C in 16-byte row pieces,
 * so tgemm_sgemm picks it only when C and ldc are 16-byte aligned, though it
 * runs on any C), "..._flat" (64-bit pointers, any leading dimension,
 * operands as stored only); NULL for an index out of range.
 */
const char *tgemm_mfma_variant_name(int variant);

/* The variant tgemm_sgemm would run for these arguments; -1 if none applies. */
int tgemm_sgemm_variant_for(int64_t M, int64_t N, int64_t K,
                            const float *A, int64_t lda,
                            const float *B, int64_t ldb,
                            const float *C, int64_t ldc);

/* The variant tgemm_sgemm_ex would run for these arguments; -1 if none applies. */
int tgemm_sgemm_variant_for_ex(tgemm_op_t op_a, tgemm_op_t op_b, int64_t M, int64_t N, int64_t K,
                               const float *A, int64_t lda,
                               const float *B, int64_t ldb,
                               const float *C, int64_t ldc);

/*
 * Ablation 1 — one thread per output (page 1, section [Matrix
 * Multiplication], the simplest kernel and "Work Flow"; page 2 §1.2, naive
 * kernel): a 16×16 thread block per 16×16 output tile; each thread reads its
 * row of A and column of B straight from device memory and adds one fused
 * multiply-add per k in ascending order.  Arguments and errors as above.
 */
tgemm_status_t tgemm_sgemm_naive(int64_t M, int64_t N, int64_t K,
                                 const float *A, int64_t lda,
                                 const float *B, int64_t ldb,
                                 float *C, int64_t ldc, hipStream_t stream);

/*
 * Ablation 2 — the shared-memory tiled kernel (page 1, section [Shared
 * Memory], "Work Flow - Compute Block(0, 0)" and "Tiled Matrix
 * Multiplication Kernel"; page 2 §1.2): tile×tile threads per block, two
 * tile×tile on-chip tiles; per phase every thread copies one element of A
 * and one of B, the block synchronises, every thread adds the tile's
 * products to its register sum (one fused multiply-add per k, ascending),
 * and the block synchronises again.  Out-of-range elements load as zero.
 * tile is 2, 8, 16 or 32.  pad = 1 adds one word to each tile row
 * (page 2 §1.4, tile[32][33]); pad = 0 does not.  Other values:
 * TGEMM_ERROR_NOT_SUPPORTED.  Arguments and errors otherwise as above.
 */
tgemm_status_t tgemm_sgemm_lds(int64_t M, int64_t N, int64_t K,
                               const float *A, int64_t lda,
                               const float *B, int64_t ldb,
                               float *C, int64_t ldc, int tile, int pad, hipStream_t stream);

/*
 * Ablation 3 — the tiled kernel with more work per thread (page 1, end of
 * section [Shared Memory], "Tile Size 결정": let each thread compute several
 * outputs to use more on-chip memory), on the vector ALUs: 256 threads per
 * 128×128 tile, an 8×8 block of outputs per thread in registers, phases of 8
 * values of k staged through LDS (A transposed on the way in, page 1 section
 * [Coalescing], "Corner Turning"), two LDS stages, one barrier per phase.
 * Every output is one fused multiply-add chain in ascending k, so the result
 * equals tgemm_sgemm_naive's bit for bit.  Arguments and errors as above.
 */
tgemm_status_t tgemm_sgemm_simt(int64_t M, int64_t N, int64_t K,
                                const float *A, int64_t lda,
                                const float *B, int64_t ldb,
                                float *C, int64_t ldc, hipStream_t stream);

/* Kernels of tgemm_transpose. */
typedef enum tgemm_transpose_kernel {
    TGEMM_TRANSPOSE_BLOCKED = 0,     /* default: 4×4 blocks per thread, whole cache lines both ways */
    TGEMM_TRANSPOSE_NAIVE = 1,       /* page 2 §1.4: rows in, strided stores out */
    TGEMM_TRANSPOSE_TILED = 2,       /* page 2 §1.4: through a 32×32 LDS tile */
    TGEMM_TRANSPOSE_TILED_PADDED = 3 /* page 2 §1.4: LDS tile with rows of 33 words */
} tgemm_transpose_kernel_t;

/*
 * B = Aᵀ: the matrix transpose of page 2 ("Lec 29 · GPU Architecture (2)"),
 * §1.4.  A is M×N row-major with leading dimension lda >= max(1, N); B is
 * N×M row-major with ldb >= max(1, M); B(j, i) = A(i, j) for i < M, j < N,
 * every element moved as a 32-bit word (bit patterns, NaN payloads and
 * signed zeros arrive unchanged); nothing else of B is written.  Device
 * pointers owned by the caller; B must not overlap A (no in-place
 * transpose).  Asynchronous on `stream`.  M = 0 or N = 0 is a no-op.
 *
 * kernel selects the page's progression on this GPU — NAIVE (32×32 tiles,
 * 32×8 threads, four elements per thread; reads along A's rows, stores down
 * B's columns), TILED (the same tile staged through LDS, barrier, swapped
 * block offsets, stores along B's rows), TILED_PADDED (LDS rows padded to 33
 * words) — or BLOCKED, this library's kernel: no LDS; each thread moves
 * 4×4 blocks, each with four 16-byte reads and four 16-byte writes, so a
 * wavefront's every access is whole 128-byte runs (when A and B are 16-byte
 * aligned and lda, ldb are multiples of 4; otherwise single-word accesses
 * with the same mapping); from 2^24 elements on, four blocks side by side
 * per thread.
 *
 * Errors: TGEMM_ERROR_INVALID_VALUE for negative sizes, short leading
 * dimensions, null or misaligned pointers, or overlap;
 * TGEMM_ERROR_NOT_SUPPORTED for an unknown kernel or a size above
 * 2^31 - 2^16; TGEMM_ERROR_HIP if the launch fails.  Nothing is queued on
 * an error.
 */
tgemm_status_t tgemm_transpose(int64_t M, int64_t N, const float *A, int64_t lda,
                               float *B, int64_t ldb, tgemm_transpose_kernel_t kernel,
                               hipStream_t stream);

/*
 * C = A·B with A, B and C in HOST memory, the transfers overlapped with the
 * product (page 1, section [CUDA Performance Considerations], "Overlap I/O
 * with Computation": host↔device copies and computation at the same time,
 * on streams).  B is copied to the device once; A and C move in panels of
 * panel_rows rows (0: about M/4, rounded up to 256): while panel p is
 * multiplied on `compute` (an ordinary tgemm_sgemm call), panel p+1 of A is
 * copied in on `copy_in` and panel p-1 of C is copied out on `copy_out`.
 * Pass three different streams for the copies to overlap (one stream, or
 * NULL for all three, is correct but serial).  A, B, C should be page-locked
 * (hipHostMalloc, or a pinned torch CPU tensor) for the copies to run
 * asynchronously; pageable memory works but serialises them.
 *
 * Layout and semantics as tgemm_sgemm (row-major, leading dimensions in
 * elements, C overwritten; K = 0 sets C to +0.0 on the host without device
 * work; M = 0 or N = 0 is a no-op).  `workspace` is caller-owned DEVICE
 * memory, 256-byte aligned, of at least tgemm_sgemm_host_workspace_size(M,
 * N, K, panel_rows) bytes (B, two A panels and two C panels); the library
 * allocates nothing.  Unlike the device entry points this call BLOCKS: it
 * returns once C is complete in host memory (or after an error, once
 * everything it queued has finished).
 *
 * Errors: TGEMM_ERROR_INVALID_VALUE for the device entry points' argument
 * errors (host C overlapping host A or B), a negative panel_rows, or a
 * missing, misaligned or too small workspace; TGEMM_ERROR_NOT_SUPPORTED for
 * sizes as above; TGEMM_ERROR_HIP if a copy, event or launch fails (C may
 * then be partly written).
 */
tgemm_status_t tgemm_sgemm_host(int64_t M, int64_t N, int64_t K,
                                const float *A, int64_t lda,
                                const float *B, int64_t ldb,
                                float *C, int64_t ldc,
                                void *workspace, int64_t workspace_bytes, int64_t panel_rows,
                                hipStream_t compute, hipStream_t copy_in, hipStream_t copy_out);

/* Device workspace bytes tgemm_sgemm_host needs; 0 if it needs none (M, N or
 * K zero); -1 for invalid sizes or a negative panel_rows. */
int64_t tgemm_sgemm_host_workspace_size(int64_t M, int64_t N, int64_t K, int64_t panel_rows);

/*
 * Losses on the product Z = X·Wᵀ of an output head
 * ------------------------------------------------
 * X is T×D (a row a token's hidden state), W is V×D (a row a word of the
 * vocabulary), both row-major with leading dimensions ldx, ldw >= D in
 * elements, of type `dtype` (both the same).  Z is T×V and read by nothing but
 * the loss; it is formed tile by tile in registers and reduced there to a
 * maximum and a sum of exponentials a row.  Its memory is the caller's choice:
 * without `logits` (NULL) it is nowhere held, and formed again in the backward
 * pass, a piece of the vocabulary at a time; with `logits` (T×V float32, ldz >=
 * V) the forward call leaves it there, and the backward call reads it from
 * there (the same array and ldz, unchanged).
 *
 * Types       dtype float32, bf16 or fp16: the type of X, W and their
 *             gradients.  Products of 16-bit values are exact and summed in
 *             float32.  A float32 operand is split into three bf16 planes (24
 *             bits) and the six products of planes that reach 2^-24 of the
 *             largest are summed in float32; an infinity there, or a value
 *             above 3.39e38, gives NaN or infinity.  Row statistics, losses and the sums over pieces are
 *             float32.  The logits' gradient is rounded to the operands' type
 *             (float32: to three planes; up to 128 rows: to two numbers of the
 *             type that add up to it) before the two gradient products.
 *             fp16 rows with factors of their own share a range of 40 binary
 *             places in dW: a row's part is rounded by up to 2^-38 of the
 *             largest product of a factor and a state besides.
 * Sizes       0 <= T < 2^24, 1 <= V <= 2^24, 1 <= D <= 2^22, 1 <= K <= 1024,
 *             leading dimensions up to 2^40; larger ones, a product of 2^31
 *             tiles and more (T·V from about 2^47 on; a tile has up to
 *             256×256 entries), and an unknown dtype:
 *             TGEMM_ERROR_NOT_SUPPORTED.  T = 0: nothing but `summary`
 *             and a zero dW is written.
 * Workspace   Device memory of the caller, 16-byte aligned, at least
 *             tgemm_linear_loss_workspace_size(...) bytes for the same
 *             arguments, overlapping none of the others.  Its contents on
 *             entry do not matter and on return are unspecified.  Two calls in
 *             flight at once need two.
 *             A backward call's holds a piece of the logits' gradient: 256
 *             MiB of it or, where that is more, 2048 words of all rows (2
 *             bytes each, float32 6, up to 128 rows 4), but no more words than
 *             there are; besides it X as the products read it and sums of dX
 *             and dW in float32.
 *             float32 operands take their planes in either call: 6·V·D bytes
 *             for W, more than W itself, and 6·T·D for X (up to 32 rows of a
 *             forward call none).  16-bit ones are read as they are stored
 *             where D and the leading dimension are multiples of 8 (forward
 *             calls and fp16: X's D one of 64) and the rows start 16-byte
 *             aligned, and copied otherwise: 2·V·D.
 * Errors      As above, before anything is queued; also
 *             TGEMM_ERROR_INVALID_VALUE for a missing, misaligned, overlapping
 *             or too small workspace, an output that overlaps an input or
 *             another output (each taken from its first element to its last,
 *             with what lies between its rows), a misaligned or missing array,
 *             a negative grad_step, a temperature that is not positive and
 *             finite.
 * Indices     An index out of [0, V) is never used as an address: its row's
 *             loss is NaN, and so are its row of dX and all of dW.
 * Rows        A row that does not count (its target is ignore_index, or all of
 *             its teacher logits are -infinity) has the loss 0, a zero row of
 *             dX and no part in dW, whatever X holds there.
 * Order       Sums are taken in a fixed order: the same call gives the same
 *             bits.  Every call can be captured into a graph.
 *
 * lse[t] = log sum_v exp(z_tv / temperature) (temperature 1 for cross entropy).
 * summary (NULL, or three floats): the sum of the losses, their mean over the
 * rows that count, and 1 / the number of those rows; 0, 0 and 1 if none does.
 *
 * Backward: dX (T×D, lddx >= D) and dW (V×D, lddw >= D) = the gradients of
 * sum_t g_t·loss_t, with g_t = grad_loss[t·grad_step]·grad_weight[0]
 * (grad_step 0: one value for every row; grad_weight NULL: 1; `summary + 2`
 * there gives the gradient of the mean).  Either of dX and dW may be NULL and
 * is then not computed.  lse and student are those of the forward call.
 */

/* Bytes of workspace of a forward (backward_pass 0) or backward (1) call with
 * these arguments; teacher_k: K, or 0 for cross entropy.  0 if T is 0 or the
 * arguments are refused. */
size_t tgemm_linear_loss_workspace_size(tgemm_dtype_t dtype, int64_t T, int64_t V, int64_t D,
                                        const void *X, int64_t ldx,
                                        const void *W, int64_t ldw,
                                        int64_t teacher_k, int backward_pass);

/* Softmax cross entropy: loss[t] = lse[t] - z_t,target[t]. */
tgemm_status_t tgemm_linear_ce_forward(tgemm_dtype_t dtype, int64_t T, int64_t V, int64_t D,
                                       const void *X, int64_t ldx,
                                       const void *W, int64_t ldw,
                                       const int64_t *target, int64_t ignore_index,
                                       float *loss, float *lse, float *logits, int64_t ldz, float *summary,
                                       void *workspace, size_t workspace_bytes, hipStream_t stream);

tgemm_status_t tgemm_linear_ce_backward(tgemm_dtype_t dtype, int64_t T, int64_t V, int64_t D,
                                        const void *X, int64_t ldx,
                                        const void *W, int64_t ldw,
                                        const int64_t *target, int64_t ignore_index,
                                        const float *lse, const float *logits, int64_t ldz,
                                        const float *grad_loss, int64_t grad_step, const float *grad_weight,
                                        void *dX, int64_t lddx, void *dW, int64_t lddw,
                                        void *workspace, size_t workspace_bytes, hipStream_t stream);

/*
 * Distillation from a teacher's top logits.  teacher_ids (T×K, leading
 * dimension ld_ids >= K) and teacher_logits (T×K of teacher_dtype, ld_logits
 * >= K) hold a row's K words and the teacher's logits of them; an entry with
 * the logit -infinity is absent, whatever its id.  With q_t the softmax of the
 * row's logits / temperature over its entries (an id that comes twice is
 * two entries), and z the student's logits / temperature,
 *   loss[t] = temperature²·sum_k q_tk·(log q_tk - (z_t,id - lse[t])),
 * the Kullback-Leibler divergence from the student's whole vocabulary to q.
 * student[t·K + k] receives z_t,id (0 for an absent entry).
 */
tgemm_status_t tgemm_linear_kd_forward(tgemm_dtype_t dtype, int64_t T, int64_t V, int64_t D,
                                       const void *X, int64_t ldx,
                                       const void *W, int64_t ldw,
                                       int64_t K, const int64_t *teacher_ids, int64_t ld_ids,
                                       tgemm_dtype_t teacher_dtype, const void *teacher_logits, int64_t ld_logits,
                                       float temperature,
                                       float *loss, float *lse, float *student,
                                       float *logits, int64_t ldz, float *summary,
                                       void *workspace, size_t workspace_bytes, hipStream_t stream);

tgemm_status_t tgemm_linear_kd_backward(tgemm_dtype_t dtype, int64_t T, int64_t V, int64_t D,
                                        const void *X, int64_t ldx,
                                        const void *W, int64_t ldw,
                                        int64_t K, const int64_t *teacher_ids, int64_t ld_ids,
                                        tgemm_dtype_t teacher_dtype, const void *teacher_logits, int64_t ld_logits,
                                        float temperature,
                                        const float *lse, const float *student, const float *logits, int64_t ldz,
                                        const float *grad_loss, int64_t grad_step, const float *grad_weight,
                                        void *dX, int64_t lddx, void *dW, int64_t lddw,
                                        void *workspace, size_t workspace_bytes, hipStream_t stream);

/*
 * Low-rank adapters of many requests beside a shared projection
 * -------------------------------------------------------------
 *   y_t = x_t·Wᵀ + scales[i]·(x_t·A_iᵀ)·B_iᵀ,   i = ids[t]
 * X (T×D) holds a row a token, W (N×D) the shared weight, A (`count` matrices
 * of rank×D, rows lda >= D apart, stride_a elements from one to the next) and B
 * (count × N×rank, ldb >= rank, stride_b) the adapters, ids (T) each token's
 * adapter, -1 for none, in any order, and scales (count floats, or NULL for 1)
 * their factors.  Y is T×N, ldy >= N.
 *
 * Types       float32, bf16 or fp16: X, W, A, B, Y and the gradients alike.
 *             Products of 16-bit values are exact and summed in float32, those
 *             of float32 ones by the planes of the loss operators or, where
 *             that is faster, in float32 (few rows, few tiles, the adapters'
 *             part).  x·Aᵀ is float32; where it meets 16-bit matrices in more
 *             than 64 rows it is held in two bf16 numbers (17 bits).  A result
 *             is rounded once.
 * Sizes       0 <= T < 2^24, 1 <= N, D <= 2^22, 1 <= count < 2^15, 1 <= rank <=
 *             1024, lda up to 2^26, the other leading dimensions and strides up
 *             to 2^40; larger ones, a product of 2^31 tiles and more, and an
 *             unknown dtype: TGEMM_ERROR_NOT_SUPPORTED.
 * hidden      T×rank floats, or NULL: the forward call leaves x_t·A_iᵀ there
 *             (rows without an adapter are not written) for the backward call,
 *             which takes NULL to form it again.
 * Workspace   As the loss operators'; tgemm_linear_adapters_workspace_size for
 *             the same arguments: need 0 for a forward call, otherwise the sum
 *             of 1 (dX), 2 (dW), 4 (dA) and 8 (dB) of a backward call, with its
 *             dY.  Up to 64 rows of a forward call take little; float32
 *             operands take their planes, 16-bit ones a copy where they cannot
 *             be read as they are stored.
 * Errors      As above, before anything is queued; also
 *             TGEMM_ERROR_INVALID_VALUE for an output that overlaps an input or
 *             another output, or whose matrices overlap one another.
 * Indices     An id other than -1 outside [0, count) is never used as an
 *             address: its row of Y and of dX is NaN, and dA and dB have
 *             nothing of it.
 * Rows        What one adapter holds, infinities and NaN too, reaches the rows
 *             of its own tokens alone.  An infinity may come out as NaN in the
 *             values that it reaches.
 * Order       Sums are taken in a fixed order: the same call gives the same
 *             bits.  Every call can be captured into a graph.
 *
 * Backward: for the gradient dY of Y (T×N, lddy >= N), with h_t = x_t·A_iᵀ and
 * u_t = dy_t·B_i,
 *   dx_t = dy_t·W + scales[i]·u_t·A_i        dW = dYᵀ·X
 *   dA_i = scales[i]·sum u_tᵀ·x_t            dB_i = scales[i]·sum dy_tᵀ·h_t
 * over the adapter's tokens; an adapter without tokens gets zeros.  Any of the
 * four may be NULL and is then not computed.  u_t is float32, held as above for
 * dX and in two bf16 numbers for dA, as h_t for dB.
 */
tgemm_status_t tgemm_linear_adapters_forward(tgemm_dtype_t dtype, int64_t T, int64_t N, int64_t D,
                                             const void *X, int64_t ldx,
                                             const void *W, int64_t ldw,
                                             int64_t count, int64_t rank,
                                             const void *A, int64_t lda, int64_t stride_a,
                                             const void *B, int64_t ldb, int64_t stride_b,
                                             const int64_t *ids, const float *scales,
                                             void *Y, int64_t ldy, float *hidden,
                                             void *workspace, size_t workspace_bytes, hipStream_t stream);

tgemm_status_t tgemm_linear_adapters_backward(tgemm_dtype_t dtype, int64_t T, int64_t N, int64_t D,
                                              const void *X, int64_t ldx,
                                              const void *W, int64_t ldw,
                                              int64_t count, int64_t rank,
                                              const void *A, int64_t lda, int64_t stride_a,
                                              const void *B, int64_t ldb, int64_t stride_b,
                                              const int64_t *ids, const float *scales,
                                              const float *hidden, const void *dY, int64_t lddy,
                                              void *dX, int64_t lddx, void *dW, int64_t lddw,
                                              void *dA, int64_t ldda, int64_t stride_da,
                                              void *dB, int64_t lddb, int64_t stride_db,
                                              void *workspace, size_t workspace_bytes, hipStream_t stream);

size_t tgemm_linear_adapters_workspace_size(tgemm_dtype_t dtype, int64_t T, int64_t N, int64_t D,
                                            const void *X, int64_t ldx,
                                            const void *W, int64_t ldw,
                                            int64_t count, int64_t rank,
                                            const void *dY, int64_t lddy, int need);

/*
 * An update made orthogonal by Newton-Schulz products
 * ---------------------------------------------------
 * For each of `batch` matrices G (M×N, rows ldg >= N apart, stride_g >= 0
 * elements from one matrix to the next), in place of G the result of
 *   X = G / (|G| + eps),                       |G| the root of the sum of squares
 *   steps times:  S = X·Xᵀ,  X <- a·X + (b·S + c·S·S)·X
 * is written to out (rows ldo >= N apart, matrices stride_out apart, which do
 * not overlap).  Where M > N, S = Xᵀ·X stands on the other side, which is the
 * same on the transpose.  With the coefficients 3.4445, -4.7750, 2.0315 five
 * steps bring the singular values of G to between 0.7 and 1.2 and leave its
 * singular vectors as they are, as the Muon optimiser takes its updates.
 *
 * Types       float32, bf16 or fp16, G and out alike.
 * Arithmetic  Where the smaller side is at most 64 the iteration runs on G·Gᵀ in
 *             float64.  Otherwise X, S and b·S + c·S·S are held in two fp16
 *             planes (22 bits, and no finer than 2^-35 of 1), every product is
 *             three of planes, summed in float32, and |G| is summed in float64:
 *             results of all types are as close as a chain of float32 products
 *             before their own rounding.  (Where a relative change of X changes
 *             the result f times as much, up to about f·2^-22 besides: f is 1 to
 *             a few hundred, but tens of thousands where coefficients without a
 *             margin meet a singular value at the end of their range.)  Entries
 *             of X, S, b·S + c·S·S or, where a lies within -16 ... 16, a·I + b·S +
 *             c·S·S beyond 60 overflow there, which coefficients that let
 *             singular values grow can come to (a itself may be of any size).
 * coefficients  3·steps floats in host memory: a, b, c of each step.
 * Sizes       0 <= batch <= 65535, M and N up to 2^20, 1 <= steps <= 32,
 *             leading dimensions and strides up to 2^40; larger ones, batches
 *             of 2^31 tiles and more, and an unknown dtype:
 *             TGEMM_ERROR_NOT_SUPPORTED.  Nothing is written if batch, M or N
 *             is 0.
 * Workspace   Device memory of the caller, 16-byte aligned, at least
 *             tgemm_orthogonalize_workspace_size(...) bytes, overlapping
 *             neither G nor out: up to 64 on the smaller side little, otherwise
 *             about 8·M·N + 8·min(M,N)² a matrix with M and N in whole 64s
 *             (4·M·N for a single step) and, for the whole call, the parts of
 *             sums that are split, which that function alone tells (up to 4 MB
 *             for a matrix of 300×1000, 0.1 GB for many large ones).  Its
 *             contents on entry do not matter.
 *             Two calls in flight at once need two.
 * Errors      As above, before anything is queued; also
 *             TGEMM_ERROR_INVALID_VALUE for an eps that is negative or not
 *             finite, missing coefficients, and an out that overlaps G or
 *             whose matrices overlap one another.
 * Values      A matrix of zeros gives zeros (NaN with an eps of 0); one that
 *             holds an infinity or NaN gives NaN everywhere.
 * Order       Sums are taken in a fixed order: the same call gives the same
 *             bits.  Every call can be captured into a graph.
 */
tgemm_status_t tgemm_orthogonalize(tgemm_dtype_t dtype, int64_t batch, int64_t M, int64_t N,
                                   const void *G, int64_t ldg, int64_t stride_g,
                                   int steps, const float *coefficients, float eps,
                                   void *out, int64_t ldo, int64_t stride_out,
                                   void *workspace, size_t workspace_bytes, hipStream_t stream);

/* Bytes of workspace of that call; 0 if batch, M or N is 0 or the arguments are refused. */
size_t tgemm_orthogonalize_workspace_size(tgemm_dtype_t dtype, int64_t batch, int64_t M, int64_t N, int steps);

/* Static, human-readable text for a status code. */
const char *tgemm_status_string(tgemm_status_t status);

/* Library version, major*10000 + minor*100 + patch. */
int tgemm_version(void);

#ifdef __cplusplus
}
#endif

#endif /* TGEMM_H */
