// Internal interface of the loss operators on an output head's product
// (linear_loss.cpp: entry points; linear_loss_product.hip: the products;
// linear_loss_rows.hip: passes over rows).  Every launcher takes validated
// arguments and returns the launch's hipError_t.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "tgemm.h"
#include "tile_walk.h"

namespace tgemm {
namespace loss {

// A fp16 gradient piece holds 2^15 times its value over the row's power of
// two (bf16 and float32 have the range to hold the value itself).
constexpr int kHalfShift = 15;

// ---- the products ----------------------------------------------------------

// Tile configurations: index, rows and columns, wavefronts along them.
#define TGEMM_TILES(X) X(0, 256, 256, 2, 4) X(1, 128, 128, 2, 2) X(2, 32, 128, 1, 4)
struct TileShape {
    int bm, bn;
    int wg_per_cu;
    int stat_columns;  // columns a wavefront's partial (maximum, sum) covers
};
constexpr TileShape kTiles[] = {{256, 256, 1, 64}, {128, 128, 2, 64}, {32, 128, 3, 32}};
constexpr int kTileCount = 3;

// Partial softmax statistics of s·X·Wᵀ: part[t][g] = (maximum, sum of
// exp2(· - maximum)) of row t's columns of group g, in units of log2;
// picked[t] = the scaled logit at target[t] (rows whose target is in [0, V)).
struct StatsArgs {
    m16::Operands op;
    float scale;
    float2 *part;
    int groups;
    const int64_t *target;  // or NULL
    float *picked;
    // a teacher's entries (linear_sort_kernel), or NULL: row t's entries in
    // column group g are list[t·K + starts[t·(groups + 1) + g]] ... up to
    // those of g + 1, each the column in its group and 256·k; student[t·K + k]
    // receives the scaled logit
    const uint16_t *starts;
    const uint32_t *list;
    int K;
    float *student;
    float *logits;  // or NULL: the products, before the scale, rows ldz apart
    int64_t ldz;
};
hipError_t launch_stats(bool half, int tile, const StatsArgs &a, hipStream_t stream);

// launch_stats for at most kFewRows rows, on operands however they are stored;
// column groups of 16 or 64 (few_columns).  A compute unit gets no more than
// about 22 GB/s of W from memory however many wavefronts ask for it, so words
// are dealt 16 at a time where 64 at a time leave compute units without any:
// one row of 4000×4096 bf16 11 against 25 µs, of 16000×4096 26 against 28, of
// 32000×4096 46 against 44, of 65536×1024 29 against 26 (the same W call after
// call; on others in turn the one that is taken needs 13, 31, 57 and 31).
constexpr int64_t kFewRows = 32, kFewBelow = 16384;
inline int few_columns(int64_t V) { return V < kFewBelow ? 16 : 64; }
hipError_t launch_stats_few(const StatsArgs &a, tgemm_dtype_t dtype, int columns, int D, hipStream_t stream);

// A piece of the logits' gradient: G[t][v - v0] = coef[t]·(exp(s·z - lse[t]) -
// [v = target[t]]), zero past the ends, 16-bit: one plane, or two or three that
// add up to it.
struct GradArgs {
    m16::Operands op;
    float scale;
    const float *lse, *coef;
    const int64_t *target;  // or NULL
    int64_t v0;
    int rows;               // rows to write (T rounded up to 64)
    void *G;
    int64_t ldg, plane;     // elements
    int planes;
};
hipError_t launch_grad(bool half, int tile, const GradArgs &a, hipStream_t stream);

// The same from the products that launch_stats kept: a.op is not used but for
// M (T) and N (columns), and a.rows rows of whole 64 columns are written.
hipError_t launch_grad_kept(bool half, const GradArgs &a, const float *logits, int64_t ldz, hipStream_t stream);

// C = A·B with A = G as stored (dX) or transposed (dW), B MN-contiguous.
struct OutArgs {
    m16::Operands op;
    void *out;
    int64_t ldo;
    tgemm_dtype_t dtype;
    bool add;                // float32 out: add to what is there
    int64_t split_stride;    // elements between the outputs of the sum's parts
    int period = 0, kept = INT32_MAX;  // of every `period` rows (a power of two; 0: one run) the first `kept` are stored
    const float *row_scale, *all_scale;  // as SumArgs
};
hipError_t launch_dx(bool half, int tile, const OutArgs &a, hipStream_t stream);
hipError_t launch_dw(bool half, int tile, const OutArgs &a, hipStream_t stream);

// ---- passes over rows ------------------------------------------------------

// The teacher's part of a row, as both passes read it.
struct Teacher {
    int K;
    const int64_t *ids;
    int64_t ld_ids;
    const void *logits;
    int64_t ld_logits;
    tgemm_dtype_t dtype;
    float scale;  // 1 / temperature
};

// Sorts each row's entries by column group for launch_stats, and sets student to 0
// where an entry is absent and NaN where its id is out of range.
struct SortArgs {
    int64_t T, V;
    int groups, columns;  // column groups, and the columns of one
    Teacher teacher;
    uint16_t *starts;
    uint32_t *list;
    float *student;
};
hipError_t launch_sort(const SortArgs &a, hipStream_t stream);

// summary (or NULL) = {sum of loss, the mean over the rows that count, 1 /
// their number} (1 / 1 where none does); `counted` is room for a flag a row.
struct JoinArgs {
    int64_t T, V;
    int groups;
    const float2 *part;
    const int64_t *target;
    int64_t ignore;
    const float *picked;
    const Teacher *teacher;  // host pointer; NULL for cross entropy
    const float *student;
    float *loss, *lse, *summary;
    int *counted;
};
hipError_t launch_join(const JoinArgs &a, hipStream_t stream);
// The summary of no rows.
hipError_t launch_summary_none(float *summary, hipStream_t stream);

// The factor c_t = grad[t·grad_step]·factor·*weight of a row's gradient, in two
// parts: coef[t] multiplies the logits' gradient before it is rounded (0 for
// rows that do not count, NaN for rows with an index out of range), the scales
// multiply the results.
// * One value for all rows (grad_step 0): coef is 1 (fp16: 2^kHalfShift), and
//   row_scale[t] and all_scale[0] hold the rest, so that its rounding is not
//   that of every element.
// * Otherwise coef is c_t; for fp16 its fraction times 2^kHalfShift, with
//   row_scale[t] = 2^(exponent - kHalfShift), exps[t] the exponent, and
//   block_max[b] the largest over a work-group's kCoefRows rows of exponent +
//   that of the row's largest finite state (X, fp16).  launch_copy scales dW's
//   rows of X by their factors' powers of two, such that the largest product of
//   the two lies just below 2^kHalfShift, and writes all_scale: a row whose
//   factor is 2^-28 of the largest keeps the bits of its states.  (Scaled by
//   their factors relative to the largest, without regard to the states, rows
//   of N(0,1) lost bits from 2^-14 on and were 29% off at 2^-24.)
constexpr int kCoefRows = 16;
inline int64_t coef_blocks(int64_t T, bool /* a row of either loss takes a wavefront */)
{
    return (T + kCoefRows - 1) / kCoefRows;
}
struct CoefArgs {
    int64_t T, V;
    const float *grad;
    int64_t grad_step;
    float factor;
    const float *weight;  // or NULL
    const int64_t *target;
    int64_t ignore;
    const Teacher *teacher;
    bool half;
    float *coef, *row_scale, *all_scale;
    int *exps, *block_max;
    const void *X;  // T×D, rows ldx apart
    int64_t ldx, D;
};
hipError_t launch_coef(const CoefArgs &a, hipStream_t stream);

// Cross entropy's factors need no pass of their own, but for fp16 with a factor
// a row, where the largest exponent has to be known first.
inline bool coef_in_copy(const CoefArgs &a) { return a.teacher == nullptr && (!a.half || a.grad_step == 0); }

// dst (planes of rows_out×ld_out 16-bit elements, zero past the ends) = src
// (rows×cols).  coef: rows with coef 0 become zero.  exps: row t is scaled by
// 2^(kHalfShift + exps[t] - the largest of block_max), if it has an exponent,
// and all_scale receives 2^(that - 2·kHalfShift).
struct CopyArgs {
    const void *src;
    int64_t ld;
    tgemm_dtype_t dtype;
    int64_t rows, cols;
    void *dst;
    int64_t rows_out, ld_out, plane;
    int planes;
    const float *coef;
    const int *exps, *block_max;
    int blocks;
    float *all_scale;
    const struct CoefArgs *make;  // host pointer, or NULL: also does launch_coef's work (coef_in_copy)
};
hipError_t launch_copy(const CopyArgs &a, hipStream_t stream);

// G[t][id - v0] = coef[t]·(exp(student - lse) - the teacher's probability of id) for the ids in [v0, v0 + cols).
struct ScatterArgs {
    int64_t T, v0, cols;
    Teacher teacher;
    const float *student, *lse, *coef;
    void *G;
    int64_t ldg, plane;
    int planes;
    bool half;
};
hipError_t launch_scatter(const ScatterArgs &a, hipStream_t stream);

// out[t][d] = scale·(part_0 + part_1 + ...)[t][d], part_s at part + s·stride,
// the scale row_scale[t], or all_scale[0], or 1 where both are NULL.
struct SumArgs {
    int64_t T, D;
    const float *part;
    int64_t ld, stride;
    int count;
    const float *row_scale, *all_scale;
    void *out;
    int64_t ldo;
    tgemm_dtype_t dtype;
};
hipError_t launch_sum(const SumArgs &a, hipStream_t stream);

// rows×cols elements of out = 0
hipError_t launch_zero(void *out, int64_t ldo, tgemm_dtype_t dtype, int64_t rows, int64_t cols, hipStream_t stream);

}  // namespace loss
}  // namespace tgemm
