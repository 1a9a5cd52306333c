// Internal interface of the projection with low-rank adapters
// (linear_adapters.cpp: entry points; linear_adapters_product.hip: the products
// with the weight; linear_adapters_rows.hip: the adapters' own sums).  Every
// launcher takes validated arguments and returns the launch's hipError_t.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "linear_loss.h"
#include "tgemm.h"
#include "tile_walk.h"

namespace tgemm {
namespace adapters {

// One of a stack of adapter matrices, as a product of few columns reads it:
// element (outer, rank) of adapter i lies at i·stride + outer·ld + rank
// (rank_inner, B's layout) or at i·stride + rank·ld + outer (A's layout).
struct Stack {
    const void *p;
    int64_t ld, stride;
    bool rank_inner;
    int count, rank;
};

// What the products read of a token's hidden values: scaled, and zero up to a
// rank of whole 32s; 16-bit operands: two bf16 planes one after the other (17
// bits), float32 ones: float32.
TGEMM_BOTH constexpr int64_t planes_rank(int64_t rank) { return (rank + 31) / 32 * 32; }

// hidden(t, rank) = sum over k of rows(t, k)·C_i(k, rank), i = ids[t], in `parts`
// parts of the sum (part p to part + p·T·rank).  One part is the whole: it goes
// to `part` if that is not NULL, and times scales[i] (NULL: 1) to `planes` if
// that is not.  Rows whose id is outside [0, count) are not written.
struct ShrinkArgs {
    tgemm_dtype_t dtype;
    int64_t T, K;
    const void *rows;
    int64_t ld;
    Stack c;
    const int64_t *ids;
    const float *scales;
    float *part;
    void *planes;
    int64_t part_k;  // values of k a part, a multiple of 256
    int parts, slots;
    int rows_each;   // 16: a work-group's wavefronts share 16 rows' sums; 64, 128: they take 16, 32 rows each
    // 16-bit rows and adapters 16-byte aligned, K in whole 64s, leading dimensions
    // below 2^22, the ranks not the inner ones, rows_each 64 and slots 1
    bool through_lds;
};
hipError_t launch_shrink(const ShrinkArgs &a, hipStream_t stream);
// Adds the parts up to `hidden` and `planes` (either may be NULL), for every row whose id is in range.
hipError_t launch_finish(const ShrinkArgs &a, float *hidden, void *planes, hipStream_t stream);

// What the products with the weight add to row t: scales[i]·hidden(t)·C_i.  A
// row whose id is neither -1 nor in range becomes NaN.  The few rows' kernel
// reads the parts of hidden, the tiles the planes.
struct Expand {
    const int64_t *ids;
    const float *scales;
    const float *hidden;
    int64_t part_stride;
    int parts;
    const void *planes;
    Stack c;
};

// C = A·B + the adapters' part (without where e.ids is NULL), A as stored along K, B along K (forward, with
// the adapters' ranks the inner ones) or not (dX).
struct ProductArgs {
    m16::Operands op;
    void *out;
    int64_t ldo;
    tgemm_dtype_t dtype;        // of out, or float32 where the sum is split
    tgemm_dtype_t stored;       // of the adapters
    int64_t split_stride;
    Expand e;
};
hipError_t launch_product(bool half, bool b_mc, int tile, const ProductArgs &a, hipStream_t stream);

// out = the sum of `count` parts + the adapters' part (with one part, out may be it).
struct AddArgs {
    int64_t T, N;
    const float *part;
    int64_t ld, stride;
    int count;
    void *out;
    int64_t ldo;
    tgemm_dtype_t dtype;
    Expand e;
};
hipError_t launch_add(const AddArgs &a, hipStream_t stream);

// The same for at most kFewRows rows, forward, on operands however they are stored.
constexpr int64_t kFewRows = 64;
struct FewArgs {
    tgemm_dtype_t dtype;
    int T, N, D;
    const void *X;
    int64_t ldx;
    const void *W;
    int64_t ldw;
    void *Y;
    int64_t ldy;
    Expand e;
    bool through_lds;  // 16-bit values, 16-byte aligned rows of whole steps of 64, ldx and ldw at most 2^22
};
hipError_t launch_few(const FewArgs &a, hipStream_t stream);

// ---- the adapters' gradients -----------------------------------------------

// Tokens in the order of their adapters: order[starts[i] ... starts[i + 1]) are
// adapter i's, ascending.  Then cut in chunks of at most `tokens`, once for
// each gradient: chunks[n] = {adapter, first place in order, tokens, slot}, the
// slot -1 where the adapter has one chunk; joins[i] = {first slot, chunks};
// *chunk_count of them.
// place: where the chunk's small values lie among the arranged ones, whole 64s.
struct Chunk {
    int adapter, first, tokens, slot;
    int64_t place;
};
constexpr int kMostTokens = 2048;  // of a chunk
struct Cut {
    int tokens;  // a multiple of 64, at most kMostTokens
    Chunk *chunks;
    int2 *joins;
    int *chunk_count;
};
struct GroupArgs {
    const int64_t *ids;
    int T, count;
    int *order, *starts;
    Cut cuts[2];
};
hipError_t launch_group(const GroupArgs &a, hipStream_t stream);
// Up to these one work-group does it next to the adapters' turn; the two launches
// that this spares take 10 µs.
constexpr int kAloneTokens = 8192, kAloneAdapters = 16;

// out_i = scales[i]·sum over adapter i's tokens of rows(t, :)ᵀ·small(t, :), laid
// out as the stack: out(outer, rank).  Adapters of several chunks leave those
// in part (slots × C × rank, as out but packed) for launch_join.
struct OuterArgs {
    tgemm_dtype_t dtype;
    int C;                    // columns of rows
    const void *rows;
    int64_t ld;
    const float *small;       // T × rank
    // small in the order of the chunks, or NULL: for each chunk rank rows of its
    // tokens in whole 64s, zero past them, high and low bf16 planes apart;
    // rows are then 16-bit, 16-byte aligned and of whole 8s
    void *arranged;
    int64_t arranged_plane;
    const float *scales;
    const int *order;
    Cut cut;
    int most_chunks;          // a launch's y
    float *part;
    void *out;
    int64_t ldo, stride_out;
    bool rank_inner;
    int count, rank;
};
constexpr int kOuterColumns = 128, kOuterTokens = 64;
// Both gradients' small values at once (either `out` may be NULL).
hipError_t launch_arrange(const OuterArgs &a, const OuterArgs &b, hipStream_t stream);
// a is A's (its ranks are not the inner ones), b is B's
hipError_t launch_outer(const OuterArgs &a, const OuterArgs &b, hipStream_t stream);
hipError_t launch_join(const OuterArgs &a, const OuterArgs &b, hipStream_t stream);

// Stacks the other way round: element (outer, rank) of adapter i, at i·to_stride
// + rank·to_ld + outer if the stack's ranks are the inner ones, otherwise at
// i·to_stride + outer·to_ld + rank.
struct TurnArgs {
    tgemm_dtype_t dtype;
    Stack from;
    int64_t outer;
    void *to;                 // or NULL: nothing to do
    int64_t to_ld, to_stride;
};
// Also does launch_group's work if `group` is not NULL.
hipError_t launch_turn(const TurnArgs &a, const TurnArgs &b, const GroupArgs *group, hipStream_t stream);

}  // namespace adapters
}  // namespace tgemm
