// Internal interface of the Newton-Schulz operator (orthogonalize.cpp: entry
// points; orthogonalize_product.hip: the chain of products;
// orthogonalize_small.hip: norms, planes, and the float64 form for a small
// side).  Every launcher takes validated arguments and returns the launch's
// hipError_t.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "tgemm.h"
#include "tile_walk.h"

namespace tgemm {
namespace ortho {

// ---- the chain of products -------------------------------------------------

// X, S = X·Xᵀ and Q = b·S + c·S² (+ a·I) are held as 2^kShift times their values
// in two fp16 planes (high, low: 22 bits, down to 2^-35 of 1), which overflow
// past 64.  With the coefficients 3.4445, -4.7750, 2.0315 singular values stay
// below 1.21, entries of X and S thus below 1.5 and those of Q below 2.9 without
// a·I (the polynomial's least value on [0, 1.5] is -2.81) and 3.45 with it.
constexpr int kShift = 10;

// Operands of a batch of products.  Two planes an operand; the three segments are
// (low, high), (high, low), (high, high).  lower: tiles on
// and below the diagonal only (square tiles).  The batch's tiles, matrix by
// matrix, are numbered through; a launch takes `count` of them from `from` on,
// each with its sum in `splits` parts.  What the epilogue is told as the part
// is the tile's number times splits and its part.
struct Chain : m16::Operands {
    int64_t batch_a, batch_b;  // elements between the matrices
    bool lower;
    int from, count;

    TGEMM_BOTH int tiles() const { return lower ? tiles_m * (tiles_m + 1) / 2 : tiles_m * tiles_n; }
    TGEMM_BOTH int ids() const { return count * splits; }
    // the row and column of tile `at` of a matrix
    TGEMM_BOTH void spot(int at, int &tm, int &tn) const
    {
        if (!lower) {
            const int per_group = 8 * tiles_n, group = at / per_group, in_group = at - group * per_group;
            const int rows = m16::least(tiles_m - group * 8, 8);
            tm = group * 8 + in_group % rows;
            tn = in_group / rows;
            return;
        }
        // groups of 8 rows of tiles: a rectangle, column by column, and the
        // triangle at its end, row by row
        int group = 0, rows = m16::least(tiles_m, 8), size = rows * (rows + 1) / 2;
        while (at >= size) {
            at -= size;
            ++group;
            rows = m16::least(tiles_m - group * 8, 8);
            size = rows * 8 * group + rows * (rows + 1) / 2;
        }
        tm = 8 * group;
        tn = 0;
        if (at < rows * 8 * group) {
            tm += at % rows;
            tn = at / rows;
        } else {
            at -= rows * 8 * group;
            int r = 0;
            while (at > r) at -= ++r;
            tm += r;
            tn = 8 * group + at;
        }
    }
    template <int BM, int BN>
    TGEMM_BOTH void tile(int id, int &m0, int &n0, int &split, int &first, int &last) const
    {
        // parts of a tile share nothing; neighbours share rows and columns
        const int logical = m16::deal(id, ids()), part = logical / count, number = from + logical - part * count;
        int tm, tn;
        spot(number % tiles(), tm, tn);
        m0 = tm * BM;
        n0 = tn * BN;
        split = number * splits + part;
        first = part * steps_per_split;
        last = m16::least(steps, first + steps_per_split);
    }
    TGEMM_BOTH int64_t plane_at_a(int seg) const { return seg == 0 ? plane_a : 0; }
    TGEMM_BOTH int64_t plane_at_b(int seg) const { return seg == 1 ? plane_b : 0; }
    TGEMM_BOTH int matrix(int split) const { return split / splits / tiles(); }
    TGEMM_BOTH int64_t start_a(int split) const { return matrix(split) * batch_a; }
    TGEMM_BOTH int64_t start_b(int split) const { return matrix(split) * batch_b; }
};

// Tile configurations: index, rows and columns, wavefronts along them.
#define TGEMM_CHAIN_TILES(X) X(0, 256, 256, 2, 4) X(1, 128, 128, 2, 2) X(2, 64, 64, 2, 2)
struct TileShape {
    int side, wg_per_cu;
};
constexpr TileShape kTiles[] = {{256, 1}, {128, 2}, {64, 4}};
constexpr int kTileCount = 3;

// alpha·add + beta·(the product) + diagonal·I, as planes or as the result.
struct ChainArgs {
    Chain op;
    float alpha, beta, diagonal;
    const void *add;            // planes, or NULL
    int64_t ld_add, plane_add, batch_add;
    void *planes;               // or NULL: rows × ldo of each plane are written, zero past M and N
    int64_t ldo, plane_out, batch_out;
    int rows;
    void *result;               // M×N, rows ldr apart
    int64_t ldr, batch_r;
    tgemm_dtype_t dtype;
    // Room for the parts of split sums, tile by tile and part by part: the launch
    // leaves the products there, and launch_join does the rest.
    float *parts;
};
// How A and B lie: both with K along their rows, both along their columns, or A along its rows and B not.
enum Order { kRows, kColumns, kMixed };
hipError_t launch_chain(Order order, int tile, const ChainArgs &a, hipStream_t stream);
hipError_t launch_join(int tile, const ChainArgs &a, hipStream_t stream);

// ---- passes over G ---------------------------------------------------------

// Partial sums of squares of a matrix, and its planes: 2^kShift·G / (|G| + eps),
// zero past the ends of the rows and columns that are written.
constexpr int kMaxSquares = 512;
struct SplitArgs {
    const void *G;
    int64_t ld, batch_g;
    tgemm_dtype_t dtype;
    int batch;
    int64_t rows, cols;
    double *squares;  // batch × parts
    int parts;
    float eps;
    void *planes;
    int64_t rows_out, ldo, plane, batch_out;
};
hipError_t launch_squares(const SplitArgs &a, hipStream_t stream);
hipError_t launch_split(const SplitArgs &a, hipStream_t stream);

// ---- one side of at most kSmallSide ----------------------------------------

// S = G·Gᵀ (of the small side) in parts, the iteration on S, and its result times G, all in float64.
constexpr int kSmallSide = 64, kMaxSteps = 32;
struct SmallArgs {
    const void *G;
    int64_t ld, batch_g;
    tgemm_dtype_t dtype;
    int batch, side;   // side ≤ kSmallSide
    int64_t length;
    bool tall;         // the small side lies along the rows
    double *grams;     // batch × parts × (blocks of 16×16, lower ones) of 256
    int64_t part_length;
    int parts;
    int steps;
    float coefficients[3 * kMaxSteps];
    float eps;
    double *factor;    // batch × (16·blocks)²
    void *out;
    int64_t ldo, batch_o;
};
inline int blocks_of(int side) { return side <= 16 ? 1 : side <= 32 ? 2 : 4; }
hipError_t launch_grams(const SmallArgs &a, hipStream_t stream);
hipError_t launch_iterate(const SmallArgs &a, hipStream_t stream);
hipError_t launch_apply(const SmallArgs &a, hipStream_t stream);

}  // namespace ortho
}  // namespace tgemm
