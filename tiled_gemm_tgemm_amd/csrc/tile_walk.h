// The way of a work-group's loads through its tiles of a 16-bit product
// (mfma16.h), and how an operand's slices lie in device memory and in LDS:
// arithmetic on addresses and nothing else, so that it also runs on the host,
// where tests follow every load.
//
// An operand is K-contiguous ("KC": element (mn, k) at mn·ld + k) or
// MN-contiguous ("MC": at k·ld + mn).  A KC slice lies in LDS as mn rows of
// 128 bytes, an MC slice as 64 rows (one a k) of 2·BM or 2·BN bytes, from
// which the transposing LDS read gathers four values of k a lane.  The loads
// into LDS write 16-byte pieces in lane order, so the pieces are permuted on
// the reading side of device memory, within a row: piece c of a KC row goes to
// c ^ (row / 2 & 7), piece c of an MC row to c ^ flip(k).  Without that the 16
// rows of a KC fragment would start in the same banks, as would the rows of a
// transposing read.
#pragma once

#include <stdint.h>

#if defined(__HIP__)
#include <hip/hip_runtime.h>
#define TGEMM_BOTH __host__ __device__ __forceinline__
#else
#define TGEMM_BOTH inline
#endif

namespace tgemm {
namespace m16 {

constexpr int kStepK = 64;
constexpr int kXcds = 8;

TGEMM_BOTH constexpr int least(int a, int b) { return a < b ? a : b; }

// The operands of a product.  Rows and columns past the ends are read from
// the last one that exists (their products are not stored, or meet zeros).
struct Operands {
    const void *A, *B;
    int64_t lda, ldb;          // elements
    int64_t plane_a, plane_b;  // elements between the planes of a split operand
    int segments;              // 1; 6: the plane pairs of kPairs; 2: the first two, with plane_b = 0
    int M, N;
    int steps;                 // steps of 64 along K
    int steps_per_split;       // part y of the sum takes steps [y·this, (y+1)·this)
    int mn_a, mn_b;            // KC: rows of A / B; MC: columns that may be read, a multiple of 8
    int k_a, k_b;              // values of k of A / B; a multiple of 8 for a KC operand, of 64 for A
    int tiles_m, tiles_n, splits;
};

// A float32 operand is the sum of three bf16 planes (high, middle, low: 24
// bits).  Of the nine products of planes the six that reach 2^-24 of the
// largest are summed, small ones first: (mid,mid), (high,low), (low,high),
// (high,mid), (mid,high), (high,high); two bits a plane.  The first two also
// serve an A of two planes and a B of one: (low of the two, B), (high, B).
constexpr int kPairsA = (1 << 0) | (0 << 2) | (2 << 4) | (0 << 6) | (1 << 8) | (0 << 10);
constexpr int kPairsB = (1 << 0) | (2 << 2) | (0 << 4) | (1 << 6) | (0 << 8) | (0 << 10);

// The exchange of 16-byte pieces in LDS.  A KC read takes 16 rows at a time,
// which lie 128 bytes apart: two rows share a position in the 256 bytes that
// the banks are wide, eight pairs are told apart by their pieces.  An MC read
// takes four (two times four) rows of 2·MN bytes at a time: 32 adjacent bytes
// of each, or, where a block's columns are 4·F apart (PERMUTE), four pieces.
TGEMM_BOTH constexpr int swizzle(int row) { return (row >> 1) & 7; }
template <int MN, int F, bool PERMUTE>
TGEMM_BOTH constexpr int flip(int k)
{
    const int j = k & 3, h = (k >> 3) & 1;
    if (PERMUTE) return F == 4 ? (j & 1) | (j >> 1) << 3 : 4 * j;
    return MN >= 128 ? 2 * j + 8 * h : 0;
}

// An operand's slices of a step.  F: the blocks of 16 that a wavefront takes.
template <int MN, int F, int THREADS, bool MC, bool PERMUTE>
struct Slice {
    static constexpr int kThreads = THREADS;
    static constexpr int kBytes = MN * kStepK * 2;
    static constexpr int kRounds = kBytes / 16 / THREADS;
    static_assert(kRounds * 16 * THREADS == kBytes, "whole rounds");
    static constexpr int kRowPieces = MC ? MN / 8 : kStepK / 8;

    // Byte offset, from the step's first row and column, of the piece that
    // goes to 16-byte position `position` of the slice.  mn_last: the last row
    // (KC) or the last 8-aligned column (MC) of the operand, relative to the
    // tile; k_last: the last row of an MC operand or the last 8-aligned column
    // of a KC one, relative to the step.  Past it an MC operand's last row
    // stands in, and a KC operand's first columns of the step: they meet zeros
    // of the other operand.
    static TGEMM_BOTH uint32_t offset(int position, int64_t ld, int mn_last, int k_last)
    {
        const int row = position / kRowPieces, slot = position % kRowPieces;
        if (MC) {
            const int mn = least((slot ^ flip<MN, F, PERMUTE>(row)) * 8, mn_last);
            return ((uint32_t)least(row, k_last) * (uint32_t)ld + (uint32_t)mn) * 2u;
        }
        int mn = row;
        if (PERMUTE) {
            const int in = row % (16 * F), b = in / 16, q = in / 4 % 4;
            mn = row - in + 4 * F * q + 4 * b + in % 4;
        }
        const int k = (slot ^ swizzle(row)) * 8;
        return ((uint32_t)least(mn, mn_last) * (uint32_t)ld + (uint32_t)(k <= k_last ? k : 0)) * 2u;
    }
};

// Tile `id` of `ids`.  The hardware deals work-groups, and a grid that is a
// multiple of 8 its tiles, round-robin to eight XCDs with an L2 each; XCD x
// takes the x-th run of logical ids.  Ids walk the tiles of one part of the
// sum, then those of the next (parts share nothing), and within a part groups
// of 8 tile rows column by column, so that the work-groups of an XCD share
// rows of A and columns of B.
TGEMM_BOTH void place_tile(int id, int ids, int tiles_m, int tiles_n, int &tm, int &tn, int &split)
{
    const int q = ids / kXcds, r = ids % kXcds;
    const int x = id % kXcds;
    const int logical = id / kXcds + x * q + least(x, r);
    const int tiles = tiles_m * tiles_n;
    split = logical / tiles;
    const int tile = logical - split * tiles, per_group = 8 * tiles_n;
    const int group = tile / per_group, in_group = tile - group * per_group;
    const int rows = least(tiles_m - group * 8, 8);
    tm = group * 8 + in_group % rows;
    tn = in_group / rows;
}

// The place of tile `id` and its steps [first, last).
template <int BM, int BN>
TGEMM_BOTH void tile_at(const Operands &p, int id, int &m0, int &n0, int &split, int &first, int &last)
{
    int tm, tn;
    place_tile(id, p.tiles_m * p.tiles_n * p.splits, p.tiles_m, p.tiles_n, tm, tn, split);
    m0 = tm * BM;
    n0 = tn * BN;
    first = split * p.steps_per_split;
    last = least(p.steps, first + p.steps_per_split);
}

// Which tile, segment and step the loads are at, and where from.
template <int BM, int BN, bool A_MC, bool B_MC>
struct Walk {
    int id, seg, k, first, last;  // k: the step to come
    int a_last, b_last, a_k_last, b_k_last;  // as Slice::offset takes them
    const char *a, *b;                       // the tile's first rows (KC) or columns (MC)
    const char *from_a, *from_b;             // the step's slices

    TGEMM_BOTH void open(const Operands &p)
    {
        int m0, n0, split;
        tile_at<BM, BN>(p, id, m0, n0, split, first, last);
        // a tile may lie past an operand's last row: it takes that one
        const int a_end = p.mn_a - (A_MC ? 8 : 1), b_end = p.mn_b - (B_MC ? 8 : 1);
        const int a0 = least(m0, a_end), b0 = least(n0, b_end);
        a_last = a_end - a0;
        b_last = b_end - b0;
        a = (const char *)p.A + (A_MC ? (int64_t)a0 : (int64_t)a0 * p.lda) * 2;
        b = (const char *)p.B + (B_MC ? (int64_t)b0 : (int64_t)b0 * p.ldb) * 2;
        seg = 0;
        k = first;
        fresh = true;
    }

    TGEMM_BOTH void begin(const Operands &p, int first_id)
    {
        id = first_id;
        open(p);
    }

    // On to the next step's slices.  What it tells: whether the offsets within
    // A's and B's are other ones now (a new tile, the end of an operand, the
    // start of the next segment after such an end).
    struct Moved {
        bool a, b;
    };
    TGEMM_BOTH Moved seek(const Operands &p, int stride)
    {
        if (k == last) {
            k = first;
            if (++seg == p.segments) {
                // after the last tile its first steps are loaded again, for nobody
                if (id + stride < p.tiles_m * p.tiles_n * p.splits) id += stride;
                open(p);
            }
        }
        const int start_a = A_MC ? least(k * kStepK, p.k_a - 1) : k * kStepK;
        const int start_b = B_MC ? least(k * kStepK, p.k_b - 1) : k * kStepK;
        from_a = a + (A_MC ? start_a * p.lda : (int64_t)start_a) * 2;
        from_b = b + (B_MC ? start_b * p.ldb : (int64_t)start_b) * 2;
        if (p.segments > 1) {
            from_a += ((kPairsA >> (2 * seg)) & 3) * p.plane_a * 2;
            from_b += ((kPairsB >> (2 * seg)) & 3) * p.plane_b * 2;
        }
        a_k_last = A_MC ? p.k_a - 1 - start_a : kStepK;  // a KC A has whole steps
        b_k_last = p.k_b - (B_MC ? 1 : 8) - start_b;
        const bool again = p.segments > 1 && k == first;
        const Moved moved{fresh || (A_MC && (again || (k + 1) * kStepK > p.k_a)),
                          fresh || (B_MC && again) || (k + 1) * kStepK > p.k_b};
        fresh = false;
        ++k;
        return moved;
    }

private:
    bool fresh;  // nothing of this tile has been asked for yet
};

}  // namespace m16
}  // namespace tgemm
