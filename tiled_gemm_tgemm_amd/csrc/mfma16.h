// Tiles of 16-bit products on the matrix cores: C = A·B with A M×K and B K×N
// of bf16 or fp16 values, summed in fp32 registers.
//
// * A work-group of WM×WN wavefronts computes BM×BN tiles of C, a wavefront
//   FM×FN blocks of 16×16 (v_mfma_f32_16x16x32).  The GPU runs these products
//   at the clock that its power allows, and this instruction needs less of it
//   than v_mfma_f32_32x32x16, which moves twice the accumulators for the same
//   work (from registers alone, random bf16: 2054 against 1834 TFLOP/s).
// * The blocks are formed transposed (B's fragment is the instruction's first
//   operand), so a lane holds values of one row of C: sums along a row stay
//   within a lane and the three that share its row, and a row's values leave
//   in 16-byte pieces.  The order of a wavefront's columns is free as long as
//   the reader of C knows it: column 4·FN·q + 4·b + r sits at index 4·q + r of
//   block b, which gives the lanes of quarter q 4·FN adjacent columns.
// * K runs in steps of 64.  A step's slices of A and B go from device memory
//   straight into LDS, 16 bytes a lane, into one of two stages; the loads of
//   the next step are under way while a step is multiplied.
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

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "mfma_common.h"

namespace tgemm {
namespace m16 {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

constexpr int kStepK = 64;

// The operands of a product.  Rows and columns past the ends are read from
// the last one that exists (their products are not stored, or meet zeros).
struct Operands {
    const void *A, *B;
    int64_t lda, ldb;          // elements
    int64_t plane_a, plane_b;  // elements between the planes of a split operand
    int segments;              // 1, or 6: the plane pairs of kPairs
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
// (high,mid), (mid,high), (high,high); two bits a plane.
constexpr int kPairsA = (1 << 0) | (0 << 2) | (2 << 4) | (0 << 6) | (1 << 8) | (0 << 10);
constexpr int kPairsB = (1 << 0) | (2 << 2) | (0 << 4) | (1 << 6) | (0 << 8) | (0 << 10);

// x = high + middle + low.  An infinity or NaN is all in the high part, and so
// is a value above 3.39e38, which rounds to infinity there.
__device__ __forceinline__ void split(float x, __bf16 &high, __bf16 &middle, __bf16 &low)
{
    high = (__bf16)x;
    float rest = x - (float)high;
    if (__builtin_isinf(rest) || __builtin_isnan(rest)) rest = 0.0f;
    middle = (__bf16)rest;
    low = (__bf16)(rest - (float)middle);
}

template <class E>
struct Frag;
template <>
struct Frag<__bf16> {
    typedef bf16x8 type;
    static __device__ __forceinline__ f32x4 mfma(bf16x8 a, bf16x8 b, f32x4 c)
    {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
    }
};
template <>
struct Frag<_Float16> {
    typedef f16x8 type;
    static __device__ __forceinline__ f32x4 mfma(f16x8 a, f16x8 b, f32x4 c)
    {
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
    }
};

// The exchange of 16-byte pieces in LDS.  A KC read takes 16 rows at a time,
// which lie 128 bytes apart: two rows share a position in the 256 bytes that
// the banks are wide, eight pairs are told apart by their pieces.  An MC read
// takes four (two times four) rows of 2·MN bytes at a time: 32 adjacent bytes
// of each, or, where a block's columns are 4·F apart (PERMUTE), four pieces.
__device__ __forceinline__ constexpr int swizzle(int row) { return (row >> 1) & 7; }
template <int MN, int F, bool PERMUTE>
__device__ __forceinline__ constexpr int flip(int k)
{
    const int j = k & 3, h = (k >> 3) & 1;
    if (PERMUTE) return F == 4 ? (j & 1) | (j >> 1) << 3 : 4 * j;
    return MN >= 128 ? 2 * j + 8 * h : 0;
}

typedef __attribute__((address_space(3))) char lds_char;

// 16 bytes a lane from base + offset to 16 adjacent bytes a lane from `to` (the
// same in all lanes).  The builtin for this makes the compiler wait for all
// such loads before the next LDS read that it cannot tell apart, which every
// transposing read is; arrive() does the waiting here.  Nothing is returned in
// a register.  m0 is reserved, which the compiler warns about where it is named
// as overwritten; it keeps nothing there.
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
__device__ __forceinline__ void load_lds(const char *base, uint32_t offset, lds_char *to)
{
    const uint32_t at = (uint32_t)(uintptr_t)to;
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2"
                 :
                 : "s"(__builtin_amdgcn_readfirstlane(at)), "v"(offset), "s"(base)
                 : "memory", "m0");
}
#pragma clang diagnostic pop

// threadIdx.x, of which nothing that is worked out from it is kept over a tile's
// products: it would cost registers there.
__device__ __forceinline__ int thread_anew()
{
    int thread = threadIdx.x;
    asm volatile("" : "+v"(thread));
    return thread;
}

// One operand's slices: where this thread's 16-byte pieces come from.  F: the
// blocks of 16 that a wavefront takes.
template <int MN, int F, int THREADS, bool MC, bool PERMUTE>
struct Loader {
    static constexpr int kBytes = MN * kStepK * 2;
    static constexpr int kRounds = kBytes / 16 / THREADS;
    static_assert(kRounds * 16 * THREADS == kBytes, "whole rounds");
    static constexpr int kRowPieces = MC ? MN / 8 : kStepK / 8;
    uint32_t off[kRounds];

    // mn_last: the last row (KC) or the last 8-aligned column (MC) of the
    // operand, relative to the tile; k_last: the last row of an MC operand or
    // the last 8-aligned column of a KC one, relative to the step.  Past it an
    // MC operand's last row stands in, and a KC operand's first columns of the
    // step: they meet zeros of the other operand.
    __device__ __forceinline__ void place(int64_t ld, int mn_last, int k_last)
    {
        const int thread = thread_anew();
#pragma unroll
        for (int r = 0; r < kRounds; ++r) {
            const int piece = r * THREADS + thread, row = piece / kRowPieces, slot = piece % kRowPieces;
            if constexpr (MC) {
                const int mn = min((slot ^ flip<MN, F, PERMUTE>(row)) * 8, mn_last);
                off[r] = ((uint32_t)min(row, k_last) * (uint32_t)ld + (uint32_t)mn) * 2u;
            } else {
                int mn = row;
                if constexpr (PERMUTE) {
                    const int in = row % (16 * F), b = in / 16, q = in / 4 % 4;
                    mn = row - in + 4 * F * q + 4 * b + in % 4;
                }
                const int k = (slot ^ swizzle(row)) * 8;
                off[r] = ((uint32_t)min(mn, mn_last) * (uint32_t)ld + (uint32_t)(k <= k_last ? k : 0)) * 2u;
            }
        }
    }

    __device__ __forceinline__ void issue_one(const char *base, lds_char *stage, int wave, int r) const
    {
        load_lds(base, off[r], stage + (r * THREADS + wave * 64) * 16);
    }
};

// Byte offsets of a wavefront's F fragments in a slice (which starts at a
// multiple of 1024 bytes).  In an MC slice a block further on is another value
// of bits that nothing else of the offset uses, so one register serves all.
template <int MN, int F, bool MC, bool PERMUTE>
struct Reader {
    int at[MC ? 1 : 2];

    // mn: the wavefront's first row or column in the tile
    __device__ __forceinline__ void place(int mn, int lane)
    {
        const int l16 = lane & 15, quarter = lane >> 4;
        if constexpr (MC) {
            const int k = 8 * quarter + (l16 >> 2), q = l16 & 3;
            const int col = mn + (PERMUTE ? 4 * F * q : 4 * q);
            at[0] = k * (2 * MN) + ((col / 8) ^ flip<MN, F, PERMUTE>(k)) * 16 + (col & 4) * 2;
        } else {
#pragma unroll
            for (int s = 0; s < 2; ++s) at[s] = (mn + l16) * 128 + (((4 * s + quarter) ^ swizzle(l16)) * 16);
        }
    }

    template <class E>
    __device__ __forceinline__ typename Frag<E>::type read(lds_char *slice, int f, int s) const
    {
        typedef typename Frag<E>::type V;
        if constexpr (MC) {
            typedef __attribute__((address_space(3))) s16x4 lds4;
            const uint32_t from = ((uint32_t)(uintptr_t)slice + (uint32_t)at[0]) ^ (uint32_t)(f << (PERMUTE ? 3 : 5));
            const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4 *)(uintptr_t)(from + (32 * s) * (2 * MN)));
            const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4 *)(uintptr_t)(from + (32 * s + 4) * (2 * MN)));
            const s16x8 v = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
            return __builtin_bit_cast(V, v);
        } else {
            typedef __attribute__((address_space(3))) V ldsv;
            return *(ldsv *)(slice + at[s] + f * 16 * 128);
        }
    }
};

// The work-group's loads into LDS have arrived but for the last FLYING of each
// thread, and its reads of LDS are done.  The compiler's own barrier would not
// wait for loads that write LDS.
template <int FLYING>
__device__ __forceinline__ void arrive()
{
    static_assert(FLYING < 16, "four bits");
    __builtin_amdgcn_s_waitcnt(0x0070 | FLYING);  // vmcnt(FLYING) lgkmcnt(0)
    __syncthreads();
}

// Tile `id` of `ids`.  The hardware deals work-groups, and a grid that is a
// multiple of 8 its tiles, round-robin to eight XCDs with an L2 each; XCD x takes the x-th run of logical ids, as in mfma::tile_of.  Ids walk the
// tiles of one part of the sum, then those of the next (parts share nothing),
// and within a part groups of 8 tile rows column by column, so that the
// work-groups of an XCD share rows of A and columns of B.
__device__ __forceinline__ void place_tile(int id, int ids, int tiles_m, int tiles_n, int &tm, int &tn, int &split)
{
    const int q = ids / mfma::kXcds, r = ids % mfma::kXcds;
    const int x = id % mfma::kXcds;
    const int logical = id / mfma::kXcds + x * q + min(x, r);
    const int tiles = tiles_m * tiles_n;
    split = logical / tiles;
    const int tile = logical - split * tiles, per_group = 8 * tiles_n;
    const int group = tile / per_group, in_group = tile - group * per_group;
    const int rows = min(tiles_m - group * 8, 8);
    tm = group * 8 + in_group % rows;
    tn = in_group / rows;
}

// Scheduling hints: READS LDS reads spread evenly among MFMAS matrix
// instructions.
template <int MFMAS, int READS, int I = 0>
__device__ __forceinline__ void spread()
{
    if constexpr (I < MFMAS) {
        constexpr int reads = (I + 1) * READS / MFMAS - I * READS / MFMAS;
        if constexpr (reads > 0) __builtin_amdgcn_sched_group_barrier(0x100, reads, 0);
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
        spread<MFMAS, READS, I + 1>();
    }
}

// The tiles of C that a work-group computes: blockIdx.x, blockIdx.x +
// gridDim.x, ...  For each, `epilogue(acc, row0, col0, split)` is called when
// the lane holds in acc[i][j][r] row row0 + 16·i + lane % 16, column col0 +
// 4·FN·(lane / 16) + 4·j + r.  The loads run two steps ahead without regard to
// where a tile ends, so the next tile's are under way by then.
template <class E, int BM, int BN, int WM, int WN, bool A_MC, bool B_MC>
struct TileProduct {
    static constexpr int kThreads = 64 * WM * WN;
    static constexpr int FM = BM / WM / 16, FN = BN / WN / 16;
    static constexpr int BK = kStepK;
    static constexpr int kStage = (BM + BN) * BK * 2;
    static constexpr int kLds = 2 * kStage;
    typedef f32x4 Acc[FM][FN];

    template <class Epilogue>
    static __device__ __forceinline__ void run(const Operands &p, lds_char *lds, Epilogue epilogue)
    {
        const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
        const int wm = wave / WN, wn = wave % WN;
        const int tiles = p.tiles_m * p.tiles_n * p.splits;
        Loader<BM, FM, kThreads, A_MC, false> la;
        Loader<BN, FN, kThreads, B_MC, true> lb;
        Reader<BM, FM, A_MC, false> ra;
        Reader<BN, FN, B_MC, true> rb;
        ra.place(wm * (FM * 16), lane);
        rb.place(wn * (FN * 16), lane);
        constexpr int kLoadsA = decltype(la)::kRounds, kLoads = kLoadsA + decltype(lb)::kRounds;
        constexpr int kReadsA = FM / 2 * (A_MC ? 2 : 1), kReadsB = FN * (B_MC ? 2 : 1);

        // A tile's place and its steps.
        auto steps_of = [&](int split, int &first, int &last) {
            first = split * p.steps_per_split;
            last = min(p.steps, first + p.steps_per_split);
        };
        auto place = [&](int id, int &m0, int &n0, int &split) {
            int tm, tn;
            place_tile(id, tiles, p.tiles_m, p.tiles_n, tm, tn, split);
            m0 = tm * BM;
            n0 = tn * BN;
        };

        // The loads: which tile, segment and step they are at.
        int at_id = blockIdx.x, seg, k, first, last, a_last, b_last;
        const char *A, *B, *from_a, *from_b;
        auto start = [](int step, int rows) { return min(step * BK, rows - 1); };
        auto open = [&]() {
            int m0, n0, split;
            place(at_id, m0, n0, split);
            steps_of(split, first, last);
            // a tile may lie past an operand's last row: it takes that one
            const int a_end = p.mn_a - (A_MC ? 8 : 1), b_end = p.mn_b - (B_MC ? 8 : 1);
            const int a0 = min(m0, a_end), b0 = min(n0, b_end);
            a_last = a_end - a0;
            b_last = b_end - b0;
            la.place(p.lda, a_last, A_MC ? p.k_a - 1 - start(first, p.k_a) : BK);
            lb.place(p.ldb, b_last, B_MC ? p.k_b - 1 - start(first, p.k_b) : p.k_b - 8 - first * BK);
            A = (const char *)p.A + (A_MC ? (int64_t)a0 : (int64_t)a0 * p.lda) * 2;
            B = (const char *)p.B + (B_MC ? (int64_t)b0 : (int64_t)b0 * p.ldb) * 2;
            seg = 0;
            k = first;
        };
        auto seek = [&]() {
            if (k == last) {
                k = first;
                if (++seg == p.segments) {
                    // after the last tile its first steps are loaded again, for nobody
                    if (at_id + (int)gridDim.x < tiles) at_id += gridDim.x;
                    open();
                }
            }
            const int start_a = A_MC ? start(k, p.k_a) : k * BK, start_b = B_MC ? start(k, p.k_b) : k * BK;
            from_a = A + (A_MC ? start_a * p.lda : (int64_t)start_a) * 2;
            from_b = B + (B_MC ? start_b * p.ldb : (int64_t)start_b) * 2;
            if (p.segments > 1) {
                from_a += ((kPairsA >> (2 * seg)) & 3) * p.plane_a * 2;
                from_b += ((kPairsB >> (2 * seg)) & 3) * p.plane_b * 2;
            }
            // an operand may end inside its last step; the next segment has whole ones again
            if (A_MC && ((k + 1) * BK > p.k_a || (p.segments > 1 && k == first))) la.place(p.lda, a_last, p.k_a - 1 - start_a);
            if ((k + 1) * BK > p.k_b || (B_MC && p.segments > 1 && k == first)) lb.place(p.ldb, b_last, p.k_b - (B_MC ? 1 : 8) - start_b);
            ++k;
        };
        // A round of a KC operand may be just the rows that the wavefronts'
        // first (or second) halves are made of.  Early loads: B and those of A.
        constexpr bool kHalves = !A_MC && kThreads / 8 == FM / 2 * 16;
        constexpr int kEarlyA = kHalves ? kLoadsA / 2 : 0, kEarly = kLoads - kLoadsA + kEarlyA;
        auto issue = [&](int stage, int n) {  // the n-th load, early ones first
            lds_char *to = lds + stage * kStage;
            if (n < kEarlyA) la.issue_one(from_a, to, wave, 2 * n);
            else if (n < kEarly) lb.issue_one(from_b, to + BM * BK * 2, wave, n - kEarlyA);
            else la.issue_one(from_a, to, wave, kHalves ? 2 * (n - kEarly) + 1 : n - kEarly);
        };
        auto issue_all = [&](int stage) {
#pragma unroll
            for (int n = 0; n < kLoads; ++n) issue(stage, n);
        };

        Acc acc;
        // A step has four phases: each half of the step's 64 values of k with
        // each half of the wavefront's rows.  Two sets of fragments: those of
        // the next phase are read while these are multiplied.
        typename Frag<E>::type a[2][FM / 2], b[2][FN];
        auto read = [&](int stage, int phase) {
            lds_char *as = lds + stage * kStage, *bs = as + BM * BK * 2;
            const int s = phase & 1, h = phase >> 1;
            if (h == 0) {
#pragma unroll
                for (int j = 0; j < FN; ++j) b[s][j] = rb.template read<E>(bs, j, s);
            }
#pragma unroll
            for (int i = 0; i < FM / 2; ++i) a[s][i] = ra.template read<E>(as, h * (FM / 2) + i, s);
        };
        constexpr int kProducts = FM / 2 * FN;
        auto multiply = [&](int phase, int m) {
            const int s = phase & 1, h = phase >> 1, i = m / FN, j = m % FN;
            acc[h * (FM / 2) + i][j] = Frag<E>::mfma(b[s][j], a[s][i], acc[h * (FM / 2) + i][j]);
        };

        at_id = blockIdx.x;
        open();
        seek();
        issue_all(0);
        seek();
        issue_all(1);
        arrive<0>();
        read(0, 0);
        int stage = 0;
        for (int id = blockIdx.x; id < tiles; id += gridDim.x) {
#pragma unroll
            for (int i = 0; i < FM; ++i)
#pragma unroll
                for (int j = 0; j < FN; ++j)
#pragma unroll
                    for (int r = 0; r < 4; ++r) acc[i][j][r] = 0.0f;
            int m0, n0, split, from, to;
            place(id, m0, n0, split);
            steps_of(split, from, to);
            for (int n = (to - from) * p.segments; n > 0; --n) {
                // A step on the slices of `stage`, its first fragments read.
                // The first barrier stands after the phases that read B and
                // the first half of A, the second before the last phase, whose
                // fragments are in registers by then: what is read no more is
                // loaded for the step after next.  At the second one the next
                // step's slices have arrived, so its first fragments are read
                // under the last products.
                seek();
                read(stage, 1);
#pragma unroll
                for (int m = 0; m < kProducts; ++m) multiply(0, m);
                spread<kProducts, kReadsA + kReadsB>();
                read(stage, 2);
#pragma unroll
                for (int m = 0; m < kProducts; ++m) multiply(1, m);
                spread<kProducts, kReadsA>();
                __syncthreads();
                read(stage, 3);
#pragma unroll
                for (int m = 0; m < kProducts; ++m) {
#pragma unroll
                    for (int n = m * kEarly / kProducts; n < (m + 1) * kEarly / kProducts; ++n) issue(stage, n);
                    multiply(2, m);
                }
                arrive<kEarly>();
                read(stage ^ 1, 0);
#pragma unroll
                for (int m = 0; m < kProducts; ++m) {
                    constexpr int kLate = kLoads - kEarly;
#pragma unroll
                    for (int n = m * kLate / kProducts; n < (m + 1) * kLate / kProducts; ++n) issue(stage, kEarly + n);
                    multiply(3, m);
                }
                stage ^= 1;
            }
            epilogue(acc, m0 + wm * (FM * 16), n0 + wn * (FN * 16), split);
        }
        __builtin_amdgcn_s_waitcnt(0x0F70);  // vmcnt(0): no load into LDS outlives the work-group
    }
};

}  // namespace m16
}  // namespace tgemm
