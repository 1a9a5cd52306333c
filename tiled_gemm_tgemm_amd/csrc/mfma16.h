// Tiles of 16-bit products on the matrix cores: C = A·B with A M×K and B K×N
// of bf16 or fp16 values, summed in fp32 registers.
//
// * A work-group of WM×WN wavefronts holds a BM×BN tile of C in registers, a
//   wavefront FM×FN blocks of 32×32 (v_mfma_f32_32x32x16).  The blocks are
//   formed transposed (B's fragment is the instruction's first operand), so a
//   lane holds 16 columns of one row of C: sums along a row of C stay within
//   a lane and its partner, and a row's values leave in 16-byte pieces.
// * K runs in steps of BK.  A step's slices of A and B go from device memory
//   straight into LDS, 16 bytes a lane, into one of STAGES stages; the loads of
//   the next steps are under way while a step is multiplied.
// * The order of the 32 columns of a block is free as long as the reader of C
//   knows it: column 16·h + 4·q + r of C sits at index 8·q + 4·h + r of the
//   instruction, which is what gives lane half h the 16 adjacent columns
//   16·h ... 16·h + 15 in accumulator order.
//
// An operand is K-contiguous ("KC": element (mn, k) at mn·ld + k) or
// MN-contiguous ("MC": at k·ld + mn).  A KC slice lies in LDS as mn rows of
// 128 bytes, an MC slice as 64 rows (one a k) of 2·BM or 2·BN bytes, from
// which the transposing LDS read gathers four values of k a lane.  The loads
// into LDS write 16-byte pieces in lane order, so the pieces are permuted on
// the reading side of device memory, within a cache line: piece c of a KC row
// goes to c ^ (row / 2 & 7), and the 64-byte quarter-lines of an MC row are
// exchanged by the row's k.  Without that the 32 rows of a KC fragment would
// start in the same banks, as would the four rows of a transposing read.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "mfma_common.h"

namespace tgemm {
namespace m16 {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
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
    int k_a, k_b;              // MC: rows (values of k) of A / B
    int tiles_m, tiles_n;
};

// A float32 operand is the sum of three bf16 planes (high, middle, low: 24
// bits).  Of the nine products of planes the six that reach 2^-24 of the
// largest are summed, small ones first: (mid,mid), (high,low), (low,high),
// (high,mid), (mid,high), (high,high); two bits a plane.
constexpr int kPairsA = (1 << 0) | (0 << 2) | (2 << 4) | (0 << 6) | (1 << 8) | (0 << 10);
constexpr int kPairsB = (1 << 0) | (2 << 2) | (0 << 4) | (1 << 6) | (0 << 8) | (0 << 10);

template <class E>
struct Frag;
template <>
struct Frag<__bf16> {
    typedef bf16x8 type;
    static __device__ __forceinline__ f32x16 mfma(bf16x8 a, bf16x8 b, f32x16 c)
    {
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
    }
};
template <>
struct Frag<_Float16> {
    typedef f16x8 type;
    static __device__ __forceinline__ f32x16 mfma(f16x8 a, f16x8 b, f32x16 c)
    {
        return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, 0, 0, 0);
    }
};

// A 16-byte read of a KC fragment takes 16 rows at a time, which span 16·2·BK
// bytes; each of them finds its piece in another 16 bytes of the 256 that the
// banks are wide.
template <int BK>
__device__ __forceinline__ constexpr int swizzle(int row) { return BK == 64 ? (row >> 1) & 7 : (row >> 2) & 3; }

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

// One operand's slices: where this thread's 16-byte pieces come from.
template <int MN, int BK, int THREADS, bool MC, bool PERMUTE>
struct Loader {
    static constexpr int kBytes = MN * BK * 2;
    static constexpr int kRounds = kBytes / 16 / THREADS;
    static_assert(kRounds * 16 * THREADS == kBytes, "whole rounds");
    static constexpr int kRowPieces = MC ? MN / 8 : BK / 8;
    uint32_t off[kRounds];

    static __device__ __forceinline__ int piece(int r) { return r * THREADS + (int)threadIdx.x; }

    // mn_last: the last row (KC) or the last 8-aligned column (MC) of the
    // operand, relative to the tile; k_last: the last row of an MC operand,
    // relative to the step.
    __device__ __forceinline__ void place(int64_t ld, int mn_last, int k_last)
    {
#pragma unroll
        for (int r = 0; r < kRounds; ++r) {
            const int row = piece(r) / kRowPieces, slot = piece(r) % kRowPieces;
            if constexpr (MC) {
                constexpr int mask = MN / 32 - 1;
                const int quarter = (slot / 4) ^ (((row & 3) | ((row >> 1) & 4)) & mask);
                const int mn = min(quarter * 32 + (slot % 4) * 8, mn_last);
                off[r] = ((uint32_t)min(row, k_last) * (uint32_t)ld + (uint32_t)mn) * 2u;
            } else {
                int mn = row;
                if constexpr (PERMUTE) mn = (row & ~31) | ((row & 4) << 2) | ((row & 24) >> 1) | (row & 3);
                off[r] = ((uint32_t)min(mn, mn_last) * (uint32_t)ld + (uint32_t)((slot ^ swizzle<BK>(row)) * 8)) * 2u;
            }
        }
    }

    __device__ __forceinline__ void issue_one(const char *base, lds_char *stage, int wave, int r) const
    {
        load_lds(base, off[r], stage + (r * THREADS + wave * 64) * 16);
    }
};

// Byte offsets of a wavefront's fragments in a slice.
template <int MN, int BK, int F, bool MC, bool PERMUTE>
struct Reader {
    int at[MC ? F : BK / 16];

    // mn: the wavefront's first row or column in the tile
    __device__ __forceinline__ void place(int mn, int lane)
    {
        if constexpr (MC) {
            constexpr int mask = MN / 32 - 1;
            const int i = lane & 15, row = i >> 2, piece = i & 3, right = (lane >> 4) & 1, half = lane >> 5;
            const int in = PERMUTE ? 32 * (piece & 1) + 16 * right + 8 * (piece >> 1) : 32 * right + 8 * piece;
#pragma unroll
            for (int f = 0; f < F; ++f)
                at[f] = (8 * half + row) * (2 * MN) + (((mn / 32 + f) ^ ((row | (half << 2)) & mask)) * 64) + in;
        } else {
            const int l32 = lane & 31, half = lane >> 5;
#pragma unroll
            for (int s = 0; s < BK / 16; ++s) at[s] = (mn + l32) * (2 * BK) + (((2 * s + half) ^ swizzle<BK>(l32)) * 16);
        }
    }

    template <class E>
    __device__ __forceinline__ typename Frag<E>::type read(lds_char *slice, int f, int s) const
    {
        typedef typename Frag<E>::type V;
        if constexpr (MC) {
            typedef __attribute__((address_space(3))) s16x4 lds4;
            const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4 *)(slice + at[f] + (16 * s) * (2 * MN)));
            const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4 *)(slice + at[f] + (16 * s + 4) * (2 * MN)));
            const s16x8 v = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
            return __builtin_bit_cast(V, v);
        } else {
            typedef __attribute__((address_space(3))) V ldsv;
            return *(ldsv *)(slice + at[s] + f * 32 * (2 * BK));
        }
    }
};

// The work-group's loads into LDS have arrived but for the last FLYING of each
// thread, and its reads of LDS are done.  The compiler's own barrier would not
// wait for loads that write LDS.
template <int FLYING>
__device__ __forceinline__ void arrive()
{
    __builtin_amdgcn_s_waitcnt((FLYING & 15) | (FLYING >> 4) << 14 | 7 << 4);  // vmcnt(FLYING) lgkmcnt(0)
    __syncthreads();
}

// The hardware deals work-groups round-robin to eight XCDs with an L2 each;
// XCD x takes the x-th run of logical ids, as in mfma::tile_of.  Ids walk the
// tiles of one part of the sum, then those of the next (parts share nothing),
// and within a part groups of 8 tile rows column by column, so that the
// work-groups of an XCD share rows of A and columns of B.
__device__ __forceinline__ void place_tile(int tiles_m, int tiles_n, int &tm, int &tn, int &split)
{
    const int groups = gridDim.x, q = groups / mfma::kXcds, r = groups % mfma::kXcds;
    const int x = blockIdx.x % mfma::kXcds;
    const int logical = blockIdx.x / mfma::kXcds + x * q + min(x, r);
    const int tiles = tiles_m * tiles_n;
    split = logical / tiles;
    const int tile = logical - split * tiles, per_group = 8 * tiles_n;
    const int group = tile / per_group, in_group = tile - group * per_group;
    const int rows = min(tiles_m - group * 8, 8);
    tm = group * 8 + in_group % rows;
    tn = in_group / rows;
}

struct Yes { static constexpr bool value = true; };
struct No { static constexpr bool value = false; };

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

// A tile of C.  After run(), lane (l32 = lane & 31, half = lane >> 5) holds in
// acc[i][j][r] row row0 + i·32 + l32, column col0 + j·32 + 16·half + r.
template <class E, int BM, int BN, int WM, int WN, bool A_MC, bool B_MC, int BK, int STAGES>
struct TileProduct {
    static constexpr int kThreads = 64 * WM * WN;
    static constexpr int FM = BM / WM / 32, FN = BN / WN / 32;
    static constexpr int kStage = (BM + BN) * BK * 2;
    static constexpr int kLds = STAGES * kStage;

    f32x16 acc[FM][FN];
    int row0, col0, split;

    __device__ __forceinline__ void run(const Operands &p, lds_char *lds)
    {
        const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
        const int wm = wave / WN, wn = wave % WN;
        int tm, tn;
        place_tile(p.tiles_m, p.tiles_n, tm, tn, split);
        const int m0 = tm * BM, n0 = tn * BN;
        row0 = m0 + wm * (FM * 32);
        col0 = n0 + wn * (FN * 32);
#pragma unroll
        for (int i = 0; i < FM; ++i)
#pragma unroll
            for (int j = 0; j < FN; ++j)
#pragma unroll
                for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.0f;

        const int first = split * p.steps_per_split * (kStepK / BK);
        const int last = min(p.steps * (kStepK / BK), first + p.steps_per_split * (kStepK / BK));
        if (first >= last) return;

        Loader<BM, BK, kThreads, A_MC, false> la;
        Loader<BN, BK, kThreads, B_MC, true> lb;
        Reader<BM, BK, FM, A_MC, false> ra;
        Reader<BN, BK, FN, B_MC, true> rb;
        ra.place(wm * (FM * 32), lane);
        rb.place(wn * (FN * 32), lane);
        const int a_last = A_MC ? p.mn_a - 8 - m0 : p.mn_a - 1 - m0;
        const int b_last = B_MC ? p.mn_b - 8 - n0 : p.mn_b - 1 - n0;
        // An MC operand may end inside a step or before its last ones (K is
        // padded to 64): such a step starts at the last row at the latest.
        auto start = [](int k, int rows) { return min(k * BK, rows - 1); };
        if constexpr (A_MC) la.place(p.lda, a_last, p.k_a - 1 - start(first, p.k_a));
        else la.place(p.lda, a_last, 0);
        if constexpr (B_MC) lb.place(p.ldb, b_last, p.k_b - 1 - start(first, p.k_b));
        else lb.place(p.ldb, b_last, 0);
        const char *A = (const char *)p.A + (A_MC ? (int64_t)m0 : (int64_t)m0 * p.lda) * 2;
        const char *B = (const char *)p.B + (B_MC ? (int64_t)n0 : (int64_t)n0 * p.ldb) * 2;
        // where the next loads come from
        int seg = 0, k = first;
        const char *from_a = nullptr, *from_b = nullptr;
        auto seek = [&]() {
            const int start_a = A_MC ? start(k, p.k_a) : k * BK, start_b = B_MC ? start(k, p.k_b) : k * BK;
            from_a = A + (A_MC ? start_a * p.lda : (int64_t)start_a) * 2;
            from_b = B + (B_MC ? start_b * p.ldb : (int64_t)start_b) * 2;
            if (p.segments > 1) {
                from_a += ((kPairsA >> (2 * seg)) & 3) * p.plane_a * 2;
                from_b += ((kPairsB >> (2 * seg)) & 3) * p.plane_b * 2;
            }
            // the last rows of an MC operand, and back to whole steps for the next segment
            if (A_MC && ((k + 1) * BK > p.k_a || (p.segments > 1 && k == first))) la.place(p.lda, a_last, p.k_a - 1 - start_a);
            if (B_MC && ((k + 1) * BK > p.k_b || (p.segments > 1 && k == first))) lb.place(p.ldb, b_last, p.k_b - 1 - start_b);
            if (++k == last) {
                k = first;
                ++seg;
            }
        };
        constexpr int kLoadsA = decltype(la)::kRounds, kLoads = kLoadsA + decltype(lb)::kRounds;
        auto issue = [&](int stage, int lo, int hi) {
#pragma unroll
            for (int r = 0; r < kLoads; ++r) {
                if (r < lo || r >= hi) continue;
                if (r < kLoadsA) la.issue_one(from_a, lds + stage * kStage, wave, r);
                else lb.issue_one(from_b, lds + stage * kStage + BM * BK * 2, wave, r - kLoadsA);
            }
        };

        // Two sets of fragments: those of the next 16 values of k are read
        // while these are multiplied.
        typename Frag<E>::type a[2][FM], b[2][FN];
        auto read = [&](int stage, int s) {
            lds_char *as = lds + stage * kStage, *bs = as + BM * BK * 2;
#pragma unroll
            for (int j = 0; j < FN; ++j) b[s & 1][j] = rb.template read<E>(bs, j, s);
#pragma unroll
            for (int i = 0; i < FM; ++i) a[s & 1][i] = ra.template read<E>(as, i, s);
        };
        auto multiply = [&](int s) {
#pragma unroll
            for (int i = 0; i < FM; ++i)
#pragma unroll
                for (int j = 0; j < FN; ++j) acc[i][j] = Frag<E>::mfma(b[s & 1][j], a[s & 1][i], acc[i][j]);
        };
        constexpr int kReads = FM * (A_MC ? 2 : 1) + FN * (B_MC ? 2 : 1);

        // A step on the slices of `stage`, its first fragments read.  The
        // barrier stands before the last 16 values of k, whose fragments are
        // in registers by then: this stage is read no more, so the loads of
        // the step STAGES further on go there, and the next step's slices
        // have arrived, so its first fragments are read under these products.
        constexpr int kSubs = BK / 16;
        auto step = [&](int stage, int after, auto load, auto next) {
#pragma unroll
            for (int s = 0; s < kSubs - 1; ++s) {
                read(stage, s + 1);
                multiply(s);
                spread<FM * FN, kReads>();
            }
            if constexpr (decltype(next)::value) {
                if constexpr (decltype(load)::value) arrive<(STAGES - 2) * kLoads>();
                else arrive<0>();
                read(after, 0);
            }
#pragma unroll
            for (int m = 0; m < FM * FN; ++m) {
                if constexpr (decltype(load)::value) issue(stage, m * kLoads / (FM * FN), (m + 1) * kLoads / (FM * FN));
                const int i = m / FN, j = m % FN, s = (kSubs - 1) & 1;
                acc[i][j] = Frag<E>::mfma(b[s][j], a[s][i], acc[i][j]);
            }
        };

        const int total = (last - first) * p.segments;
        int ahead = 0;
        for (; ahead < STAGES && ahead < total; ++ahead) {
            seek();
            issue(ahead, 0, kLoads);
        }
        arrive<0>();
        read(0, 0);
        int n = 0, stage = 0;
        auto following = [](int st) { return st + 1 == STAGES ? 0 : st + 1; };
        for (; n + STAGES < total; ++n) {
            seek();
            step(stage, following(stage), Yes{}, Yes{});
            stage = following(stage);
        }
        for (; n + 1 < total; ++n) {
            step(stage, following(stage), No{}, Yes{});
            stage = following(stage);
        }
        step(stage, stage, No{}, No{});
    }
};

}  // namespace m16
}  // namespace tgemm
