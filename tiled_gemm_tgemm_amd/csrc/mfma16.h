// Tiles of 16-bit products on the matrix cores: C = A·B with A M×K and B K×N
// of bf16 or fp16 values, summed in fp32 registers.
//
// * A work-group of WM×WN wavefronts holds a BM×BN tile of C in registers, a
//   wavefront FM×FN blocks of 32×32 (v_mfma_f32_32x32x16).  The blocks are
//   formed transposed (B's fragment is the instruction's first operand), so a
//   lane holds 16 columns of one row of C: sums along a row of C stay within
//   a lane and its partner, and a row's values leave in 16-byte pieces.
// * K runs in steps of 64.  A step's slices of A and B go from device memory
//   straight into LDS, 16 bytes a lane, into one of two stages; the loads of
//   the next step are under way while a step is multiplied.
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
// goes to c ^ (row & 7), and the 64-byte quarter-lines of an MC row are
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
    int steps_per_split;       // blockIdx.y takes steps [y·this, (y+1)·this)
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

typedef __attribute__((address_space(3))) char lds_char;
typedef const __attribute__((address_space(1))) char global_char;

// One operand's slices: where this thread's 16-byte pieces come from.
template <int MN, int THREADS, bool MC, bool PERMUTE>
struct Loader {
    static constexpr int kBytes = MN * kStepK * 2;
    static constexpr int kRounds = kBytes / 16 / THREADS;
    static_assert(kRounds * 16 * THREADS == kBytes, "whole rounds");
    static constexpr int kRowPieces = MC ? MN / 8 : 8;
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
                off[r] = ((uint32_t)min(mn, mn_last) * (uint32_t)ld + (uint32_t)((slot ^ (row & 7)) * 8)) * 2u;
            }
        }
    }

    __device__ __forceinline__ void issue(const char *base, lds_char *stage, int wave) const
    {
#pragma unroll
        for (int r = 0; r < kRounds; ++r) {
            // kept as 32 bits in the loop: the load then adds it to the scalar base by itself
            uint32_t o = off[r];
            asm volatile("" : "+v"(o));
            __builtin_amdgcn_global_load_lds((global_char *)(base + o), stage + (r * THREADS + wave * 64) * 16, 16, 0, 0);
        }
    }
};

// Byte offsets of a wavefront's fragments in a slice.
template <int MN, int F, bool MC, bool PERMUTE>
struct Reader {
    int at[MC ? F : 4];

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
            for (int s = 0; s < 4; ++s) at[s] = (mn + l32) * 128 + (((2 * s + half) ^ (l32 & 7)) * 16);
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
            return *(ldsv *)(slice + at[s] + f * 32 * 128);
        }
    }
};

// The work-group's loads into LDS have arrived, and its reads of LDS are done.
// A barrier's fence does not by itself wait for loads that write LDS.
__device__ __forceinline__ void arrive()
{
    __builtin_amdgcn_s_waitcnt(0x0F70);  // vmcnt(0)
    __syncthreads();
}

struct Yes { static constexpr bool value = true; };
struct No { static constexpr bool value = false; };

// Scheduling hints: READS LDS reads and LOADS loads spread evenly among MFMAS
// matrix instructions.
template <int MFMAS, int READS, int LOADS, int I = 0>
__device__ __forceinline__ void spread()
{
    if constexpr (I < MFMAS) {
        constexpr int reads = (I + 1) * READS / MFMAS - I * READS / MFMAS;
        constexpr int loads = (I + 1) * LOADS / MFMAS - I * LOADS / MFMAS;
        if constexpr (reads > 0) __builtin_amdgcn_sched_group_barrier(0x100, reads, 0);
        if constexpr (loads > 0) __builtin_amdgcn_sched_group_barrier(0x020, loads, 0);
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
        spread<MFMAS, READS, LOADS, I + 1>();
    }
}

// A tile of C.  After run(), lane (l32 = lane & 31, half = lane >> 5) holds in
// acc[i][j][r] row row0 + i·32 + l32, column col0 + j·32 + 16·half + r.
template <class E, int BM, int BN, int WM, int WN, bool A_MC, bool B_MC>
struct TileProduct {
    static constexpr int kThreads = 64 * WM * WN;
    static constexpr int FM = BM / WM / 32, FN = BN / WN / 32;
    static constexpr int kStage = (BM + BN) * kStepK * 2;
    static constexpr int kLds = 2 * kStage;

    f32x16 acc[FM][FN];
    int row0, col0;

    __device__ __forceinline__ void run(const Operands &p, lds_char *lds)
    {
        const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
        const int wm = wave / WN, wn = wave % WN;
        int tm, tn;
        mfma::tile_of(p.tiles_m, p.tiles_n, 8, tm, tn);
        const int m0 = tm * BM, n0 = tn * BN;
        row0 = m0 + wm * (FM * 32);
        col0 = n0 + wn * (FN * 32);
#pragma unroll
        for (int i = 0; i < FM; ++i)
#pragma unroll
            for (int j = 0; j < FN; ++j)
#pragma unroll
                for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.0f;

        const int first = blockIdx.y * p.steps_per_split;
        const int last = min(p.steps, first + p.steps_per_split);
        if (first >= last) return;

        Loader<BM, kThreads, A_MC, false> la;
        Loader<BN, kThreads, B_MC, true> lb;
        Reader<BM, FM, A_MC, false> ra;
        Reader<BN, FN, B_MC, true> rb;
        ra.place(wm * (FM * 32), lane);
        rb.place(wn * (FN * 32), lane);
        const int a_last = A_MC ? p.mn_a - 8 - m0 : p.mn_a - 1 - m0;
        const int b_last = B_MC ? p.mn_b - 8 - n0 : p.mn_b - 1 - n0;
        la.place(p.lda, a_last, A_MC ? p.k_a - 1 - first * kStepK : 0);
        lb.place(p.ldb, b_last, B_MC ? p.k_b - 1 - first * kStepK : 0);
        const char *A = (const char *)p.A + (A_MC ? (int64_t)m0 : (int64_t)m0 * p.lda) * 2;
        const char *B = (const char *)p.B + (B_MC ? (int64_t)n0 : (int64_t)n0 * p.ldb) * 2;
        const int64_t step_a = (A_MC ? (int64_t)kStepK * p.lda : (int64_t)kStepK) * 2;
        const int64_t step_b = (B_MC ? (int64_t)kStepK * p.ldb : (int64_t)kStepK) * 2;

        // where the next loads come from
        int seg = 0, k = first;
        const char *from_a = nullptr, *from_b = nullptr;
        auto seek = [&]() {
            from_a = A + k * step_a;
            from_b = B + k * step_b;
            if (p.segments > 1) {
                from_a += ((kPairsA >> (2 * seg)) & 3) * p.plane_a * 2;
                from_b += ((kPairsB >> (2 * seg)) & 3) * p.plane_b * 2;
            }
            // the last rows of an MC operand, and back to whole steps for the next segment
            if (A_MC && ((k + 1) * kStepK > p.k_a || (p.segments > 1 && k == first)))
                la.place(p.lda, a_last, p.k_a - 1 - k * kStepK);
            if (B_MC && ((k + 1) * kStepK > p.k_b || (p.segments > 1 && k == first)))
                lb.place(p.ldb, b_last, p.k_b - 1 - k * kStepK);
            if (++k == last) {
                k = first;
                ++seg;
            }
        };
        auto issue = [&](int stage) {
            la.issue(from_a, lds + stage * kStage, wave);
            lb.issue(from_b, lds + stage * kStage + BM * kStepK * 2, wave);
        };

        // Two sets of fragments: those of the next 16 values of k are read
        // while these are multiplied.
        typename Frag<E>::type a[2][FM], b[2][FN];
        auto read = [&](int stage, int s) {
            lds_char *as = lds + stage * kStage, *bs = as + BM * kStepK * 2;
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
        constexpr int kLoads = decltype(la)::kRounds + decltype(lb)::kRounds;

        // A step on the slices of `stage`, its first fragments read.  The
        // barrier stands before the last quarter, whose fragments are in
        // registers by then: this stage is read no more, so the loads of the
        // step after next go there, and the next step's slices have arrived,
        // so its first fragments are read under the last quarter's products.
        auto step = [&](int stage, auto load, auto next) {
#pragma unroll
            for (int s = 0; s < 3; ++s) {
                read(stage, s + 1);
                multiply(s);
                spread<FM * FN, kReads, 0>();
            }
            if constexpr (decltype(next)::value) {
                arrive();
                if constexpr (decltype(load)::value) issue(stage);
                read(stage ^ 1, 0);
            }
            multiply(3);
            spread<FM * FN, decltype(next)::value ? kReads : 0, decltype(load)::value ? kLoads : 0>();
        };

        const int total = (last - first) * p.segments;
        seek();
        issue(0);
        if (total > 1) {
            seek();
            issue(1);
        }
        arrive();
        read(0, 0);
        int n = 0;
        for (; n + 2 < total; ++n) {
            seek();
            step(n & 1, Yes{}, Yes{});
        }
        if (n + 1 < total) {
            step(n & 1, No{}, Yes{});
            ++n;
        }
        step(n & 1, No{}, No{});
    }
};

}  // namespace m16
}  // namespace tgemm
