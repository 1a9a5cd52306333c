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
// tile_walk.h says how the operands lie in memory and in LDS.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "tile_walk.h"

namespace tgemm {
namespace m16 {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

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

// a·b, where 0 times anything, NaN and infinity too, is 0.
__device__ __forceinline__ float mul_zero(float a, float b)
{
    float r;
    asm("v_mul_legacy_f32 %0, %1, %2" : "=v"(r) : "v"(a), "v"(b));
    return r;
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

// One operand's slices: where this thread's 16-byte pieces come from.
template <class Slice>
struct Loader {
    static constexpr int kRounds = Slice::kRounds;
    uint32_t off[kRounds];

    __device__ __forceinline__ void place(int64_t ld, int mn_last, int k_last)
    {
        const int thread = thread_anew();
#pragma unroll
        for (int r = 0; r < kRounds; ++r) off[r] = Slice::offset(r * Slice::kThreads + thread, ld, mn_last, k_last);
    }

    __device__ __forceinline__ void issue_one(const char *base, lds_char *stage, int wave, int r) const
    {
        load_lds(base, off[r], stage + (r * Slice::kThreads + wave * 64) * 16);
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
// gridDim.x, ...  For each, `epilogue(acc, row0, col0, split, ahead)` is called
// when the lane holds in acc[i][j][r] row row0 + 16·i + lane % 16, column col0 +
// 4·FN·(lane / 16) + 4·j + r.  The loads run two steps ahead without regard to
// where a tile ends, so the next tile's are under way by then; as loads come
// back in order, the epilogue would wait for those with its own.  What it needs
// for its rows is what `prologue(row0, col0)` returned before the products.
// ANEW: a tile's first fragments are read once more where it begins, so that
// the epilogue before it has their registers.
template <class E, int BM, int BN, int WM, int WN, bool A_MC, bool B_MC, class Op = Operands, bool ANEW = false>
struct TileProduct {
    static constexpr int kThreads = 64 * WM * WN;
    static constexpr int FM = BM / WM / 16, FN = BN / WN / 16;
    static constexpr int BK = kStepK;
    static constexpr int kStage = (BM + BN) * BK * 2;
    static constexpr int kLds = 2 * kStage;
    typedef f32x4 Acc[FM][FN];

    template <class Prologue, class Epilogue>
    static __device__ __forceinline__ void run(const Op &p, lds_char *lds, Prologue prologue, Epilogue epilogue)
    {
        const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
        const int wm = wave / WN, wn = wave % WN;
        const int tiles = p.ids();
        typedef Slice<BM, FM, kThreads, A_MC, false> SliceA;
        typedef Slice<BN, FN, kThreads, B_MC, true> SliceB;
        Loader<SliceA> la;
        Loader<SliceB> lb;
        Reader<BM, FM, A_MC, false> ra;
        Reader<BN, FN, B_MC, true> rb;
        ra.place(wm * (FM * 16), lane);
        rb.place(wn * (FN * 16), lane);
        constexpr int kLoadsA = decltype(la)::kRounds, kLoads = kLoadsA + decltype(lb)::kRounds;
        constexpr int kReadsA = FM / 2 * (A_MC ? 2 : 1), kReadsB = FN * (B_MC ? 2 : 1);

        // the loads' way through the tiles
        Walk<BM, BN, A_MC, B_MC, Op> walk;
        walk.begin(p, blockIdx.x);
        auto seek = [&]() {
            const auto moved = walk.seek(p, gridDim.x);
            if (moved.a) la.place(p.lda, walk.a_last, walk.a_k_last);
            if (moved.b) lb.place(p.ldb, walk.b_last, walk.b_k_last);
        };
        // A round of a KC operand may be just the rows that the wavefronts'
        // first (or second) halves are made of.  Early loads: B and those of A.
        constexpr bool kHalves = !A_MC && kThreads / 8 == FM / 2 * 16;
        constexpr int kEarlyA = kHalves ? kLoadsA / 2 : 0, kEarly = kLoads - kLoadsA + kEarlyA;
        auto issue = [&](int stage, int n) {  // the n-th load, early ones first
            lds_char *to = lds + stage * kStage;
            if (n < kEarlyA) la.issue_one(walk.from_a, to, wave, 2 * n);
            else if (n < kEarly) lb.issue_one(walk.from_b, to + BM * BK * 2, wave, n - kEarlyA);
            else la.issue_one(walk.from_a, to, wave, kHalves ? 2 * (n - kEarly) + 1 : n - kEarly);
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
            tile_at<BM, BN>(p, id, m0, n0, split, from, to);
            const int row0 = m0 + wm * (FM * 16), col0 = n0 + wn * (FN * 16);
            const auto ahead = prologue(row0, col0);
            if constexpr (ANEW) read(stage, 0);
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
            epilogue(acc, row0, col0, split, ahead);
        }
        __builtin_amdgcn_s_waitcnt(0x0F70);  // vmcnt(0): no load into LDS outlives the work-group
    }
};

}  // namespace m16
}  // namespace tgemm
