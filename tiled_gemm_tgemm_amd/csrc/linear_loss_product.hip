// The products of the loss operators: logits reduced to row statistics, a
// piece of the logits' gradient, and the two gradients.  See mfma16.h for the
// tiles.
#include "linear_loss.h"
#include "mfma16.h"

namespace tgemm {
namespace loss {
namespace {

using m16::f32x4;
using m16::lds_char;
using m16::Operands;
using m16::TileProduct;

constexpr float kLog2e = 1.44269504088896340736f;

// A row's adjacent columns that a lane holds.
template <class Tile>
constexpr int kHeld = 4 * Tile::FN;

__device__ __forceinline__ uint32_t pack(__bf16 a, __bf16 b)
{
    return (uint32_t)__builtin_bit_cast(uint16_t, a) | (uint32_t)__builtin_bit_cast(uint16_t, b) << 16;
}
__device__ __forceinline__ uint32_t pack(_Float16 a, _Float16 b)
{
    return (uint32_t)__builtin_bit_cast(uint16_t, a) | (uint32_t)__builtin_bit_cast(uint16_t, b) << 16;
}

// Device memory takes 16-byte stores at any address.
typedef uint32_t u32x4_anywhere __attribute__((ext_vector_type(4), aligned(2)));
typedef f32x4 f32x4_anywhere __attribute__((aligned(4)));

// N (a multiple of 8) adjacent values as 16-bit numbers.
template <class E, int N>
__device__ __forceinline__ void store_packed(E *to, const float (&v)[N])
{
#pragma unroll
    for (int q = 0; q < N / 8; ++q) {
        uint32_t w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) w[e] = pack((E)v[8 * q + 2 * e], (E)v[8 * q + 2 * e + 1]);
        reinterpret_cast<u32x4_anywhere *>(to)[q] = u32x4_anywhere{w[0], w[1], w[2], w[3]};
    }
}

// N adjacent values of a row of the result, `left` of them inside it.
template <class T, int N>
__device__ __forceinline__ void store_row(T *to, const float (&v)[N], int left)
{
    if (left >= N) {
        if constexpr (sizeof(T) == 2) {
            store_packed<T, N>(to, v);
        } else {
#pragma unroll
            for (int q = 0; q < N / 4; ++q) {
                f32x4 w;
#pragma unroll
                for (int e = 0; e < 4; ++e) w[e] = v[4 * q + e];
                reinterpret_cast<f32x4_anywhere *>(to)[q] = w;
            }
        }
    } else {
#pragma unroll
        for (int e = 0; e < N; ++e)
            if (e < left) to[e] = (T)v[e];
    }
}

// The four lanes that share a row (16 apart) exchange their four times four
// columns, so that what they store at once lies side by side: lane q's v[j]
// becomes lane j's v[q].
__device__ __forceinline__ void turn(f32x4 (&v)[4])
{
    auto word = [](float f) { return __builtin_bit_cast(uint32_t, f); };
    auto value = [](uint32_t w) { return __builtin_bit_cast(float, w); };
#pragma unroll
    for (int e = 0; e < 4; ++e) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {  // lanes 2, 3 of one and 0, 1 of the other
            const auto r = __builtin_amdgcn_permlane32_swap(word(v[j][e]), word(v[j + 2][e]), false, false);
            v[j][e] = value(r[0]);
            v[j + 2][e] = value(r[1]);
        }
#pragma unroll
        for (int j = 0; j < 4; j += 2) {  // lanes 1, 3 of one and 0, 2 of the other
            const auto r = __builtin_amdgcn_permlane16_swap(word(v[j][e]), word(v[j + 1][e]), false, false);
            v[j][e] = value(r[0]);
            v[j + 1][e] = value(r[1]);
        }
    }
}

// Row statistics of the logits: a tile's logits never leave the registers (but
// for the copy that the backward pass may ask for); a row's maximum and sum
// over 64 columns take the lane's own 16 values and two exchanges with the
// three lanes that hold the rest, 8 bytes a row and column group in all.
// Columns past the last of the vocabulary do not count.  Bound by the matrix
// cores and what the GPU's power lets them run at: 4096×32768×2048 bf16 takes
// 436 µs (1.26 PFLOP/s), of which the exponentials are 20 and the loads' way
// through LDS 80; 4096×32000×4096 790 with the join.  The copy of the logits
// adds 160 µs for 537 MB: loads and stores come back in order, so the next
// tile's loads wait for it.
template <class E, int BM, int BN, int WM, int WN>
__global__ __launch_bounds__(64 * WM * WN) void linear_stats_kernel(StatsArgs a)
{
    typedef TileProduct<E, BM, BN, WM, WN, false, false> Tile;
    constexpr int H = kHeld<Tile>;
    __shared__ __align__(1024) char lds[Tile::kLds];
    const float scale2 = a.scale * kLog2e;
    // a row's target, as this lane's column (negative: another's), or where its
    // entries in this column group start (low half) and end
    struct Ahead {
        int what[Tile::FM];
    };
    auto prologue = [&](int row0, int col0) {
        const int lane = m16::thread_anew() & 63, l16 = lane & 15, quarter = lane >> 4;
        Ahead ahead;
        const int group = col0 / (Tile::FN * 16);
#pragma unroll
        for (int i = 0; i < Tile::FM; ++i) {
            const int64_t row = min(row0 + i * 16 + l16, a.op.M - 1);
            ahead.what[i] = 0;
            if (a.target != nullptr) {
                const int64_t y = a.target[row];
                ahead.what[i] = y >= 0 && y < a.op.N ? (int)y - (col0 + H * quarter) : -1;
            } else if (group < a.groups) {
                const uint16_t *from = a.starts + row * (a.groups + 1) + group;
                ahead.what[i] = from[0] | (int)from[1] << 16;
            }
        }
        return ahead;
    };
    Tile::run(a.op, (lds_char *)lds, prologue, [&](typename Tile::Acc &acc, int row0, int col0, int, const Ahead &ahead) {
        const int lane = m16::thread_anew() & 63, l16 = lane & 15, quarter = lane >> 4;
        const int left = a.op.N - (col0 + H * quarter);  // this lane's columns that exist
        if (a.logits != nullptr) {
#pragma unroll
            for (int i = 0; i < Tile::FM; ++i) {
                const int row = row0 + i * 16 + l16;
                f32x4 v[Tile::FN];
#pragma unroll
                for (int j = 0; j < Tile::FN; ++j) v[j] = acc[i][j];
                if constexpr (Tile::FN == 4) turn(v);
                if (row >= a.op.M) continue;
#pragma unroll
                for (int j = 0; j < Tile::FN; ++j) {
                    const int col = col0 + (Tile::FN == 4 ? 16 * j + 4 * quarter : H * quarter + 4 * j);
                    const float one[4] = {v[j][0], v[j][1], v[j][2], v[j][3]};
                    store_row<float, 4>(a.logits + (int64_t)row * a.ldz + col, one, a.op.N - col);
                }
            }
        }
        if (a.op.N - col0 < Tile::FN * 16) {
#pragma unroll
            for (int i = 0; i < Tile::FM; ++i)
#pragma unroll
                for (int e = 0; e < H; ++e)
                    if (e >= left) acc[i][e / 4][e % 4] = -INFINITY;
        }
        const int group = col0 / (Tile::FN * 16);
        if (a.target != nullptr) {
#pragma unroll
            for (int i = 0; i < Tile::FM; ++i) {
                const int row = row0 + i * 16 + l16, want = ahead.what[i];
                if (row >= a.op.M || want < 0 || want >= H) continue;
                float z = 0.0f;
#pragma unroll
                for (int e = 0; e < H; ++e) z = want == e ? acc[i][e / 4][e % 4] : z;
                a.picked[row] = z * a.scale;
            }
        } else if (group < a.groups) {
            // the first entry of every row at once: most have one or none
            uint32_t entry[Tile::FM];
#pragma unroll
            for (int i = 0; i < Tile::FM; ++i) {
                const int row = row0 + i * 16 + l16, from = ahead.what[i] & 0xFFFF, to = ahead.what[i] >> 16;
                entry[i] = 0;
                if (row < a.op.M && from < to) entry[i] = a.list[(int64_t)row * a.K + from];
            }
#pragma unroll
            for (int i = 0; i < Tile::FM; ++i) {
                const int row = row0 + i * 16 + l16, from = ahead.what[i] & 0xFFFF, to = row < a.op.M ? ahead.what[i] >> 16 : 0;
                const int64_t base = (int64_t)row * a.K;
                for (int c = from; c < to; ++c) {
                    const uint32_t what = c == from ? entry[i] : a.list[base + c];
                    const int e = (int)(what & 255) - H * quarter;
                    if (e < 0 || e >= H) continue;
                    float z = 0.0f;
#pragma unroll
                    for (int j = 0; j < H; ++j) z = e == j ? acc[i][j / 4][j % 4] : z;
                    a.student[base + (what >> 8)] = z * a.scale;
                }
            }
        }
        // the scale is positive, so the largest product is the largest logit
        float high[Tile::FM], sum[Tile::FM];
#pragma unroll
        for (int i = 0; i < Tile::FM; ++i) {
            high[i] = acc[i][0][0];
#pragma unroll
            for (int e = 1; e < H; ++e) high[i] = fmaxf(high[i], acc[i][e / 4][e % 4]);
        }
#pragma unroll
        for (int i = 0; i < Tile::FM; ++i) high[i] = fmaxf(high[i], __shfl_xor(high[i], 16));
#pragma unroll
        for (int i = 0; i < Tile::FM; ++i) high[i] = fmaxf(high[i], __shfl_xor(high[i], 32)) * scale2;
#pragma unroll
        for (int i = 0; i < Tile::FM; ++i) {
            const float from = high[i] == -INFINITY ? 0.0f : high[i];
            sum[i] = 0.0f;
#pragma unroll
            for (int e = 0; e < H; ++e) sum[i] += __builtin_amdgcn_exp2f(fmaf(acc[i][e / 4][e % 4], scale2, -from));
        }
#pragma unroll
        for (int i = 0; i < Tile::FM; ++i) sum[i] += __shfl_xor(sum[i], 16);
#pragma unroll
        for (int i = 0; i < Tile::FM; ++i) sum[i] += __shfl_xor(sum[i], 32);
        if (quarter == 0 && group < a.groups) {
#pragma unroll
            for (int i = 0; i < Tile::FM; ++i) {
                const int row = row0 + i * 16 + l16;
                if (row < a.op.M) a.part[(int64_t)row * a.groups + group] = make_float2(high[i], sum[i]);
            }
        }
    });
}

// A piece of the logits' gradient: the product as above, then coef·(exp(z -
// lse) - [the target]) rounded once.  Bound as the statistics are, and by its
// stores: 4096×32768×2048 bf16 takes 470 µs (1.17 PFLOP/s, 268 MB written).
template <class E, int BM, int BN, int WM, int WN>
__global__ __launch_bounds__(64 * WM * WN) void linear_grad_kernel(GradArgs a)
{
    typedef TileProduct<E, BM, BN, WM, WN, false, false> Tile;
    constexpr int H = kHeld<Tile>;
    __shared__ __align__(1024) char lds[Tile::kLds];
    // a row's factor, its logarithm of the sum, and its target as this lane's
    // column (negative: another's)
    struct Ahead {
        float coef[Tile::FM], lse[Tile::FM];
        int want[Tile::FM];
    };
    auto prologue = [&](int row0, int col0) {
        const int lane = m16::thread_anew() & 63, l16 = lane & 15, quarter = lane >> 4;
        Ahead ahead;
#pragma unroll
        for (int i = 0; i < Tile::FM; ++i) {
            const int row = min(row0 + i * 16 + l16, a.op.M - 1);
            ahead.coef[i] = a.coef[row];
            ahead.lse[i] = a.lse[row];
            ahead.want[i] = -1;
            if (a.target != nullptr) {
                const int64_t y = a.target[row] - a.v0;
                if (y >= 0 && y < a.op.N) ahead.want[i] = (int)y - (col0 + H * quarter);
            }
        }
        return ahead;
    };
    Tile::run(a.op, (lds_char *)lds, prologue, [&](typename Tile::Acc &acc, int row0, int col0, int, const Ahead &ahead) {
        const int lane = m16::thread_anew() & 63, l16 = lane & 15, quarter = lane >> 4;
        const int col = col0 + H * quarter;
        if (col >= a.ldg) return;
#pragma unroll
        for (int i = 0; i < Tile::FM; ++i) {
            const int row = row0 + i * 16 + l16;
            if (row >= a.rows) continue;
            const bool real = row < a.op.M;
            const float c = real ? ahead.coef[i] : 0.0f;
            const float lse = !real ? 0.0f : c == c ? ahead.lse[i] : c;
            const int want = ahead.want[i];
            float g[H];
            // in 16 bits the exponent's argument may be rounded once more
            if (a.planes == 1) {
                const float scale2 = a.scale * kLog2e, lse2 = lse * kLog2e;
#pragma unroll
                for (int e = 0; e < H; ++e) g[e] = __builtin_amdgcn_exp2f(fmaf(acc[i][e / 4][e % 4], scale2, -lse2));
            } else {
#pragma unroll
                for (int e = 0; e < H; ++e) g[e] = __builtin_amdgcn_exp2f(fmaf(acc[i][e / 4][e % 4], a.scale, -lse) * kLog2e);
            }
            if (want >= 0 && want < H) {
#pragma unroll
                for (int e = 0; e < H; ++e) g[e] = want == e ? g[e] - 1.0f : g[e];
            }
            if (col + H > a.op.N) {
#pragma unroll
                for (int e = 0; e < H; ++e) g[e] = col + e < a.op.N ? g[e] : 0.0f;
            }
            // 0 times anything is 0 here: a row that does not count is zero
            // whatever its logits are
#pragma unroll
            for (int e = 0; e < H; ++e) g[e] = m16::mul_zero(c, g[e]);
            E *to = (E *)a.G + (int64_t)row * a.ldg + col;
            if (a.planes == 1) {
                store_packed<E, H>(to, g);
            } else {
#pragma unroll
                for (int q = 0; q < 3; ++q) {
                    if (q == a.planes) break;
                    store_packed<E, H>(to + q * a.plane, g);
#pragma unroll
                    for (int e = 0; e < H; ++e) g[e] -= (float)(E)g[e];
                }
            }
        }
    });
}

// The two products with the logits' gradient, with the sum split where their
// tiles would not fill the GPU (dX: few rows and a long sum), as the time model
// of the entry points decides.  B and dW's A are read as they lie, through the
// transposing LDS read, instead of being transposed in memory first.  Bound by
// the matrix cores: 4096×32768×2048 bf16 takes 435 µs for either (1.26
// PFLOP/s; the library's products of such operands 1.22 and 1.09).
template <class E, int BM, int BN, int WM, int WN, bool A_MC>
__global__ __launch_bounds__(64 * WM * WN) void linear_out_kernel(OutArgs a)
{
    typedef TileProduct<E, BM, BN, WM, WN, A_MC, true> Tile;
    constexpr int H = kHeld<Tile>;
    __shared__ __align__(1024) char lds[Tile::kLds];
    const bool scaled = a.row_scale != nullptr || a.all_scale != nullptr;
    const float all = a.all_scale != nullptr ? *a.all_scale : 1.0f;
    struct Ahead {};
    Tile::run(a.op, (lds_char *)lds, [](int, int) { return Ahead{}; },
              [&](typename Tile::Acc &acc, int row0, int col0, int split, Ahead) {
        const int lane = m16::thread_anew() & 63, l16 = lane & 15, quarter = lane >> 4;
        const int col = col0 + H * quarter, left = a.op.N - col;
        if (left <= 0) return;
#pragma unroll
        for (int i = 0; i < Tile::FM; ++i) {
            const int row = row0 + i * 16 + l16;
            if (row >= a.op.M || (row & (a.period - 1)) >= a.kept) continue;
            float v[H];
#pragma unroll
            for (int e = 0; e < H; ++e) v[e] = acc[i][e / 4][e % 4];
            if (scaled) {
                const float s = a.row_scale != nullptr ? a.row_scale[row] : all;
#pragma unroll
                for (int e = 0; e < H; ++e) v[e] = m16::mul_zero(s, v[e]);
            }
            const int64_t at = (int64_t)row * a.ldo + col + (int64_t)split * a.split_stride;
            if (a.dtype == TGEMM_F32) {
                float *to = (float *)a.out + at;
                if (a.add) {
#pragma unroll
                    for (int e = 0; e < H; ++e)
                        if (e < left) v[e] += to[e];
                }
                store_row<float, H>(to, v, left);
            } else {
                store_row<E, H>((E *)a.out + at, v, left);
            }
        }
    });
}

// The logits' gradient from logits that were kept, eight columns a thread; a
// work-group stays in a row.  Bound by memory: 4096×32768 bf16 reads 537 MB and
// writes 268 in 152 µs (5.3 TB/s).
template <class E>
__global__ __launch_bounds__(256) void linear_grad_kept_kernel(GradArgs a, const float *logits, int64_t ldz,
                                                               int64_t blocks, int per_row)
{
    typedef float f32x8 __attribute__((ext_vector_type(8)));
    typedef f32x8 f32x8_anywhere __attribute__((aligned(4)));
    const int whole = (a.op.N + 63) / 64 * 64;
    const float scale2 = a.scale * kLog2e;
    for (int64_t b = blockIdx.x; b < blocks; b += gridDim.x) {
        const int row = (int)(b / per_row), col = (int)(b % per_row) * 2048 + threadIdx.x * 8;
        if (col >= whole) continue;
        const float c = row < a.op.M ? a.coef[row] : 0.0f;
        float g[8] = {};
        if (c != 0.0f) {  // a row that does not count is zero whatever its logits are
            const float lse = c == c ? a.lse[row] : c, lse2 = lse * kLog2e;
            const int64_t y = a.target != nullptr ? a.target[row] - a.v0 - col : -1;
            const float *from = logits + row * ldz + col;
            f32x8 z{};
            if (col + 8 <= a.op.N) {
                z = *(const f32x8_anywhere *)from;
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if (col + e < a.op.N) z[e] = from[e];
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float x = a.planes == 1 ? fmaf(z[e], scale2, -lse2) : fmaf(z[e], a.scale, -lse) * kLog2e;
                float p = __builtin_amdgcn_exp2f(x);
                if (e == y) p -= 1.0f;
                g[e] = col + e < a.op.N ? m16::mul_zero(c, p) : 0.0f;
            }
        }
        E *to = (E *)a.G + (int64_t)row * a.ldg + col;
        for (int q = 0; q < a.planes; ++q) {
            store_packed<E, 8>(to + q * a.plane, g);
#pragma unroll
            for (int e = 0; e < 8; ++e) g[e] -= (float)(E)g[e];
        }
    }
}

// As many work-groups as the GPU holds at once (a multiple of 8, so that a
// work-group's tiles stay on its XCD).
template <class Args>
unsigned grid_of(const Args &a, int tile)
{
    const int64_t tiles = (int64_t)a.op.tiles_m * a.op.tiles_n * a.op.splits;
    const int64_t most = (int64_t)256 * kTiles[tile].wg_per_cu;
    return (unsigned)(tiles < most ? tiles : most);
}

}  // namespace

hipError_t launch_stats(bool half, int tile, const StatsArgs &a, hipStream_t stream)
{
    switch (tile) {
#define X(I, BM, BN, WM, WN)                                                                            \
    case I:                                                                                             \
        if (half) linear_stats_kernel<_Float16, BM, BN, WM, WN><<<grid_of(a, I), 64 * WM * WN, 0, stream>>>(a); \
        else linear_stats_kernel<__bf16, BM, BN, WM, WN><<<grid_of(a, I), 64 * WM * WN, 0, stream>>>(a);        \
        break;
        TGEMM_TILES(X)
#undef X
    }
    return hipGetLastError();
}

hipError_t launch_grad(bool half, int tile, const GradArgs &a, hipStream_t stream)
{
    switch (tile) {
#define X(I, BM, BN, WM, WN)                                                                            \
    case I:                                                                                             \
        if (half) linear_grad_kernel<_Float16, BM, BN, WM, WN><<<grid_of(a, I), 64 * WM * WN, 0, stream>>>(a); \
        else linear_grad_kernel<__bf16, BM, BN, WM, WN><<<grid_of(a, I), 64 * WM * WN, 0, stream>>>(a);        \
        break;
        TGEMM_TILES(X)
#undef X
    }
    return hipGetLastError();
}

hipError_t launch_grad_kept(bool half, const GradArgs &a, const float *logits, int64_t ldz, hipStream_t stream)
{
    const int per_row = (a.op.N + 2047) / 2048;
    const int64_t blocks = (int64_t)a.rows * per_row;
    const unsigned grid = (unsigned)(blocks < (1 << 20) ? blocks : 1 << 20);
    if (half) linear_grad_kept_kernel<_Float16><<<grid, 256, 0, stream>>>(a, logits, ldz, blocks, per_row);
    else linear_grad_kept_kernel<__bf16><<<grid, 256, 0, stream>>>(a, logits, ldz, blocks, per_row);
    return hipGetLastError();
}

hipError_t launch_dx(bool half, int tile, const OutArgs &a, hipStream_t stream)
{
    switch (tile) {
#define X(I, BM, BN, WM, WN)                                                                                     \
    case I:                                                                                                      \
        if (half) linear_out_kernel<_Float16, BM, BN, WM, WN, false><<<grid_of(a, I), 64 * WM * WN, 0, stream>>>(a); \
        else linear_out_kernel<__bf16, BM, BN, WM, WN, false><<<grid_of(a, I), 64 * WM * WN, 0, stream>>>(a);        \
        break;
        TGEMM_TILES(X)
#undef X
    }
    return hipGetLastError();
}

hipError_t launch_dw(bool half, int tile, const OutArgs &a, hipStream_t stream)
{
    switch (tile) {
#define X(I, BM, BN, WM, WN)                                                                                    \
    case I:                                                                                                     \
        if (half) linear_out_kernel<_Float16, BM, BN, WM, WN, true><<<grid_of(a, I), 64 * WM * WN, 0, stream>>>(a); \
        else linear_out_kernel<__bf16, BM, BN, WM, WN, true><<<grid_of(a, I), 64 * WM * WN, 0, stream>>>(a);        \
        break;
        TGEMM_TILES(X)
#undef X
    }
    return hipGetLastError();
}

}  // namespace loss
}  // namespace tgemm
