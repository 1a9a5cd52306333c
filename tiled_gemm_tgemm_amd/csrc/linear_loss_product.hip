// The products of the loss operators: logits reduced to row statistics, a
// piece of the logits' gradient, and the two gradients.  See mfma16.h for the
// tiles.
#include "linear_loss.h"

namespace tgemm {
namespace loss {
namespace {

using m16::f32x16;
using m16::f32x4;
using m16::lds_char;
using m16::Operands;
using m16::TileProduct;

constexpr float kLog2e = 1.44269504088896340736f;

// Columns past the last of the vocabulary do not count; a wavefront's
// columns are 16 per lane and block, so a row's maximum and sum take the
// lane's own values and one exchange with the lane of the other half.
template <class E, int BM, int BN, int WM, int WN>
__global__ __launch_bounds__(64 * WM * WN) void linear_stats_kernel(StatsArgs a)
{
    typedef TileProduct<E, BM, BN, WM, WN, false, false, 64, 2> Tile;
    __shared__ __align__(1024) char lds[Tile::kLds];
    Tile t;
    t.run(a.op, (lds_char *)lds);

    const int lane = threadIdx.x & 63, l32 = lane & 31, half = lane >> 5;
    const float scale2 = a.scale * kLog2e;
    const int group = t.col0 / (Tile::FN * 32);
#pragma unroll
    for (int i = 0; i < Tile::FM; ++i) {
        const int row = t.row0 + i * 32 + l32;
        if (a.target != nullptr && row < a.op.M) {
            const int64_t want = a.target[row] - (t.col0 + 16 * half);
#pragma unroll
            for (int j = 0; j < Tile::FN; ++j) {
                const int64_t r = want - j * 32;
                if (r >= 0 && r < 16 && want + t.col0 + 16 * half < a.op.N) {
                    float z = 0.0f;
#pragma unroll
                    for (int e = 0; e < 16; ++e) z = r == e ? t.acc[i][j][e] : z;
                    a.picked[row] = z * a.scale;
                }
            }
        }
        float high = -INFINITY;
#pragma unroll
        for (int j = 0; j < Tile::FN; ++j)
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                const float z = t.col0 + j * 32 + 16 * half + r < a.op.N ? t.acc[i][j][r] * scale2 : -INFINITY;
                t.acc[i][j][r] = z;
                high = fmaxf(high, z);
            }
        high = fmaxf(high, __shfl_xor(high, 32));
        const float from = high == -INFINITY ? 0.0f : high;
        float sum = 0.0f;
#pragma unroll
        for (int j = 0; j < Tile::FN; ++j)
#pragma unroll
            for (int r = 0; r < 16; ++r) sum += __builtin_amdgcn_exp2f(t.acc[i][j][r] - from);
        sum += __shfl_xor(sum, 32);
        if (half == 0 && row < a.op.M && group < a.groups)
            a.part[(int64_t)row * a.groups + group] = make_float2(high, sum);
    }
}

__device__ __forceinline__ uint32_t pack(__bf16 a, __bf16 b)
{
    return (uint32_t)__builtin_bit_cast(uint16_t, a) | (uint32_t)__builtin_bit_cast(uint16_t, b) << 16;
}
__device__ __forceinline__ uint32_t pack(_Float16 a, _Float16 b)
{
    return (uint32_t)__builtin_bit_cast(uint16_t, a) | (uint32_t)__builtin_bit_cast(uint16_t, b) << 16;
}

template <class E>
__device__ __forceinline__ void store16(E *to, const float (&v)[16])
{
    uint32_t w[8];
#pragma unroll
    for (int q = 0; q < 8; ++q) w[q] = pack((E)v[2 * q], (E)v[2 * q + 1]);
    uint4 *p = reinterpret_cast<uint4 *>(to);
    p[0] = make_uint4(w[0], w[1], w[2], w[3]);
    p[1] = make_uint4(w[4], w[5], w[6], w[7]);
}

template <class E, int BM, int BN, int WM, int WN>
__global__ __launch_bounds__(64 * WM * WN) void linear_grad_kernel(GradArgs a)
{
    typedef TileProduct<E, BM, BN, WM, WN, false, false, 64, 2> Tile;
    __shared__ __align__(1024) char lds[Tile::kLds];
    Tile t;
    t.run(a.op, (lds_char *)lds);

    const int lane = threadIdx.x & 63, l32 = lane & 31, half = lane >> 5;
#pragma unroll
    for (int i = 0; i < Tile::FM; ++i) {
        const int row = t.row0 + i * 32 + l32;
        if (row >= a.rows) continue;
        const bool real = row < a.op.M;
        const float c = real ? a.coef[row] : 0.0f;
        const float lse = real ? a.lse[row] : 0.0f;
        const int64_t want = real && a.target != nullptr ? a.target[row] - a.v0 : -1;
#pragma unroll
        for (int j = 0; j < Tile::FN; ++j) {
            const int col = t.col0 + j * 32 + 16 * half;
            if (col >= a.ldg) continue;
            float g[16];
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                const float p = __builtin_amdgcn_exp2f(fmaf(t.acc[i][j][r], a.scale, -lse) * kLog2e);
                // a row that does not count is zero whatever its logits are
                g[r] = c != 0.0f && col + r < a.op.N ? c * (col + r == want ? p - 1.0f : p) : 0.0f;
            }
            E *to = (E *)a.G + (int64_t)row * a.ldg + col;
            if constexpr (sizeof(E) == 2) {
                if (a.planes == 1) {
                    store16<E>(to, g);
                } else {
#pragma unroll
                    for (int q = 0; q < 3; ++q) {
                        store16<E>(to + q * a.plane, g);
#pragma unroll
                        for (int r = 0; r < 16; ++r) g[r] -= (float)(E)g[r];
                    }
                }
            }
        }
    }
}

// 16 adjacent values of a row of the result, `left` of them inside it.
template <class T>
__device__ __forceinline__ void store_row(T *to, const float (&v)[16], int left, bool vec)
{
    if (vec && left >= 16) {
        if constexpr (sizeof(T) == 2) {
            store16<T>(to, v);
        } else {
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                f32x4 w;
#pragma unroll
                for (int e = 0; e < 4; ++e) w[e] = v[4 * q + e];
                reinterpret_cast<f32x4 *>(to)[q] = w;
            }
        }
    } else {
#pragma unroll
        for (int r = 0; r < 16; ++r)
            if (r < left) to[r] = (T)v[r];
    }
}

template <class E, int BM, int BN, int WM, int WN, bool A_MC>
__global__ __launch_bounds__(64 * WM * WN) void linear_out_kernel(OutArgs a)
{
    typedef TileProduct<E, BM, BN, WM, WN, A_MC, true, BM >= 128 ? 32 : 64, BM >= 128 ? 4 : 2> Tile;
    __shared__ __align__(1024) char lds[Tile::kLds];
    Tile t;
    t.run(a.op, (lds_char *)lds);

    const int lane = threadIdx.x & 63, l32 = lane & 31, half = lane >> 5;
    const float all = a.all_scale != nullptr ? *a.all_scale : 1.0f;
#pragma unroll
    for (int i = 0; i < Tile::FM; ++i) {
        const int row = t.row0 + i * 32 + l32;
        if (row >= a.op.M) continue;
        const float s = a.row_scale != nullptr ? a.row_scale[row] * all : all;
#pragma unroll
        for (int j = 0; j < Tile::FN; ++j) {
            const int col = t.col0 + j * 32 + 16 * half;
            const int left = a.op.N - col;
            if (left <= 0) continue;
            float v[16];
#pragma unroll
            for (int r = 0; r < 16; ++r) v[r] = t.acc[i][j][r] * s;
            const int64_t at = (int64_t)row * a.ldo + col + (int64_t)t.split * a.split_stride;
            if (a.dtype == TGEMM_F32) {
                float *to = (float *)a.out + at;
                if (a.add) {
#pragma unroll
                    for (int r = 0; r < 16; ++r)
                        if (r < left) v[r] += to[r];
                }
                store_row<float>(to, v, left, a.vec);
            } else {
                store_row<E>((E *)a.out + at, v, left, a.vec);
            }
        }
    }
}

constexpr TileShape kTiles[] = {
    {256, 256, 1, 64},
    {128, 128, 2, 64},
    {32, 128, 3, 32},
};

#define TGEMM_TILES(X) X(0, 256, 256, 2, 4) X(1, 128, 128, 2, 2) X(2, 32, 128, 1, 4)

template <class Args>
unsigned grid_of(const Args &a, int splits) { return (unsigned)(a.op.tiles_m * a.op.tiles_n) * (unsigned)splits; }

}  // namespace

int tile_count() { return (int)(sizeof(kTiles) / sizeof(kTiles[0])); }
const TileShape &tile_shape(int index) { return kTiles[index]; }

hipError_t launch_stats(bool half, int tile, const StatsArgs &a, hipStream_t stream)
{
    switch (tile) {
#define X(I, BM, BN, WM, WN)                                                                            \
    case I:                                                                                             \
        if (half) linear_stats_kernel<_Float16, BM, BN, WM, WN><<<grid_of(a, 1), 64 * WM * WN, 0, stream>>>(a); \
        else linear_stats_kernel<__bf16, BM, BN, WM, WN><<<grid_of(a, 1), 64 * WM * WN, 0, stream>>>(a);        \
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
        if (half) linear_grad_kernel<_Float16, BM, BN, WM, WN><<<grid_of(a, 1), 64 * WM * WN, 0, stream>>>(a); \
        else linear_grad_kernel<__bf16, BM, BN, WM, WN><<<grid_of(a, 1), 64 * WM * WN, 0, stream>>>(a);        \
        break;
        TGEMM_TILES(X)
#undef X
    }
    return hipGetLastError();
}

hipError_t launch_dx(bool half, int tile, const OutArgs &a, hipStream_t stream)
{
    switch (tile) {
#define X(I, BM, BN, WM, WN)                                                                                     \
    case I:                                                                                                      \
        if (half) linear_out_kernel<_Float16, BM, BN, WM, WN, false><<<grid_of(a, a.splits), 64 * WM * WN, 0, stream>>>(a); \
        else linear_out_kernel<__bf16, BM, BN, WM, WN, false><<<grid_of(a, a.splits), 64 * WM * WN, 0, stream>>>(a);        \
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
        if (half) linear_out_kernel<_Float16, BM, BN, WM, WN, true><<<grid_of(a, a.splits), 64 * WM * WN, 0, stream>>>(a); \
        else linear_out_kernel<__bf16, BM, BN, WM, WN, true><<<grid_of(a, a.splits), 64 * WM * WN, 0, stream>>>(a);        \
        break;
        TGEMM_TILES(X)
#undef X
    }
    return hipGetLastError();
}

}  // namespace loss
}  // namespace tgemm
