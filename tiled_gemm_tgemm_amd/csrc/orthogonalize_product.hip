// The products of the Newton-Schulz operator on 16-bit tiles (mfma16.h): S =
// X·Xᵀ, Q = b·S + c·S·S and a·X + Q·X (or Q = a + b·S + c·S·S and Q·X), each with
// its sum and the split into planes in the epilogue.
#include "mfma16.h"
#include "mfma16_store.h"
#include "orthogonalize.h"

namespace tgemm {
namespace ortho {
namespace {

using m16::f32x4;
using m16::kHeld;
using m16::lds_char;
using m16::store_packed;
using m16::store_row;
using m16::TileProduct;

typedef _Float16 f16x8_anywhere __attribute__((ext_vector_type(8), aligned(2)));

// Bound by the matrix cores where sums are long (Q·X of 8192×8192 in three
// products of planes 2440 µs, 1.35 PFLOP/s), otherwise by the planes' way in
// the epilogue besides (of 8×1024×4096 193, 1.07 PFLOP/s; 268 MB).  S and Q are
// symmetric: where that takes fewer rounds, only the tiles on and below the
// diagonal are formed and each is stored a second time across it.
template <int BM, int BN, int WM, int WN, bool A_MC, bool B_MC>
__global__ __launch_bounds__(64 * WM * WN) void chain_kernel(ChainArgs a)
{
    typedef TileProduct<_Float16, BM, BN, WM, WN, A_MC, B_MC, Chain, BM == 256> Tile;
    constexpr int H = kHeld<Tile>;
    __shared__ __align__(1024) char lds[Tile::kLds];
    struct Ahead {};
    Tile::run(a.op, (lds_char *)lds, [](int, int) { return Ahead{}; },
              [&](typename Tile::Acc &acc, int row0, int col0, int split, Ahead) {
        const int lane = m16::thread_anew() & 63, l16 = lane & 15, quarter = lane >> 4;
        const int col = col0 + H * quarter;
        if (a.op.splits > 1) {
            float *to = a.parts + (int64_t)(split - a.op.from * a.op.splits) * (BM * BN) + row0 % BM * BN + col % BN;
#pragma unroll
            for (int i = 0; i < Tile::FM; ++i) {
                float v[H];
#pragma unroll
                for (int e = 0; e < H; ++e) v[e] = acc[i][e / 4][e % 4];
                store_row<float, H>(to + (i * 16 + l16) * BN, v, H);
            }
            return;
        }
        const int matrix = a.op.matrix(split);
        const bool mirrored = a.op.lower && row0 / BM != col0 / BN;
#pragma unroll
        for (int i = 0; i < Tile::FM; ++i) {
            const int row = row0 + i * 16 + l16;
            float v[H];
#pragma unroll
            for (int e = 0; e < H; ++e) v[e] = fmaf(a.beta, acc[i][e / 4][e % 4], row == col + e ? a.diagonal : 0.0f);
            if (a.add != nullptr && row < a.op.M && col < a.ld_add) {
                const _Float16 *from = (const _Float16 *)a.add + matrix * a.batch_add + (int64_t)row * a.ld_add + col;
#pragma unroll
                for (int q = 0; q < H / 8; ++q) {
                    const f16x8_anywhere high = ((const f16x8_anywhere *)from)[q];
                    const f16x8_anywhere low = ((const f16x8_anywhere *)(from + a.plane_add))[q];
#pragma unroll
                    for (int e = 0; e < 8; ++e) v[8 * q + e] = fmaf(a.alpha, (float)high[e] + (float)low[e], v[8 * q + e]);
                }
            }
            if (a.planes == nullptr) {
                if (row >= a.op.M) continue;
#pragma unroll
                for (int e = 0; e < H; ++e) v[e] *= 1.0f / (1 << kShift);
                const int64_t at = matrix * a.batch_r + (int64_t)row * a.ldr + col;
                if (a.dtype == TGEMM_F32) store_row<float, H>((float *)a.result + at, v, a.op.N - col);
                else if (a.dtype == TGEMM_BF16) store_row<__bf16, H>((__bf16 *)a.result + at, v, a.op.N - col);
                else store_row<_Float16, H>((_Float16 *)a.result + at, v, a.op.N - col);
                continue;
            }
#pragma unroll
            for (int e = 0; e < H; ++e) v[e] = row < a.op.M && col + e < a.op.N ? v[e] : 0.0f;
            _Float16 *to = (_Float16 *)a.planes + matrix * a.batch_out;
            float low[H];
#pragma unroll
            for (int e = 0; e < H; ++e) low[e] = v[e] - (float)(_Float16)v[e];
            if (row < a.rows && col < a.ldo) {
                store_packed<_Float16, H>(to + (int64_t)row * a.ldo + col, v);
                store_packed<_Float16, H>(to + a.plane_out + (int64_t)row * a.ldo + col, low);
            }
            if (mirrored && row < a.ldo) {
#pragma unroll
                for (int e = 0; e < H; ++e) {
                    if (col + e < a.rows) {
                        _Float16 *across = to + (int64_t)(col + e) * a.ldo + row;
                        across[0] = (_Float16)v[e];
                        across[a.plane_out] = (_Float16)low[e];
                    }
                }
            }
        }
    });
}

// The rest of a tile whose sum came in parts, 64×64 entries a work-group, four
// adjacent ones a thread and round; across the diagonal through LDS.  Bound by
// reading the parts (those of 8192×8192's last tiles 13 µs, of 1000×1000 in
// seven 8).
template <int SIDE>
__global__ __launch_bounds__(256) void chain_join_kernel(ChainArgs a)
{
    constexpr int kPer = SIDE / 64;
    __shared__ _Float16 across[2][64][66];
    typedef _Float16 f16x4 __attribute__((ext_vector_type(4)));
    typedef f16x4 f16x4_anywhere __attribute__((aligned(2)));
    const int number = a.op.from + blockIdx.x / (kPer * kPer), block = blockIdx.x % (kPer * kPer);
    const int matrix = number / a.op.tiles();
    int tm, tn;
    a.op.spot(number % a.op.tiles(), tm, tn);
    const int in_row = block / kPer * 64, in_col = block % kPer * 64, row0 = tm * SIDE + in_row, col0 = tn * SIDE + in_col;
    const bool mirrored = a.op.lower && tm != tn;
    const float *from = a.parts + (int64_t)(number - a.op.from) * a.op.splits * (SIDE * SIDE);
    _Float16 *to = (_Float16 *)a.planes + matrix * a.batch_out;
#pragma unroll
    for (int n = 0; n < 4; ++n) {
        const int r = n * 16 + threadIdx.x / 16, c = threadIdx.x % 16 * 4, row = row0 + r, col = col0 + c;
        const float *part = from + (in_row + r) * SIDE + in_col + c;
        f32x4 sum = *(const f32x4 *)part;
        for (int s = 1; s < a.op.splits; s += 4) {
            f32x4 next[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) next[u] = s + u < a.op.splits ? *(const f32x4 *)(part + (s + u) * (SIDE * SIDE)) : f32x4{};
#pragma unroll
            for (int u = 0; u < 4; ++u) sum += next[u];
        }
        float v[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = fmaf(a.beta, sum[e], row == col + e ? a.diagonal : 0.0f);
        if (a.add != nullptr && row < a.op.M && col < a.ld_add) {
            const _Float16 *plane = (const _Float16 *)a.add + matrix * a.batch_add + (int64_t)row * a.ld_add + col;
            const f16x4 high = *(const f16x4_anywhere *)plane, low = *(const f16x4_anywhere *)(plane + a.plane_add);
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = fmaf(a.alpha, (float)high[e] + (float)low[e], v[e]);
        }
        if (a.planes == nullptr) {
            if (row >= a.op.M) continue;
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] *= 1.0f / (1 << kShift);
            const int64_t at = matrix * a.batch_r + (int64_t)row * a.ldr + col;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                if (col + e >= a.op.N) continue;
                if (a.dtype == TGEMM_F32) ((float *)a.result)[at + e] = v[e];
                else if (a.dtype == TGEMM_BF16) ((__bf16 *)a.result)[at + e] = (__bf16)v[e];
                else ((_Float16 *)a.result)[at + e] = (_Float16)v[e];
            }
            continue;
        }
        f16x4 high, low;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float x = row < a.op.M && col + e < a.op.N ? v[e] : 0.0f;
            high[e] = (_Float16)x;
            low[e] = (_Float16)(x - (float)high[e]);
        }
        if (row < a.rows && col < a.ldo) {
            *(f16x4_anywhere *)(to + (int64_t)row * a.ldo + col) = high;
            *(f16x4_anywhere *)(to + a.plane_out + (int64_t)row * a.ldo + col) = low;
        }
        if (mirrored) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                across[0][c + e][r] = high[e];
                across[1][c + e][r] = low[e];
            }
        }
    }
    if (!mirrored) return;
    __syncthreads();
#pragma unroll
    for (int n = 0; n < 4; ++n) {
        const int r = n * 16 + threadIdx.x / 16, c = threadIdx.x % 16 * 4, row = col0 + r, col = row0 + c;
        if (row >= a.rows || col >= a.ldo) continue;
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            f16x4 w;
#pragma unroll
            for (int e = 0; e < 4; ++e) w[e] = across[q][r][c + e];
            *(f16x4_anywhere *)(to + q * a.plane_out + (int64_t)row * a.ldo + col) = w;
        }
    }
}

}  // namespace

hipError_t launch_chain(Order order, int tile, const ChainArgs &a, hipStream_t stream)
{
    const int64_t ids = a.op.ids(), most = (int64_t)256 * kTiles[tile].wg_per_cu;
    const unsigned grid = (unsigned)(ids < most ? ids : most);
    switch (tile) {
#define X(I, BM, BN, WM, WN)                                                                                        \
    case I:                                                                                                         \
        if (order == kRows) chain_kernel<BM, BN, WM, WN, false, false><<<grid, 64 * WM * WN, 0, stream>>>(a);       \
        else if (order == kColumns) chain_kernel<BM, BN, WM, WN, true, true><<<grid, 64 * WM * WN, 0, stream>>>(a); \
        else chain_kernel<BM, BN, WM, WN, false, true><<<grid, 64 * WM * WN, 0, stream>>>(a);                       \
        break;
        TGEMM_CHAIN_TILES(X)
#undef X
    }
    return hipGetLastError();
}

hipError_t launch_join(int tile, const ChainArgs &a, hipStream_t stream)
{
    const int side = kTiles[tile].side;
    const unsigned grid = (unsigned)a.op.count * (side / 64) * (side / 64);
    if (side == 256) chain_join_kernel<256><<<grid, 256, 0, stream>>>(a);
    else if (side == 128) chain_join_kernel<128><<<grid, 256, 0, stream>>>(a);
    else chain_join_kernel<64><<<grid, 256, 0, stream>>>(a);
    return hipGetLastError();
}

}  // namespace ortho
}  // namespace tgemm
