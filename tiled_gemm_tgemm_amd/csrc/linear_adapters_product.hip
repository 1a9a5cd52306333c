// The products with a projection's weight and, in their epilogue, the
// adapters' part: X·Wᵀ + s·H·Bᵀ forward, dY·W + s·U·A backward.
#include "linear_adapters.h"
#include "mfma16.h"
#include "mfma16_store.h"
#include "some.h"

#include <type_traits>

namespace tgemm {
namespace adapters {
namespace {

using m16::bf16x8;
using m16::f32x4;
using m16::Frag;
using m16::kHeld;
using m16::kStepK;
using m16::lds_char;
using m16::load_some;
using m16::store_row;
using m16::TileProduct;

// Sums over ranks on the matrix cores, 32 ranks (8 a lane) at a time: the hidden
// values in two bf16 planes (a rounding to 2^-17) with B as it is (bf16) or in
// two bf16 planes (fp16, whose range bf16 holds); float32 in float32.
struct TwoPlanes {
    bf16x8 high, low;
};
struct EightFloats {
    f32x4 v[2];
};
// lane's eight ranks from k on of a row's planes
__device__ __forceinline__ void read_planes(const void *planes, int64_t row, int k, int padded, TwoPlanes &h)
{
    const __bf16 *from = (const __bf16 *)planes + row * 2 * padded + k;
    h.high = *(const bf16x8 *)from;
    h.low = *(const bf16x8 *)(from + padded);
}
__device__ __forceinline__ void read_planes(const void *planes, int64_t row, int k, int padded, EightFloats &h)
{
    const f32x4 *from = (const f32x4 *)((const float *)planes + row * padded + k);
    h.v[0] = from[0];
    h.v[1] = from[1];
}
template <class C>
struct Ranks;
template <>
struct Ranks<__bf16> {
    typedef TwoPlanes H;
    typedef bf16x8 F;
    static __device__ __forceinline__ F stored(const __bf16 (&v)[8])
    {
        F f;
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = v[e];
        return f;
    }
    static __device__ __forceinline__ f32x4 add(const F &c, const H &h, f32x4 acc)
    {
        return Frag<__bf16>::mfma(c, h.high, Frag<__bf16>::mfma(c, h.low, acc));
    }
};
template <>
struct Ranks<_Float16> {
    typedef TwoPlanes H;
    typedef TwoPlanes F;
    static __device__ __forceinline__ F stored(const _Float16 (&v)[8])
    {
        F f;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float x = (float)v[e], high = (float)(__bf16)x;
            f.high[e] = (__bf16)x;
            f.low[e] = (__bf16)(__builtin_isinf(x) || __builtin_isnan(x) ? 0.0f : x - high);
        }
        return f;
    }
    static __device__ __forceinline__ f32x4 add(const F &c, const H &h, f32x4 acc)
    {
        return Frag<__bf16>::mfma(c.high, h.high, Frag<__bf16>::mfma(c.high, h.low, Frag<__bf16>::mfma(c.low, h.high, acc)));
    }
};
template <>
struct Ranks<float> {
    typedef EightFloats H;
    typedef EightFloats F;
    static __device__ __forceinline__ F stored(const float (&v)[8])
    {
        F f;
#pragma unroll
        for (int e = 0; e < 8; ++e) f.v[e / 4][e % 4] = v[e];
        return f;
    }
    static __device__ __forceinline__ f32x4 add(const F &c, const H &h, f32x4 acc)
    {
#pragma unroll
        for (int e = 0; e < 8; ++e) acc = __builtin_amdgcn_mfma_f32_16x16x4f32(c.v[e / 4][e % 4], h.v[e / 4][e % 4], acc, 0, 0, 0);
        return acc;
    }
};

// Eight ranks of a row's hidden values, from rank k on, four parts' loads at once.
__device__ __forceinline__ void load_hidden(const Expand &e, int64_t row, int k, float (&v)[8])
{
    const float *from = e.hidden + row * e.c.rank + k;
#pragma unroll
    for (int n = 0; n < 8; ++n) v[n] = 0.0f;
    for (int p = 0; p < e.parts; p += 4) {
        float next[4][8];
#pragma unroll
        for (int u = 0; u < 4; ++u) load_some<float, 8>(from + (p + u) * e.part_stride, p + u < e.parts ? e.c.rank - k : 0, next[u]);
#pragma unroll
        for (int u = 0; u < 4; ++u)
#pragma unroll
            for (int n = 0; n < 8; ++n) v[n] += next[u][n];
    }
}

// A row's adapter: -1 for none, -2 for an id out of range.
__device__ __forceinline__ int id_of(const Expand &e, int64_t row, int64_t rows)
{
    if (row >= rows || e.ids == nullptr) return -1;
    const int64_t id = e.ids[row];
    return id >= 0 && id < e.c.count ? (int)id : id == -1 ? -1 : -2;
}

// Eight hidden values of a row.
__device__ __forceinline__ void eight_hidden(const __bf16 *planes, int64_t row, int k, int padded, float (&h)[8])
{
    TwoPlanes both;
    read_planes(planes, row, k, padded, both);
#pragma unroll
    for (int n = 0; n < 8; ++n) h[n] = (float)both.high[n] + (float)both.low[n];
}
__device__ __forceinline__ void eight_hidden(const float *planes, int64_t row, int k, int padded, float (&h)[8])
{
    EightFloats all;
    read_planes(planes, row, k, padded, all);
#pragma unroll
    for (int n = 0; n < 8; ++n) h[n] = all.v[n / 4][n % 4];
}

// The adapters' part of a lane's row and H adjacent columns on the vector units:
// every lane reads its own adapter.
template <class C, int H, bool RANK_INNER, class Acc>
__device__ __forceinline__ void add_lanes(const Expand &e, int id, int64_t row, int col, int columns, Acc &acc)
{
    typedef typename std::conditional<sizeof(C) == 4, float, __bf16>::type P;
    const int padded = (int)planes_rank(e.c.rank);
    const C *c = (const C *)e.c.p + id * e.c.stride;
    const int left = columns - col;
    if constexpr (RANK_INNER) {
        for (int k = 0; k < e.c.rank; k += 8) {
            int first = col;  // addresses are worked out anew, not kept in registers over the loop
            asm volatile("" : "+v"(first));
            float h[8];
            eight_hidden((const P *)e.planes, row, k, padded, h);
#pragma unroll
            for (int j = 0; j < H / 4; ++j) {
                C v[4][8];
#pragma unroll
                for (int x = 0; x < 4; ++x)
                    load_some<C, 8>(c + (int64_t)min(first + 4 * j + x, columns - 1) * e.c.ld + k, e.c.rank - k, v[x]);
#pragma unroll
                for (int n = 0; n < 8; ++n)
#pragma unroll
                    for (int x = 0; x < 4; ++x) acc[j][x] = fmaf(h[n], (float)v[x][n], acc[j][x]);
            }
        }
    } else {
        for (int k = 0; k < e.c.rank; k += 8) {
            float h[8];
            eight_hidden((const P *)e.planes, row, k, padded, h);
#pragma unroll
            for (int n = 0; n < 8; ++n) {
                C v[H];
                load_some<C, H>(c + (k + n) * e.c.ld + min(col, columns - 1), k + n < e.c.rank ? left : 0, v);
#pragma unroll
                for (int x = 0; x < H; ++x) acc[x / 4][x % 4] = fmaf(h[n], (float)v[x], acc[x / 4][x % 4]);
            }
        }
    }
}

// Eight ranks, from k0 + 8·(lane / 16) on, of the column at index lane % 16 of
// block j (mfma16.h), of an adapter at c.
template <class Tile, class C, bool RANK_INNER>
__device__ __forceinline__ typename Ranks<C>::F column_ranks(const ProductArgs &a, const C *c, int col0, int j, int k0)
{
    const int lane = m16::thread_anew() & 63, l16 = lane & 15, quarter = lane >> 4, k = k0 + 8 * quarter;
    const int col = min(col0 + 4 * Tile::FN * (l16 >> 2) + 4 * j + (l16 & 3), a.op.N - 1);
    C v[8];
    if constexpr (!RANK_INNER) {
        const C *from = c + k0 * a.e.c.ld;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int r = min(8 * quarter + e, a.e.c.rank - 1 - k0);  // ranks past the last meet zeros
            const C x = from[(uint32_t)r * (uint32_t)a.e.c.ld + (uint32_t)col];
            v[e] = k + e < a.e.c.rank ? x : (C)0.0f;
        }
    } else {
        load_some<C, 8>(c + (int64_t)col * a.e.c.ld + k, a.e.c.rank - k, v);
    }
    return Ranks<C>::stored(v);
}

// One adapter's part of all of a wavefront's rows.
template <class Tile, class C, bool RANK_INNER>
__device__ __forceinline__ void add_one(const ProductArgs &a, int adapter, int row0, int col0, typename Tile::Acc &acc)
{
    const int padded = (int)planes_rank(a.e.c.rank);
    const C *c = (const C *)a.e.c.p + adapter * a.e.c.stride;
    for (int k0 = 0; k0 < padded; k0 += 32) {
        const int lane = m16::thread_anew() & 63, l16 = lane & 15, quarter = lane >> 4;
        typename Ranks<C>::H h[Tile::FM];
#pragma unroll
        for (int i = 0; i < Tile::FM; ++i) read_planes(a.e.planes, min(row0 + i * 16 + l16, a.op.M - 1), k0 + 8 * quarter, padded, h[i]);
#pragma unroll
        for (int j = 0; j < Tile::FN; ++j) {
            const typename Ranks<C>::F f = column_ranks<Tile, C, RANK_INNER>(a, c, col0, j, k0);
#pragma unroll
            for (int i = 0; i < Tile::FM; ++i) acc[i][j] = Ranks<C>::add(f, h[i], acc[i][j]);
        }
    }
}

// E: the tiles' type; C: the adapters'.  The wavefront's rows are taken adapter
// by adapter: tokens of a sequence share theirs.  Where 32 rows have more than
// kMixed, each lane reads its own instead, which takes the vector units as long
// as about three adapters take the loads' way there and back (in a 256×256
// tile, whose registers do not hold that, they are taken one by one all the
// same).  The bound on registers is that of kTiles' work-groups a compute unit.
// Bound by the matrix cores, as the product alone is: 8192×16384×4096 with 8
// adapters of 32 ranks in runs 871 µs, 1.27 PFLOP/s (in random order 1306);
// 2003×4096×4096 with 6 of 64 85 µs, 0.8 PFLOP/s, one round of 128×128 tiles.
constexpr int kMixed = 3;
template <class E, class C, int BM, int BN, int WM, int WN, bool B_MC, bool RANK_INNER>
__global__ __launch_bounds__(64 * WM * WN, BM == 32 ? 3 : 2) void adapted_kernel(ProductArgs a)
{
    typedef TileProduct<E, BM, BN, WM, WN, false, B_MC, m16::Operands, true> Tile;
    constexpr int H = kHeld<Tile>;
    __shared__ __align__(1024) char lds[Tile::kLds];
    struct Ahead {
        int id[Tile::FM];
    };
    auto prologue = [&](int row0, int) {
        const int l16 = m16::thread_anew() & 15;
        Ahead ahead;
#pragma unroll
        for (int i = 0; i < Tile::FM; ++i) ahead.id[i] = id_of(a.e, row0 + i * 16 + l16, a.op.M);
        return ahead;
    };
    Tile::run(a.op, (lds_char *)lds, prologue, [&](typename Tile::Acc &acc, int row0, int col0, int split, const Ahead &ahead) {
        const int lane = m16::thread_anew() & 63, l16 = lane & 15, quarter = lane >> 4;
        // One adapter for all of the wavefront's rows: everything is loaded at once.
        int one = -1;
#pragma unroll
        for (int i = 0; i < Tile::FM; ++i) {
            const uint32_t some = (uint32_t)__ballot(ahead.id[i] >= 0) & 0xFFFF;
            if (one < 0 && some != 0) one = __builtin_amdgcn_readlane(ahead.id[i], __builtin_ctz(some));
        }
        bool alone = one >= 0;
#pragma unroll
        for (int i = 0; i < Tile::FM; ++i) alone = alone && __ballot(ahead.id[i] == one || row0 + i * 16 + l16 >= a.op.M) == ~(uint64_t)0;
        if (alone) add_one<Tile, C, RANK_INNER>(a, one, row0, col0, acc);
        // 32 rows at a time, which leaves the other accumulators where they are
        const int padded = (int)planes_rank(a.e.c.rank);
#pragma unroll
        for (int i0 = 0; i0 < Tile::FM; i0 += 2) {
            int id[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) id[i] = alone ? -1 : ahead.id[i0 + i];
            uint64_t left = (__ballot(id[0] >= 0) & 0xFFFF) | __ballot(id[1] >= 0) << 16;
            left &= 0xFFFFFFFF;
            auto next = [&]() {
                const int at = __builtin_ctzll(left), now = __builtin_amdgcn_readlane(at < 16 ? id[0] : id[1], at & 15);
                left &= ~((__ballot(id[0] == now) & 0xFFFF) | __ballot(id[1] == now) << 16);
                return now;
            };
            const uint64_t rows = left;
            int adapters = 0;
            while (left != 0) {
                next();
                ++adapters;
            }
            if (Tile::FM < 8 && adapters > kMixed) {
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    if (id[i] >= 0) add_lanes<C, H, RANK_INNER>(a.e, id[i], row0 + (i0 + i) * 16 + l16, col0 + H * quarter, a.op.N, acc[i0 + i]);
                left = 0;
            } else {
                left = rows;
            }
            while (left != 0) {
                const int now = next();
                const C *c = (const C *)a.e.c.p + now * a.e.c.stride;
                // summed apart and added to its own rows alone: what another
                // adapter holds, infinities and NaN too, does not reach them
                f32x4 more[2][Tile::FN] = {};
                for (int k0 = 0; k0 < padded; k0 += 32) {
                    // worked out anew, not kept in registers over the loop
                    const int lane = m16::thread_anew() & 63, l16 = lane & 15, quarter = lane >> 4;
                    const int k = k0 + 8 * quarter;
                    typename Ranks<C>::H h[2];
#pragma unroll
                    for (int i = 0; i < 2; ++i) read_planes(a.e.planes, min(row0 + (i0 + i) * 16 + l16, a.op.M - 1), k, padded, h[i]);
#pragma unroll
                    for (int j = 0; j < Tile::FN; ++j) {
                        // (the registers hold no more than one block's loads)
                        if (Tile::FM == 8 && sizeof(C) == 2 && !RANK_INNER) asm volatile("" ::: "memory");
                        const typename Ranks<C>::F f = column_ranks<Tile, C, RANK_INNER>(a, c, col0, j, k0);
#pragma unroll
                        for (int i = 0; i < 2; ++i) more[i][j] = Ranks<C>::add(f, h[i], more[i][j]);
                    }
                }
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    if (id[i] == now) {
#pragma unroll
                        for (int j = 0; j < Tile::FN; ++j) acc[i0 + i][j] += more[i][j];
                    }
            }
#pragma unroll
            for (int i = 0; i < 2; ++i)
                if (id[i] == -2) {
#pragma unroll
                    for (int j = 0; j < Tile::FN; ++j) acc[i0 + i][j] = f32x4{NAN, NAN, NAN, NAN};
                }
        }
        const int col = col0 + H * quarter, left = a.op.N - col;
        if (left <= 0) return;
#pragma unroll
        for (int i = 0; i < Tile::FM; ++i) {
            const int row = row0 + i * 16 + l16;
            if (row >= a.op.M) continue;
            float v[H];
#pragma unroll
            for (int e = 0; e < H; ++e) v[e] = acc[i][e / 4][e % 4];
            const int64_t at = (int64_t)row * a.ldo + col + (int64_t)split * a.split_stride;
            if (a.dtype == TGEMM_F32) store_row<float, H>((float *)a.out + at, v, left);
            else store_row<E, H>((E *)a.out + at, v, left);
        }
    });
}

// The sum over parts and the adapters' part, four columns a thread: adjacent
// ones, or 64 apart where a column's ranks are, so that a wavefront's loads of
// an adapter lie side by side.  (In the tiles of a
// split sum, which are few and short, the adapters' loads would be waited for:
// 256×4096×4096 with 32 adapters 49 µs and 5 for the sum, against 23 and 7.5.)
// Bound by the parts' and the adapters' loads (777×3000 float32 of one part with ranks of 10: 14 µs).
template <class C, bool RANK_INNER>
__global__ __launch_bounds__(256) void adapted_sum_kernel(AddArgs a)
{
    typedef typename std::conditional<sizeof(C) == 4, float, __bf16>::type P;
    const int64_t per_row = (a.N + 255) / 256, total = a.T * per_row;
    const int padded = (int)planes_rank(a.e.c.rank), lane = threadIdx.x & 63;
    for (int64_t p = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6); p < total; p += (int64_t)gridDim.x * 4) {
        constexpr int kApart = RANK_INNER ? 64 : 1;
        const int64_t row = p / per_row, col0 = p % per_row * 256 + (RANK_INNER ? lane : 4 * lane);
        // columns past the last are read from it and not stored
        int64_t col[4];
        float v[4];
#pragma unroll
        for (int x = 0; x < 4; ++x) {
            col[x] = min(col0 + kApart * x, a.N - 1);
            v[x] = a.part[row * a.ld + col[x]];
        }
        for (int s = 1; s < a.count; s += 4) {  // four parts on their way at once
            float next[4][4];
#pragma unroll
            for (int u = 0; u < 4; ++u)
#pragma unroll
                for (int x = 0; x < 4; ++x) next[u][x] = s + u < a.count ? a.part[row * a.ld + col[x] + (s + u) * a.stride] : 0.0f;
#pragma unroll
            for (int u = 0; u < 4; ++u)
#pragma unroll
                for (int x = 0; x < 4; ++x) v[x] += next[u][x];
        }
        const int id = id_of(a.e, row, a.T);
        if (id >= 0) {
            const C *c = (const C *)a.e.c.p + id * a.e.c.stride;
            for (int k = 0; k < a.e.c.rank; k += 8) {
                float h[8];
                eight_hidden((const P *)a.e.planes, row, k, padded, h);
                if constexpr (RANK_INNER) {
                    C w[4][8];
#pragma unroll
                    for (int x = 0; x < 4; ++x) load_some<C, 8>(c + col[x] * a.e.c.ld + k, a.e.c.rank - k, w[x]);
#pragma unroll
                    for (int n = 0; n < 8; ++n)
#pragma unroll
                        for (int x = 0; x < 4; ++x) v[x] = fmaf(h[n], (float)w[x][n], v[x]);
                } else {
                    C w[8][4];
#pragma unroll
                    for (int n = 0; n < 8; ++n) load_some<C, 4>(c + (k + n) * a.e.c.ld + col[0], k + n < a.e.c.rank ? a.N - col0 : 0, w[n]);
#pragma unroll
                    for (int n = 0; n < 8; ++n)
#pragma unroll
                        for (int x = 0; x < 4; ++x) v[x] = fmaf(h[n], (float)w[n][x], v[x]);
                }
            }
        } else if (id == -2) {
#pragma unroll
            for (int x = 0; x < 4; ++x) v[x] = NAN;
        }
        C *to = (C *)a.out + row * a.ldo;
#pragma unroll
        for (int x = 0; x < 4; ++x)
            if (col0 + kApart * x < a.N) to[col0 + kApart * x] = (C)v[x];
    }
}

// ---- a few rows ------------------------------------------------------------

// The end of a few rows' products: wavefront n of S adds up the S parts of the
// n-th blocks (row lane % 16, columns 4·(lane / 16) + r) and the adapters' part
// on the vector units: there may be as many adapters as rows, and their loads
// do not wait for one another.
template <class In, int R, int COLS, int S, class Sum>
__device__ __forceinline__ void finish_few(const FewArgs &a, int col0, int part, int lane, Sum sum)
{
    const int l16 = lane & 15, quarter = lane >> 4;
    for (int n = part; n < R * COLS; n += S) {
        const int i = n / COLS, j = n % COLS;
        f32x4 v = sum(0, i, j);
#pragma unroll
        for (int s = 1; s < S; ++s) v += sum(s, i, j);
        const int row = 16 * i + l16, col = col0 + 16 * j + 4 * quarter;
        if (row >= a.T) continue;
        const int id = id_of(a.e, row, a.T);
        if (id >= 0) {
            const In *c[4];
#pragma unroll
            for (int r = 0; r < 4; ++r) c[r] = (const In *)a.e.c.p + id * a.e.c.stride + (int64_t)min(col + r, a.N - 1) * a.e.c.ld;
            f32x4 more{0, 0, 0, 0};
            for (int k = 0; k < a.e.c.rank; k += 8) {
                In b[4][8];
                float h[8];
#pragma unroll
                for (int r = 0; r < 4; ++r) load_some<In, 8>(c[r] + k, a.e.c.rank - k, b[r]);
                load_hidden(a.e, row, k, h);
#pragma unroll
                for (int e = 0; e < 8; ++e)
#pragma unroll
                    for (int r = 0; r < 4; ++r) more[r] = fmaf(h[e], (float)b[r][e], more[r]);
            }
            const float factor = a.e.scales != nullptr ? a.e.scales[id] : 1.0f;
#pragma unroll
            for (int r = 0; r < 4; ++r) v[r] = fmaf(factor, more[r], v[r]);
        } else if (id == -2) {
            v = f32x4{NAN, NAN, NAN, NAN};
        }
        In *to = (In *)a.Y + row * a.ldy + col;
#pragma unroll
        for (int r = 0; r < 4; ++r)
            if (col + r < a.N) to[r] = (In)v[r];
    }
}

// This wavefront's loads into LDS have arrived but for the last FLYING.
template <int FLYING>
__device__ __forceinline__ void arrived()
{
    static_assert(FLYING < 64, "six bits");
    asm volatile("s_waitcnt vmcnt(%0)" : : "n"(FLYING) : "memory");
}

// Fragments straight from device memory, no LDS stage and no barrier, as the
// loss operators take a few rows: a wavefront takes COLS blocks of 16 columns of
// the result, R blocks of 16 rows and an eighth of the sum, in steps of 64
// values of k of which a lane takes 16 adjacent ones in two fragments: a row's
// loads are whole cache lines.  Then each
// lane adds its own rows' adapters on the vector units: there may be as many as
// rows, and their matrices' loads do not wait for one another.
constexpr int kFewParts = 8, kFewLdsParts = 4;
template <class In, int R, int COLS>
__global__ __launch_bounds__(64 * kFewParts) void adapted_few_kernel(FewArgs a)
{
    constexpr int S = kFewParts, kHeld = (R + COLS) * (sizeof(In) == 4 ? 2 : 1), U = kHeld <= 3 ? 4 : 2;
    __shared__ f32x4 sums[S][R][COLS][64];
    const int lane = threadIdx.x & 63, part = threadIdx.x >> 6, l16 = lane & 15, quarter = lane >> 4;
    const int col0 = blockIdx.x * (16 * COLS);
    const In *w[COLS], *x[R];
#pragma unroll
    for (int j = 0; j < COLS; ++j) w[j] = (const In *)a.W + (int64_t)min(col0 + 16 * j + l16, a.N - 1) * a.ldw + 16 * quarter;
#pragma unroll
    for (int i = 0; i < R; ++i) x[i] = (const In *)a.X + (int64_t)min(16 * i + l16, a.T - 1) * a.ldx + 16 * quarter;
    f32x4 acc[R][COLS];
#pragma unroll
    for (int i = 0; i < R; ++i)
#pragma unroll
        for (int j = 0; j < COLS; ++j) acc[i][j] = f32x4{0, 0, 0, 0};
    auto multiply = [&](const In (&vw)[COLS][8], const In (&vx)[R][8]) {
        if constexpr (sizeof(In) == 2) {
            typename Frag<In>::type fw[COLS], fx[R];
#pragma unroll
            for (int j = 0; j < COLS; ++j)
#pragma unroll
                for (int e = 0; e < 8; ++e) fw[j][e] = vw[j][e];
#pragma unroll
            for (int i = 0; i < R; ++i)
#pragma unroll
                for (int e = 0; e < 8; ++e) fx[i][e] = vx[i][e];
#pragma unroll
            for (int i = 0; i < R; ++i)
#pragma unroll
                for (int j = 0; j < COLS; ++j) acc[i][j] = Frag<In>::mfma(fw[j], fx[i], acc[i][j]);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
#pragma unroll
                for (int i = 0; i < R; ++i)
#pragma unroll
                    for (int j = 0; j < COLS; ++j)
                        acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x4f32(vw[j][e], vx[i][e], acc[i][j], 0, 0, 0);
        }
    };
    In vw[2][U][COLS][8], vx[2][U][R][8];
    auto load = [&](int set, int k) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
#pragma unroll
            for (int j = 0; j < COLS; ++j) load_some<In, 8>(w[j] + k + 64 * (u / 2) + 8 * (u % 2), 8, vw[set][u][j]);
#pragma unroll
            for (int i = 0; i < R; ++i) load_some<In, 8>(x[i] + k + 64 * (u / 2) + 8 * (u % 2), 8, vx[set][u][i]);
        }
    };
    auto use = [&](int set) {
#pragma unroll
        for (int u = 0; u < U; ++u) multiply(vw[set][u], vx[set][u]);
    };
    const int all = a.D / (32 * U), each = (all + S - 1) / S, whole = min(all, (part + 1) * each);
    int n = part * each;
    if (n < whole) {
        load(0, n * 32 * U);
        for (++n; n + 1 < whole; n += 2) {
            load(1, n * 32 * U);
            use(0);
            load(0, (n + 1) * 32 * U);
            use(1);
        }
        if (n < whole) {
            load(1, n * 32 * U);
            use(0);
            use(1);
        } else {
            use(0);
        }
    }
    if (part == S - 1) {
        for (int k = all * 32 * U; k < a.D; k += 64) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int left = a.D - (k + 16 * quarter + 8 * h);
                In zw[COLS][8], zx[R][8];
#pragma unroll
                for (int j = 0; j < COLS; ++j) load_some<In, 8>(w[j] + k + 8 * h, left, zw[j]);
#pragma unroll
                for (int i = 0; i < R; ++i) load_some<In, 8>(x[i] + k + 8 * h, left, zx[i]);
                multiply(zw, zx);
            }
        }
    }
#pragma unroll
    for (int i = 0; i < R; ++i)
#pragma unroll
        for (int j = 0; j < COLS; ++j) sums[part][i][j][lane] = acc[i][j];
    __syncthreads();
    finish_few<In, R, COLS, S>(a, col0, part, lane, [&](int s, int i, int j) { return sums[s][i][j][lane]; });
}

// The same on 16-bit operands with aligned rows of whole steps of 64.  A
// fragment's load from device memory takes 16 bytes of 16 rows in turn and so
// 16 bytes a clock of a compute unit: enough for W's way in once, not for X's
// in every work-group.  Here both go straight to LDS in 128 adjacent bytes a row, into
// `STAGES` stages of a wavefront's own, so that it waits for nobody and the loads
// of all the stages are under way at once.  Wavefront n takes steps n, n + 4, ...
// Bound by W's way from memory and, with more rows, by X's from the L2s.  With W
// not in any cache (µs, T×N×D): 1×4096×4096 11.7 (2.9 TB/s), 16×4096×4096 11.6 against 14.5 straight from
// memory, 48×8192×2048 15.9 against 17.6, 64×4096×4096 17.6 against 26.9,
// 48×2048×8192 21.4 against 35.6; of these the adapters' part is 3 to 5.
template <class In, int R, int COLS, int STAGES>
__global__ __launch_bounds__(64 * kFewLdsParts) void adapted_few_lds_kernel(FewArgs a)
{
    constexpr int S = kFewLdsParts, kLoads = 2 * (R + COLS), kStage = kLoads * 1024;
    typedef m16::Slice<16 * R, R, 64, false, false> SliceX;
    typedef m16::Slice<16 * COLS, COLS, 64, false, false> SliceW;
    static_assert(SliceX::kBytes + SliceW::kBytes == kStage && R * COLS <= kLoads * STAGES, "room");
    __shared__ __align__(1024) char lds[S * STAGES * kStage];
    const int lane = threadIdx.x & 63, part = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int col0 = blockIdx.x * (16 * COLS);
    const char *x = (const char *)a.X, *w = (const char *)((const In *)a.W + col0 * a.ldw);
    lds_char *own = (lds_char *)lds + part * STAGES * kStage;
    m16::Loader<SliceX> lx;
    m16::Loader<SliceW> lw;
#pragma unroll
    for (int r = 0; r < 2 * R; ++r) lx.off[r] = SliceX::offset(r * 64 + lane, a.ldx, a.T - 1, kStepK);
#pragma unroll
    for (int r = 0; r < 2 * COLS; ++r) lw.off[r] = SliceW::offset(r * 64 + lane, a.ldw, a.N - 1 - col0, kStepK);
    auto issue = [&](int stage, int step) {
#pragma unroll
        for (int r = 0; r < 2 * COLS; ++r) lw.issue_one(w + (int64_t)step * (2 * kStepK), own + stage * kStage + SliceX::kBytes, 0, r);
#pragma unroll
        for (int r = 0; r < 2 * R; ++r) lx.issue_one(x + (int64_t)step * (2 * kStepK), own + stage * kStage, 0, r);
    };
    m16::Reader<16 * R, R, false, false> rx;
    m16::Reader<16 * COLS, COLS, false, false> rw;
    rx.place(0, lane);
    rw.place(0, lane);
    f32x4 acc[R][COLS];
#pragma unroll
    for (int i = 0; i < R; ++i)
#pragma unroll
        for (int j = 0; j < COLS; ++j) acc[i][j] = f32x4{0, 0, 0, 0};
    const int steps = a.D / kStepK, count = part < steps ? (steps - part + S - 1) / S : 0;
    // the work-groups of an XCD begin at steps apart: rows that lie a power of
    // two apart would have them all at the same few of the L2's channels
    int next = count > 0 ? (int)(blockIdx.x / m16::kXcds % (unsigned)count) : 0;
    auto issue_next = [&](int stage) {
        issue(stage, part + S * next);
        if (++next == count) next = 0;
    };
#pragma unroll
    for (int n = 0; n < STAGES; ++n)
        if (n < count) issue_next(n);
    int stage = 0;
    for (int n = 0; n < count; ++n) {
        // this stage's loads have arrived; those of the later ones may be under way
        const int later = count - 1 - n;
        if (later >= STAGES - 1) arrived<(STAGES - 1) * kLoads>();
        else if (STAGES > 3 && later == 2) arrived<2 * kLoads>();
        else if (later == 1) arrived<kLoads>();
        else arrived<0>();
        typename Frag<In>::type fx[2][R], fw[2][COLS];
        lds_char *at = own + stage * kStage;
#pragma unroll
        for (int s = 0; s < 2; ++s) {
#pragma unroll
            for (int i = 0; i < R; ++i) fx[s][i] = rx.template read<In>(at, i, s);
#pragma unroll
            for (int j = 0; j < COLS; ++j) fw[s][j] = rw.template read<In>(at + SliceX::kBytes, j, s);
        }
        // the stage has been read
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        if (n + STAGES < count) issue_next(stage);
        if (++stage == STAGES) stage = 0;
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
            for (int i = 0; i < R; ++i)
#pragma unroll
                for (int j = 0; j < COLS; ++j) acc[i][j] = Frag<In>::mfma(fw[s][j], fx[s][i], acc[i][j]);
    }
    // every wavefront's sums go where its stages were
    f32x4 *sums = (f32x4 *)(lds + part * STAGES * kStage);
#pragma unroll
    for (int i = 0; i < R; ++i)
#pragma unroll
        for (int j = 0; j < COLS; ++j) sums[(i * COLS + j) * 64 + lane] = acc[i][j];
    __syncthreads();
    finish_few<In, R, COLS, S>(a, col0, part, lane, [&](int s, int i, int j) {
        return ((const f32x4 *)(lds + s * STAGES * kStage))[(i * COLS + j) * 64 + lane];
    });
}

template <class In, int COLS>
void few(const FewArgs &a, hipStream_t stream)
{
    const unsigned grid = (unsigned)((a.N + 16 * COLS - 1) / (16 * COLS));
    if constexpr (sizeof(In) == 2) {
        if (a.through_lds) {
            if (a.T <= 16) adapted_few_lds_kernel<In, 1, COLS, 4><<<grid, 64 * kFewLdsParts, 0, stream>>>(a);
            else if (a.T <= 32) adapted_few_lds_kernel<In, 2, COLS, 4><<<grid, 64 * kFewLdsParts, 0, stream>>>(a);
            else if (a.T <= 48) adapted_few_lds_kernel<In, 3, COLS, COLS == 1 ? 4 : 3><<<grid, 64 * kFewLdsParts, 0, stream>>>(a);
            else adapted_few_lds_kernel<In, 4, COLS, 3><<<grid, 64 * kFewLdsParts, 0, stream>>>(a);
            return;
        }
    }
    if (a.T <= 16) adapted_few_kernel<In, 1, COLS><<<grid, 64 * kFewParts, 0, stream>>>(a);
    else if (a.T <= 32) adapted_few_kernel<In, 2, COLS><<<grid, 64 * kFewParts, 0, stream>>>(a);
    else if (a.T <= 48) adapted_few_kernel<In, 3, COLS><<<grid, 64 * kFewParts, 0, stream>>>(a);
    else adapted_few_kernel<In, 4, COLS><<<grid, 64 * kFewParts, 0, stream>>>(a);
}
// Two blocks of columns halve the rows' way from the caches, where they leave
// no compute unit without any.
template <class In>
void few(const FewArgs &a, hipStream_t stream)
{
    if (a.N >= 8192 && a.T > 16) few<In, 2>(a, stream);
    else few<In, 1>(a, stream);
}

template <bool B_MC, bool RANK_INNER>
hipError_t product(bool half, int tile, const ProductArgs &a, hipStream_t stream)
{
    const int64_t ids = a.op.ids(), most = (int64_t)256 * loss::kTiles[tile].wg_per_cu;
    const unsigned grid = (unsigned)(ids < most ? ids : most);
    switch (tile) {
#define X(I, BM, BN, WM, WN)                                                                                                     \
    case I:                                                                                                                      \
        if (a.stored == TGEMM_F32)                                                                                               \
            adapted_kernel<__bf16, float, BM, BN, WM, WN, B_MC, RANK_INNER><<<grid, 64 * WM * WN, 0, stream>>>(a);               \
        else if (half) adapted_kernel<_Float16, _Float16, BM, BN, WM, WN, B_MC, RANK_INNER><<<grid, 64 * WM * WN, 0, stream>>>(a); \
        else adapted_kernel<__bf16, __bf16, BM, BN, WM, WN, B_MC, RANK_INNER><<<grid, 64 * WM * WN, 0, stream>>>(a);             \
        break;
        TGEMM_TILES(X)
#undef X
    }
    return hipGetLastError();
}

}  // namespace

hipError_t launch_product(bool half, bool b_mc, int tile, const ProductArgs &a, hipStream_t stream)
{
    if (!b_mc) return product<false, true>(half, tile, a, stream);
    return a.e.c.rank_inner ? product<true, true>(half, tile, a, stream) : product<true, false>(half, tile, a, stream);
}

hipError_t launch_add(const AddArgs &a, hipStream_t stream)
{
    const int64_t blocks = (a.T * ((a.N + 255) / 256) + 3) / 4;
    const unsigned grid = (unsigned)(blocks < (1 << 20) ? blocks : 1 << 20);
    const bool inner = a.e.c.rank_inner;
    if (a.dtype == TGEMM_F32) {
        if (inner) adapted_sum_kernel<float, true><<<grid, 256, 0, stream>>>(a);
        else adapted_sum_kernel<float, false><<<grid, 256, 0, stream>>>(a);
    } else if (a.dtype == TGEMM_BF16) {
        if (inner) adapted_sum_kernel<__bf16, true><<<grid, 256, 0, stream>>>(a);
        else adapted_sum_kernel<__bf16, false><<<grid, 256, 0, stream>>>(a);
    } else {
        if (inner) adapted_sum_kernel<_Float16, true><<<grid, 256, 0, stream>>>(a);
        else adapted_sum_kernel<_Float16, false><<<grid, 256, 0, stream>>>(a);
    }
    return hipGetLastError();
}

hipError_t launch_few(const FewArgs &a, hipStream_t stream)
{
    if (a.dtype == TGEMM_F32) few<float>(a, stream);
    else if (a.dtype == TGEMM_BF16) few<__bf16>(a, stream);
    else few<_Float16>(a, stream);
    return hipGetLastError();
}

}  // namespace adapters
}  // namespace tgemm
