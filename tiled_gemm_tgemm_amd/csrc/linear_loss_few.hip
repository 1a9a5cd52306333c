// Row statistics of s·X·Wᵀ for a few rows of X (scoring tokens as they are
// served): bound by reading W once.
//
// A wavefront takes 16 words (rows of W) and R blocks of 16 rows of X, a
// work-group 64 words, or 16 with four wavefronts along k.  Fragments come
// straight from device memory into registers, eight values a lane, and the
// loads of the next 128 values of k are under way while these are multiplied:
// there is no LDS stage and no barrier, so each wavefront keeps 4 (float32: 8)
// KB of W on its way by itself.  The rows of X come from the caches.  A float32
// operand is split into its bf16 planes in registers, which spares a copy of W
// in planes, and rows may lie anywhere and have any length, which spares a copy
// of W in rows of whole steps.
//
// With the join, on Ws of 1 GiB together in turn: one row of 32000×4096 bf16 57
// µs (4.6 TB/s), one of 131072×2048 108 (5.0 TB/s), 4 of 56852×2752 float32 161
// (3.9 TB/s).  The same W call after call stays in the last-level cache in
// part, and the first takes 45.  So measured: 4×56852×2752 float32 155 against
// 185 with one wavefront along k, whose splitting of the operands the loads
// then wait for; 32×32768×1024 with one block of rows 52, with two 55, so
// those keep one.  Rows that start at odd multiples of 2 bytes cost their
// 16-byte loads twice the time: one row of 32000×4097 112 µs on Ws in turn (a
// copy and the tiles take 200).
#include "linear_loss.h"
#include "mfma16.h"

namespace tgemm {
namespace loss {
namespace {

using m16::f32x4;
using m16::Frag;

constexpr float kLog2e = 1.44269504088896340736f;

// Eight values of an operand as they are stored (device memory takes 16-byte
// loads at any address), and as fragments.
template <class In>
struct Eight {
    typedef typename Frag<In>::type Raw;
    typedef Raw Anywhere __attribute__((aligned(2)));
    static constexpr int kPlanes = 1;
    typedef In Element;
    static __device__ __forceinline__ Raw load(const In *p) { return *(const Anywhere *)p; }
    static __device__ __forceinline__ void set(Raw &raw, int e, In v) { raw[e] = v; }
    static __device__ __forceinline__ void planes(const Raw &raw, typename Frag<In>::type (&out)[1]) { out[0] = raw; }
};
template <>
struct Eight<float> {
    struct Raw {
        f32x4 lo, hi;
    };
    typedef f32x4 Anywhere __attribute__((aligned(4)));
    static constexpr int kPlanes = 3;
    typedef __bf16 Element;
    static __device__ __forceinline__ Raw load(const float *p) { return Raw{((const Anywhere *)p)[0], ((const Anywhere *)p)[1]}; }
    static __device__ __forceinline__ void set(Raw &raw, int e, float v) { (e < 4 ? raw.lo : raw.hi)[e & 3] = v; }
    static __device__ __forceinline__ void planes(const Raw &raw, m16::bf16x8 (&out)[3])
    {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            __bf16 h, m, l;
            m16::split(e < 4 ? raw.lo[e & 3] : raw.hi[e & 3], h, m, l);
            out[0][e] = h;
            out[1][e] = m;
            out[2][e] = l;
        }
    }
};

// C: the blocks of 16 words; S: the parts of the sum over k, each with
// wavefronts of its own, which are added through LDS.
template <class In, int R, int C, int S>
__global__ __launch_bounds__(64 * C * S) void linear_few_kernel(StatsArgs a, int D)
{
    typedef Eight<In> X8;
    typedef typename X8::Raw Raw;
    // 32 values of k each; two blocks of float32 rows fill the registers sooner,
    // as do 16 wavefronts
    constexpr int U = sizeof(In) == 4 && (R == 2 || C * S == 16) ? 2 : 4;
    const int lane = threadIdx.x & 63, wave = (threadIdx.x >> 6) % C, part = (threadIdx.x >> 6) / C;
    const int l16 = lane & 15, quarter = lane >> 4;
    const int group = blockIdx.x, col0 = (group * C + wave) * 16;
    // words and rows past the last are read from it and do not count
    const In *w = (const In *)a.op.B + (int64_t)min(col0 + l16, a.op.N - 1) * a.op.ldb + 8 * quarter;
    const In *x[R];
#pragma unroll
    for (int i = 0; i < R; ++i) x[i] = (const In *)a.op.A + (int64_t)min(16 * i + l16, a.op.M - 1) * a.op.lda + 8 * quarter;

    f32x4 acc[R];
#pragma unroll
    for (int i = 0; i < R; ++i) acc[i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    auto multiply = [&](const Raw &rw, const Raw (&rx)[R]) {
        typename Frag<typename X8::Element>::type fw[X8::kPlanes], fx[X8::kPlanes];
        X8::planes(rw, fw);
#pragma unroll
        for (int i = 0; i < R; ++i) {
            X8::planes(rx[i], fx);
            if constexpr (X8::kPlanes == 1) {
                acc[i] = Frag<In>::mfma(fw[0], fx[0], acc[i]);
            } else {
#pragma unroll
                for (int pair = 0; pair < 6; ++pair)
                    acc[i] = Frag<__bf16>::mfma(fw[(m16::kPairsB >> (2 * pair)) & 3], fx[(m16::kPairsA >> (2 * pair)) & 3],
                                                acc[i]);
            }
        }
    };

    Raw rw[2][U], rx[2][U][R];
    auto load = [&](int set, int k) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            rw[set][u] = X8::load(w + k + 32 * u);
#pragma unroll
            for (int i = 0; i < R; ++i) rx[set][u][i] = X8::load(x[i] + k + 32 * u);
        }
    };
    auto use = [&](int set) {
#pragma unroll
        for (int u = 0; u < U; ++u) multiply(rw[set][u], rx[set][u]);
    };
    const int each = (D / (32 * U) + S - 1) / S, whole = min(D / (32 * U), (part + 1) * each);
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
    for (int k = D / (32 * U) * 32 * U; k < D && part == S - 1; k += 32) {
        Raw zw{}, zx[R] = {};
        const int left = D - (k + 8 * quarter);
        if (left >= 8) {
            zw = X8::load(w + k);
#pragma unroll
            for (int i = 0; i < R; ++i) zx[i] = X8::load(x[i] + k);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (e < left) {
                    X8::set(zw, e, w[k + e]);
#pragma unroll
                    for (int i = 0; i < R; ++i) X8::set(zx[i], e, x[i][k + e]);
                }
        }
        multiply(zw, zx);
    }

    if constexpr (S > 1) {
        __shared__ f32x4 sums[S - 1][C][R][64];
        if (part > 0) {
#pragma unroll
            for (int i = 0; i < R; ++i) sums[part - 1][wave][i][lane] = acc[i];
        }
        __syncthreads();
        if (part == 0) {
#pragma unroll
            for (int q = 0; q < S - 1; ++q)
#pragma unroll
                for (int i = 0; i < R; ++i) acc[i] += sums[q][wave][i][lane];
        }
    }

    // acc[i][r]: row 16·i + l16, column col0 + 4·quarter + r
    const int left = a.op.N - (col0 + 4 * quarter);
    const float scale2 = a.scale * kLog2e;
    __shared__ float2 parts[C][16 * R];
#pragma unroll
    for (int i = 0; i < R; ++i) {
        const int row = 16 * i + l16;
        if (row < a.op.M && part == 0) {
            if (a.logits != nullptr) {
                float *to = a.logits + (int64_t)row * a.ldz + col0 + 4 * quarter;
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    if (r < left) to[r] = acc[i][r];
            }
            if (a.target != nullptr) {
                const int64_t want = a.target[row] - (col0 + 4 * quarter);
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    if (want == r && r < left) a.picked[row] = acc[i][r] * a.scale;
            }
            if (a.starts != nullptr) {
                const uint16_t *from = a.starts + (int64_t)row * (a.groups + 1) + group;
                for (int c = from[0]; c < from[1]; ++c) {
                    const uint32_t what = a.list[(int64_t)row * a.K + c];
                    const int e = (int)(what & 255) - (16 * wave + 4 * quarter);
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        if (e == r) a.student[(int64_t)row * a.K + (what >> 8)] = acc[i][r] * a.scale;
                }
            }
        }
        float high = -INFINITY;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            if (r >= left) acc[i][r] = -INFINITY;
            high = fmaxf(high, acc[i][r]);
        }
        high = fmaxf(high, __shfl_xor(high, 16));
        high = fmaxf(high, __shfl_xor(high, 32)) * scale2;
        const float from = high == -INFINITY ? 0.0f : high;
        float sum = 0.0f;
#pragma unroll
        for (int r = 0; r < 4; ++r) sum += __builtin_amdgcn_exp2f(fmaf(acc[i][r], scale2, -from));
        sum += __shfl_xor(sum, 16);
        sum += __shfl_xor(sum, 32);
        if (quarter == 0 && part == 0) parts[wave][row] = make_float2(high, sum);
    }
    __syncthreads();
    const int row = threadIdx.x;
    if (row < 16 * R && row < a.op.M) {
        float high = -INFINITY, sum = 0.0f;
#pragma unroll
        for (int v = 0; v < C; ++v) high = fmaxf(high, parts[v][row].x);
        const float from = high == -INFINITY ? 0.0f : high;
#pragma unroll
        for (int v = 0; v < C; ++v) sum += parts[v][row].y * __builtin_amdgcn_exp2f(parts[v][row].x - from);
        a.part[(int64_t)row * a.groups + group] = make_float2(high, sum);
    }
}

template <class In, int R>
void launch(const StatsArgs &a, int columns, int D, hipStream_t stream)
{
    const unsigned groups = (unsigned)a.groups;
    if (columns == 16) linear_few_kernel<In, R, 1, 4><<<groups, 256, 0, stream>>>(a, D);
    else if (sizeof(In) == 4 && R == 1) linear_few_kernel<In, R, 4, 4><<<groups, 1024, 0, stream>>>(a, D);
    else linear_few_kernel<In, R, 4, 1><<<groups, 256, 0, stream>>>(a, D);
}
template <class In>
void launch(const StatsArgs &a, int columns, int D, hipStream_t stream)
{
    if (a.op.M <= 16) launch<In, 1>(a, columns, D, stream);
    else launch<In, 2>(a, columns, D, stream);
}

}  // namespace

hipError_t launch_stats_few(const StatsArgs &a, tgemm_dtype_t dtype, int columns, int D, hipStream_t stream)
{
    if (dtype == TGEMM_F32) launch<float>(a, columns, D, stream);
    else if (dtype == TGEMM_BF16) launch<__bf16>(a, columns, D, stream);
    else launch<_Float16>(a, columns, D, stream);
    return hipGetLastError();
}

}  // namespace loss
}  // namespace tgemm
