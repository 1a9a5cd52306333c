// Passes over the rows of G for the Newton-Schulz operator: its norm, its
// planes, and the whole iteration in float64 where one side is small.
#include "orthogonalize.h"
#include "some.h"

#include <math.h>

namespace tgemm {
namespace ortho {
namespace {

using m16::load_some;
using m16::Some;

typedef double f64x4 __attribute__((ext_vector_type(4)));

// The work-group's sum, in every thread, in a fixed order.
__device__ __forceinline__ double sum_of_group(double v, double *room)
{
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) v += __shfl_xor(v, d);
    if ((threadIdx.x & 63) == 0) room[threadIdx.x >> 6] = v;
    __syncthreads();
    double all = 0;
    for (unsigned w = 0; w < blockDim.x / 64; ++w) all += room[w];
    __syncthreads();
    return all;
}

// Squares are summed in float64: those of float32 values may lie past float32's ends.
// Bound by reading G once (8192×8192 bf16 50 µs, 2.7 TB/s).
template <class In>
__global__ __launch_bounds__(256) void squares_kernel(SplitArgs a)
{
    __shared__ double room[4];
    const In *g = (const In *)a.G + blockIdx.y * a.batch_g;
    const int64_t per_row = (a.cols + 7) / 8, pieces = a.rows * per_row;
    double sum = 0;
    for (int64_t n = (int64_t)blockIdx.x * 256 + threadIdx.x; n < pieces; n += (int64_t)gridDim.x * 256) {
        const int64_t row = n / per_row, col = n % per_row * 8;
        In v[8];
        load_some<In, 8>(g + row * a.ld + col, a.cols - col, v);
#pragma unroll
        for (int e = 0; e < 8; ++e) sum += (double)(float)v[e] * (double)(float)v[e];
    }
    sum = sum_of_group(sum, room);
    if (threadIdx.x == 0) a.squares[(int64_t)blockIdx.y * a.parts + blockIdx.x] = sum;
}

// Bound by memory: G is read and as many bytes (float32), or twice as many, are
// written (8192×8192 bf16 84 µs, 4.8 TB/s).
template <class In>
__global__ __launch_bounds__(256) void split_kernel(SplitArgs a)
{
    __shared__ double room[4];
    double sum = 0;
    for (int p = threadIdx.x; p < a.parts; p += 256) sum += a.squares[(int64_t)blockIdx.y * a.parts + p];
    sum = sum_of_group(sum, room);
    // in float64: a norm below 2^-126 has a reciprocal past float32's end
    const double factor = (double)(1 << kShift) / (sqrt(sum) + (double)a.eps);
    const In *g = (const In *)a.G + blockIdx.y * a.batch_g;
    _Float16 *to = (_Float16 *)a.planes + blockIdx.y * a.batch_out;
    const int64_t per_row = a.ldo / 8, pieces = a.rows_out * per_row;
    for (int64_t n = (int64_t)blockIdx.x * 256 + threadIdx.x; n < pieces; n += (int64_t)gridDim.x * 256) {
        const int64_t row = n / per_row, col = n % per_row * 8;
        In v[8];
        const int64_t left = row < a.rows ? a.cols - col : 0;
        load_some<In, 8>(g + row * a.ld + col, left, v);
        typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
        f16x8 high, low;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            // zeros past the ends stay zeros, whatever the factor
            const float x = e < left ? (float)((double)(float)v[e] * factor) : 0.0f;
            high[e] = (_Float16)x;
            low[e] = (_Float16)(x - (float)high[e]);
        }
        *(f16x8 *)(to + row * a.ldo + col) = high;
        *(f16x8 *)(to + a.plane + row * a.ldo + col) = low;
    }
}

// ---- a small side, in float64 ----------------------------------------------
//
// With S_0 = X_0·X_0ᵀ all iterates are X_k = Q_k·X_0 with Q_k a polynomial of
// S_0, so the whole iteration runs on side×side matrices: P = a + b·S + c·S²,
// Q <- P·Q, S <- P·S·P.  That squares the singular values' range: float32 would
// lose what is below 2^-12 of the largest, float64 keeps as much of S as the
// products with X keep of X.  The matrix cores multiply float64 at 78 TFLOP/s,
// which for a side of 64 is little, and G is read twice and nothing of its size
// is held in between.  (24 of 16×4096: 4.2, 8.0 and 5.2 µs.)
//
// v_mfma_f64_16x16x4: a lane holds A(lane % 16, lane / 16), B(lane / 16, lane %
// 16) and the four results (4·r + lane / 16, lane % 16).

// Part of S: element (i, k) of the small side's matrix lies at i·ld + k, or at
// k·ld + i (tall).  The order of the k's in an instruction is free as long as
// both operands have the same.
template <class In, int BLOCKS, bool TALL>
__global__ __launch_bounds__(256) void gram_kernel(SmallArgs a)
{
    constexpr int kPairs = BLOCKS * (BLOCKS + 1) / 2;
    __shared__ f64x4 sums[3][kPairs][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, l16 = lane & 15, quarter = lane >> 4;
    const In *g = (const In *)a.G + blockIdx.y * a.batch_g;
    f64x4 acc[kPairs];
#pragma unroll
    for (int p = 0; p < kPairs; ++p) acc[p] = f64x4{0, 0, 0, 0};
    const int64_t end = min((blockIdx.x + 1) * a.part_length, a.length);
    for (int64_t k0 = blockIdx.x * a.part_length + 32 * wave; k0 < end; k0 += 128) {
        In v[BLOCKS][8];
#pragma unroll
        for (int b = 0; b < BLOCKS; ++b) {
            const int i = min(16 * b + l16, a.side - 1);
            if constexpr (TALL) {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const int64_t k = k0 + 4 * e + quarter;
                    v[b][e] = k < end ? g[k * a.ld + i] : (In)0.0f;
                }
            } else {
                const int64_t k = k0 + 8 * quarter;
                load_some<In, 8>(g + (int64_t)i * a.ld + k, end - k, v[b]);
            }
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            double x[BLOCKS];
#pragma unroll
            for (int b = 0; b < BLOCKS; ++b) x[b] = (double)(float)v[b][e];
#pragma unroll
            for (int i = 0; i < BLOCKS; ++i)
#pragma unroll
                for (int j = 0; j < BLOCKS; ++j)
                    if (j <= i) acc[i * (i + 1) / 2 + j] = __builtin_amdgcn_mfma_f64_16x16x4f64(x[i], x[j], acc[i * (i + 1) / 2 + j], 0, 0, 0);
        }
    }
    if (wave > 0) {
#pragma unroll
        for (int p = 0; p < kPairs; ++p) sums[wave - 1][p][lane] = acc[p];
    }
    __syncthreads();
    if (wave == 0) {
        f64x4 *to = (f64x4 *)a.grams + ((int64_t)blockIdx.y * a.parts + blockIdx.x) * kPairs * 64;
#pragma unroll
        for (int p = 0; p < kPairs; ++p) to[p * 64 + lane] = acc[p] + sums[0][p][lane] + sums[1][p][lane] + sums[2][p][lane];
    }
}

// The iteration on one matrix's S, a wavefront a block of 16×16 of the results
// (with one block the other three help to add S's parts up).  Bound by the chain
// of 17 products, 4·BLOCKS instructions each.
template <int BLOCKS>
constexpr int kIterate = BLOCKS == 1 ? 256 : 64 * BLOCKS * BLOCKS;
template <int BLOCKS>
__global__ __launch_bounds__(kIterate<BLOCKS>) void iterate_kernel(SmallArgs a)
{
    constexpr int N = 16 * BLOCKS, kLd = N + 2, kPairs = BLOCKS * (BLOCKS + 1) / 2;
    __shared__ double S[N * kLd], P[N * kLd], Q[N * kLd], W[N * kLd];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, l16 = lane & 15, quarter = lane >> 4;
    const int bi = BLOCKS == 1 ? 0 : wave / BLOCKS, bj = BLOCKS == 1 ? 0 : wave % BLOCKS;

    // S, both halves, from its parts; zero past the side, where the loads stood in
    const double *from = a.grams + (int64_t)blockIdx.x * a.parts * kPairs * 256;
    for (int n = threadIdx.x; n < kPairs * 256; n += blockDim.x) {
        double sum = 0;
        for (int p = 0; p < a.parts; p += 8) {  // eight parts on their way at once
            double next[8];
#pragma unroll
            for (int u = 0; u < 8; ++u) next[u] = p + u < a.parts ? from[(int64_t)(p + u) * kPairs * 256 + n] : 0.0;
#pragma unroll
            for (int u = 0; u < 8; ++u) sum += next[u];
        }
        const int pair = n / 256, at = n / 4 % 64, r = n % 4;
        const int ib = pair == 0 ? 0 : pair < 3 ? 1 : pair < 6 ? 2 : 3, jb = pair - ib * (ib + 1) / 2;
        const int i = 16 * ib + 4 * r + at / 16, j = 16 * jb + at % 16;
        const double v = i < a.side && j < a.side ? sum : 0;
        S[i * kLd + j] = v;
        S[j * kLd + i] = v;
    }
    __syncthreads();
    double trace = lane < a.side ? S[lane * kLd + lane] : 0.0;
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) trace += __shfl_xor(trace, d);
    __syncthreads();
    const double scale = 1 / (sqrt(trace) + (double)a.eps);
    for (int n = threadIdx.x; n < N * N; n += blockDim.x) S[n / N * kLd + n % N] *= scale * scale;
    __syncthreads();
    if (BLOCKS == 1 && wave > 0) return;  // one wavefront needs no barrier with the others

    auto multiply = [&](const double *x, const double *y) {
        f64x4 acc{0, 0, 0, 0};
#pragma unroll
        for (int k = 0; k < N; k += 4)
            acc = __builtin_amdgcn_mfma_f64_16x16x4f64(x[(16 * bi + l16) * kLd + k + quarter],
                                                       y[(k + quarter) * kLd + 16 * bj + l16], acc, 0, 0, 0);
        return acc;
    };
    auto store = [&](double *to, const f64x4 &v) {
#pragma unroll
        for (int r = 0; r < 4; ++r) to[(16 * bi + 4 * r + quarter) * kLd + 16 * bj + l16] = v[r];
    };
    // what the others stored is there; a wavefront's own LDS accesses come in order
    auto settle = [&]() {
        if constexpr (BLOCKS > 1) __syncthreads();
        else __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    };
    f64x4 q{};
    for (int step = 0; step < a.steps; ++step) {
        const double c0 = a.coefficients[3 * step], c1 = a.coefficients[3 * step + 1], c2 = a.coefficients[3 * step + 2];
        f64x4 p = multiply(S, S);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int i = 16 * bi + 4 * r + quarter, j = 16 * bj + l16;
            p[r] = c2 * p[r] + c1 * S[i * kLd + j] + (i == j ? c0 : 0.0);
        }
        store(P, p);
        settle();
        q = step == 0 ? p : multiply(P, Q);
        if (step + 1 == a.steps) break;
        store(W, multiply(S, P));
        settle();
        store(Q, q);
        store(S, multiply(P, W));
        settle();
    }
    double *to = a.factor + (int64_t)blockIdx.x * N * N;
#pragma unroll
    for (int r = 0; r < 4; ++r) to[(16 * bi + 4 * r + quarter) * N + 16 * bj + l16] = q[r] * scale;
}

template <class Out, int N>
__device__ __forceinline__ void put(Out *to, const double (&v)[N], int64_t left)
{
    if (left >= N) {
        typename Some<Out, N>::type w;
#pragma unroll
        for (int e = 0; e < N; ++e) w[e] = (Out)(float)v[e];
        *(typename Some<Out, N>::type *)to = w;
    } else {
#pragma unroll
        for (int e = 0; e < N; ++e)
            if (e < left) to[e] = (Out)(float)v[e];
    }
}

// The result: Q·G, or G·Q (tall), 64 columns (rows) a wavefront.  The sum's
// rounding to float32 before that to 16 bits is 2^-16 of the latter's.
template <class In, int BLOCKS, bool TALL>
__global__ __launch_bounds__(256) void apply_kernel(SmallArgs a)
{
    constexpr int N = 16 * BLOCKS, kLd = N + 2;
    __shared__ double Q[N * kLd];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, l16 = lane & 15, quarter = lane >> 4;
    const double *factor = a.factor + (int64_t)blockIdx.y * N * N;
    for (int n = threadIdx.x; n < N * N; n += 256) Q[n / N * kLd + n % N] = factor[n];
    __syncthreads();
    const In *g = (const In *)a.G + blockIdx.y * a.batch_g;
    In *out = (In *)a.out + blockIdx.y * a.batch_o;
    const int64_t x0 = ((int64_t)blockIdx.x * 4 + wave) * 64;
    if (x0 >= a.length) return;
    f64x4 acc[BLOCKS][4];
#pragma unroll
    for (int b = 0; b < BLOCKS; ++b)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[b][e] = f64x4{0, 0, 0, 0};
    if constexpr (!TALL) {
        // block e of columns: x0 + 4·l16 + e
        const int64_t col = x0 + 4 * l16, left = a.length - col;
#pragma unroll
        for (int k = 0; k < N; k += 4) {
            In v[4];
            // rows past the side meet zeros of Q
            load_some<In, 4>(g + (int64_t)min(k + quarter, a.side - 1) * a.ld + col, left, v);
#pragma unroll
            for (int b = 0; b < BLOCKS; ++b) {
                const double q = Q[(16 * b + l16) * kLd + k + quarter];
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[b][e] = __builtin_amdgcn_mfma_f64_16x16x4f64(q, (double)(float)v[e], acc[b][e], 0, 0, 0);
            }
        }
#pragma unroll
        for (int b = 0; b < BLOCKS; ++b)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int row = 16 * b + 4 * r + quarter;
                const double v[4] = {acc[b][0][r], acc[b][1][r], acc[b][2][r], acc[b][3][r]};
                if (row < a.side && left > 0) put<In, 4>(out + (int64_t)row * a.ldo + col, v, left);
            }
    } else {
        // block e of rows: x0 + 16·e + l16.  Q's columns are taken in an order
        // that gives a lane four adjacent ones.
        const int turned = 4 * (l16 & 3) + (l16 >> 2);
#pragma unroll
        for (int k = 0; k < N; k += 32) {
            In v[4][8];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int64_t row = min(x0 + 16 * e + l16, a.length - 1);
                load_some<In, 8>(g + row * a.ld + k + 8 * quarter, a.side - (k + 8 * quarter), v[e]);
            }
#pragma unroll
            for (int s = 0; s < 8; ++s) {
                const int j = k + 8 * quarter + s;
#pragma unroll
                for (int b = 0; b < BLOCKS; ++b) {
                    const double q = j < N ? Q[j * kLd + 16 * b + turned] : 0;
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        acc[b][e] = __builtin_amdgcn_mfma_f64_16x16x4f64(q, (double)(float)v[e][s], acc[b][e], 0, 0, 0);
                }
            }
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int64_t row = x0 + 16 * e + l16;
            if (row >= a.length) continue;
#pragma unroll
            for (int b = 0; b < BLOCKS; ++b) {
                // result (4·r + quarter) of the block is column 4·quarter + r
                const int col = 16 * b + 4 * quarter;
                const double v[4] = {acc[b][e][0], acc[b][e][1], acc[b][e][2], acc[b][e][3]};
                if (col < a.side) put<In, 4>(out + row * a.ldo + col, v, a.side - col);
            }
        }
    }
}

template <class In, int BLOCKS>
void grams(const SmallArgs &a, hipStream_t stream)
{
    const dim3 grid(a.parts, a.batch);
    if (a.tall) gram_kernel<In, BLOCKS, true><<<grid, 256, 0, stream>>>(a);
    else gram_kernel<In, BLOCKS, false><<<grid, 256, 0, stream>>>(a);
}
template <class In, int BLOCKS>
void apply(const SmallArgs &a, hipStream_t stream)
{
    const dim3 grid((unsigned)((a.length + 255) / 256), a.batch);
    if (a.tall) apply_kernel<In, BLOCKS, true><<<grid, 256, 0, stream>>>(a);
    else apply_kernel<In, BLOCKS, false><<<grid, 256, 0, stream>>>(a);
}
template <class In>
void grams(const SmallArgs &a, hipStream_t stream)
{
    switch (blocks_of(a.side)) {
    case 1: return grams<In, 1>(a, stream);
    case 2: return grams<In, 2>(a, stream);
    default: return grams<In, 4>(a, stream);
    }
}
template <class In>
void apply(const SmallArgs &a, hipStream_t stream)
{
    switch (blocks_of(a.side)) {
    case 1: return apply<In, 1>(a, stream);
    case 2: return apply<In, 2>(a, stream);
    default: return apply<In, 4>(a, stream);
    }
}

}  // namespace

hipError_t launch_squares(const SplitArgs &a, hipStream_t stream)
{
    const dim3 grid(a.parts, a.batch);
    if (a.dtype == TGEMM_F32) squares_kernel<float><<<grid, 256, 0, stream>>>(a);
    else if (a.dtype == TGEMM_BF16) squares_kernel<__bf16><<<grid, 256, 0, stream>>>(a);
    else squares_kernel<_Float16><<<grid, 256, 0, stream>>>(a);
    return hipGetLastError();
}

hipError_t launch_split(const SplitArgs &a, hipStream_t stream)
{
    const int64_t pieces = a.rows_out * (a.ldo / 8), blocks = (pieces + 1023) / 1024;
    const dim3 grid((unsigned)(blocks < 4096 ? blocks : 4096), a.batch);
    if (a.dtype == TGEMM_F32) split_kernel<float><<<grid, 256, 0, stream>>>(a);
    else if (a.dtype == TGEMM_BF16) split_kernel<__bf16><<<grid, 256, 0, stream>>>(a);
    else split_kernel<_Float16><<<grid, 256, 0, stream>>>(a);
    return hipGetLastError();
}

hipError_t launch_grams(const SmallArgs &a, hipStream_t stream)
{
    if (a.dtype == TGEMM_F32) grams<float>(a, stream);
    else if (a.dtype == TGEMM_BF16) grams<__bf16>(a, stream);
    else grams<_Float16>(a, stream);
    return hipGetLastError();
}

hipError_t launch_iterate(const SmallArgs &a, hipStream_t stream)
{
    switch (blocks_of(a.side)) {
    case 1: iterate_kernel<1><<<a.batch, kIterate<1>, 0, stream>>>(a); break;
    case 2: iterate_kernel<2><<<a.batch, kIterate<2>, 0, stream>>>(a); break;
    default: iterate_kernel<4><<<a.batch, kIterate<4>, 0, stream>>>(a); break;
    }
    return hipGetLastError();
}

hipError_t launch_apply(const SmallArgs &a, hipStream_t stream)
{
    if (a.dtype == TGEMM_F32) apply<float>(a, stream);
    else if (a.dtype == TGEMM_BF16) apply<__bf16>(a, stream);
    else apply<_Float16>(a, stream);
    return hipGetLastError();
}

}  // namespace ortho
}  // namespace tgemm
