// Passes over rows for the loss operators: operands laid out for the matrix
// cores, partial statistics joined into losses, the teacher's entries, the
// rows' gradient factors and the sum of partial gradients.  Each touches its
// data once and is bound by device memory (or, on few rows, by its launch).
#include "linear_loss.h"

namespace tgemm {
namespace loss {
namespace {

typedef unsigned short u16x8 __attribute__((ext_vector_type(8)));

// No factor of a float32 row can be as low: the largest exponent of rows that all do not count.
constexpr int kNoExponent = -100000;

__device__ __forceinline__ float load_as_float(const void *p, int64_t at, tgemm_dtype_t dtype)
{
    if (dtype == TGEMM_F32) return ((const float *)p)[at];
    if (dtype == TGEMM_BF16) return (float)((const __bf16 *)p)[at];
    return (float)((const _Float16 *)p)[at];
}

// The largest / the sum of a value over the 64 lanes, in every lane.
__device__ __forceinline__ float wave_max(float v)
{
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) v = fmaxf(v, __shfl_xor(v, d));
    return v;
}
__device__ __forceinline__ float wave_sum(float v)
{
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) v += __shfl_xor(v, d);
    return v;
}

// The high part of a float32 as bf16.  A finite value that would round to
// infinity keeps the largest bf16, so that the rest can hold what is missing.
__device__ __forceinline__ __bf16 plane_of(float x)
{
    const __bf16 h = (__bf16)x;
    if (__builtin_isinf((float)h) && !__builtin_isinf(x))
        return __builtin_bit_cast(__bf16, (uint16_t)(0x7F7F | (__builtin_bit_cast(uint32_t, x) >> 16 & 0x8000)));
    return h;
}

__device__ __forceinline__ uint16_t bits(__bf16 v) { return __builtin_bit_cast(uint16_t, v); }
__device__ __forceinline__ uint16_t bits(_Float16 v) { return __builtin_bit_cast(uint16_t, v); }

__global__ __launch_bounds__(256) void linear_copy_kernel(CopyArgs a)
{
    int top = 0;
    if (a.exps != nullptr) {
        __shared__ int best[4];
        int m = kNoExponent;
        for (int b = threadIdx.x; b < a.blocks; b += 256) m = max(m, a.block_max[b]);
#pragma unroll
        for (int d = 32; d > 0; d >>= 1) m = max(m, __shfl_xor(m, d));
        if ((threadIdx.x & 63) == 0) best[threadIdx.x >> 6] = m;
        __syncthreads();
        top = max(max(best[0], best[1]), max(best[2], best[3]));
        if (top == kNoExponent) top = 0;
        if (blockIdx.x == 0 && threadIdx.x == 0) *a.all_scale = ldexpf(1.0f, top - kHalfShift);
    }
    const int64_t per_row = a.ld_out / 8, total = a.rows_out * per_row;
    for (int64_t p = (int64_t)blockIdx.x * 256 + threadIdx.x; p < total; p += (int64_t)gridDim.x * 256) {
        const int64_t row = p / per_row, col = (p - row * per_row) * 8;
        const int left = row < a.rows ? (int)min((int64_t)8, a.cols - col) : 0;
        uint16_t *to = (uint16_t *)a.dst + row * a.ld_out + col;
        const bool counts = left > 0 && (a.coef == nullptr || a.coef[row] != 0.0f);
        u16x8 v[3] = {};
        if (counts && a.dtype == TGEMM_F32) {
            const float *from = (const float *)a.src + row * a.ld + col;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float x = e < left ? from[e] : 0.0f;
                const __bf16 h = plane_of(x);
                const bool finite = !__builtin_isinf(x) && !__builtin_isnan(x);
                const float r = finite ? x - (float)h : 0.0f;
                const __bf16 m = (__bf16)r;
                v[0][e] = bits(h);
                v[1][e] = bits(m);
                v[2][e] = bits((__bf16)(r - (float)m));
            }
        } else if (counts) {
            const uint16_t *from = (const uint16_t *)a.src + row * a.ld + col;
            if (a.vec && left == 8) {
                v[0] = *(const u16x8 *)from;
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e) v[0][e] = e < left ? from[e] : (uint16_t)0;
            }
            if (a.exps != nullptr) {
                const int shift = a.exps[row] - top;
                if (shift != 0) {
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        v[0][e] = bits((_Float16)ldexpf((float)__builtin_bit_cast(_Float16, (uint16_t)v[0][e]), shift));
                }
            }
        }
        *(u16x8 *)to = v[0];
        if (a.planes == 3) {
            *(u16x8 *)(to + a.plane) = v[1];
            *(u16x8 *)(to + 2 * a.plane) = v[2];
        }
    }
}

// A row of the teacher's entries, a wavefront a row: whether any is kept (its
// logit is not -infinity), whether a kept one's id is out of range, and over
// the kept ones the largest logit and the sum of exp((logit - largest)·scale).
struct TeacherRow {
    bool any, bad;
    float high, sum;
};

__device__ __forceinline__ TeacherRow read_teacher(const Teacher &t, int64_t row, int64_t V, int lane)
{
    TeacherRow r;
    bool any = false, bad = false;
    float high = -INFINITY;
    for (int k = lane; k < t.K; k += 64) {
        const float v = load_as_float(t.logits, row * t.ld_logits + k, t.dtype);
        if (v == -INFINITY) continue;
        const int64_t id = t.ids[row * t.ld_ids + k];
        any = true;
        bad |= id < 0 || id >= V;
        high = fmaxf(high, v);
    }
    r.any = __any(any);
    r.bad = __any(bad);
    r.high = wave_max(high);
    float sum = 0.0f;
    for (int k = lane; k < t.K; k += 64) {
        const float v = load_as_float(t.logits, row * t.ld_logits + k, t.dtype);
        if (v != -INFINITY) sum += expf((v - r.high) * t.scale);
    }
    r.sum = wave_sum(sum);
    return r;
}

// A wavefront a row: the pairs (maximum, sum) of its column groups joined,
// then the row's loss.
__global__ __launch_bounds__(256) void linear_join_kernel(JoinArgs a, Teacher t, bool distill)
{
    const int64_t row = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
    const int lane = threadIdx.x & 63;
    if (row >= a.T) return;
    const float2 *part = a.part + row * a.groups;
    float high = -INFINITY, sum = 0.0f;
    for (int g = lane; g < a.groups; g += 64) {
        const float2 p = part[g];
        const float to = fmaxf(high, p.x);
        if (to != -INFINITY) sum = sum * __builtin_amdgcn_exp2f(high - to) + p.y * __builtin_amdgcn_exp2f(p.x - to);
        else sum += p.y;  // nothing yet, or a NaN
        high = to;
    }
    const float top = wave_max(high);
    sum = wave_sum(top == -INFINITY ? sum : sum * __builtin_amdgcn_exp2f(high - top));
    const float lse = fmaf(top, 0.693147180559945309417f, logf(sum));
    if (lane == 0) a.lse[row] = lse;
    if (!distill) {
        if (lane == 0) {
            const int64_t y = a.target[row];
            a.loss[row] = y == a.ignore ? 0.0f : y < 0 || y >= a.V ? NAN : lse - a.picked[row];
            if (a.counted != nullptr) a.counted[row] = y != a.ignore;
        }
        return;
    }
    const TeacherRow r = read_teacher(t, row, a.V, lane);
    const float log_sum = logf(r.sum);
    float loss = 0.0f;
    for (int k = lane; k < t.K; k += 64) {
        const float v = load_as_float(t.logits, row * t.ld_logits + k, t.dtype);
        if (v == -INFINITY) continue;
        const float d = (v - r.high) * t.scale;
        const float q = expf(d) / r.sum;
        // an entry whose probability is below the least float32 adds nothing
        if (q != 0.0f) loss += q * (d - log_sum - (a.student[row * t.K + k] - lse));
    }
    loss = wave_sum(loss) / (t.scale * t.scale);
    if (lane == 0) {
        a.loss[row] = !r.any ? 0.0f : r.bad ? NAN : loss;
        if (a.counted != nullptr) a.counted[row] = r.any;
    }
}

// One work-group: the order of the sum does not depend on timing.
__global__ __launch_bounds__(1024) void linear_summary_kernel(int64_t T, const float *loss, const int *counted,
                                                              float *summary)
{
    __shared__ double sums[16];
    __shared__ int counts[16];
    double sum = 0.0;
    int count = 0;
    for (int64_t t = threadIdx.x; t < T; t += 1024) {
        sum += (double)loss[t];
        count += counted[t];
    }
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) {
        sum += __shfl_xor(sum, d);
        count += __shfl_xor(count, d);
    }
    if ((threadIdx.x & 63) == 0) {
        sums[threadIdx.x >> 6] = sum;
        counts[threadIdx.x >> 6] = count;
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int w = 1; w < 16; ++w) {
            sum += sums[w];
            count += counts[w];
        }
        const double n = count > 0 ? (double)count : 1.0;
        summary[0] = (float)sum;
        summary[1] = (float)(sum / n);
        summary[2] = (float)(1.0 / n);
    }
}

// Eight adjacent values of a row, `left` of which are there.
__device__ __forceinline__ void load8(const void *p, int64_t at, tgemm_dtype_t dtype, bool vec, int64_t left,
                                      float (&v)[8])
{
    if (vec && left >= 8) {
        if (dtype == TGEMM_F32) {
            const m16::f32x4 *q = (const m16::f32x4 *)((const float *)p + at);
            const m16::f32x4 lo = q[0], hi = q[1];
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = e < 4 ? lo[e & 3] : hi[e & 3];
        } else {
            const u16x8 w = *(const u16x8 *)((const uint16_t *)p + at);
#pragma unroll
            for (int e = 0; e < 8; ++e)
                v[e] = dtype == TGEMM_BF16 ? (float)__builtin_bit_cast(__bf16, (uint16_t)w[e])
                                           : (float)__builtin_bit_cast(_Float16, (uint16_t)w[e]);
        }
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = e < left ? load_as_float(p, at + e, dtype) : 0.0f;
    }
}

// A wavefront takes kTogether entries of a row at a time, so that as many
// rows of W are on their way.
__global__ __launch_bounds__(256) void linear_pick_kernel(PickArgs a)
{
    constexpr int kTogether = 8;
    const int64_t row = blockIdx.x;
    const int lane = threadIdx.x & 63, K = a.teacher.K;
    for (int k0 = (threadIdx.x >> 6) * kTogether; k0 < K; k0 += 4 * kTogether) {
        int64_t id[kTogether];
        float sum[kTogether];
#pragma unroll
        for (int j = 0; j < kTogether; ++j) {
            const int k = min(k0 + j, K - 1);
            const float v = load_as_float(a.teacher.logits, row * a.teacher.ld_logits + k, a.teacher.dtype);
            id[j] = a.teacher.ids[row * a.teacher.ld_ids + k];
            sum[j] = v == -INFINITY ? 0.0f : id[j] < 0 || id[j] >= a.V ? NAN : 0.0f;
            // an entry that is absent or out of range adds nothing: row 0 stands in for it
            if (v == -INFINITY || id[j] < 0 || id[j] >= a.V) id[j] = -1;
        }
        for (int64_t d = lane * 8; d < a.D; d += 512) {
            float x[8];
            load8(a.X, row * a.ldx + d, a.dtype, a.vec, a.D - d, x);
            float w[kTogether][8];
#pragma unroll
            for (int j = 0; j < kTogether; ++j) load8(a.W, max(id[j], (int64_t)0) * a.ldw + d, a.dtype, a.vec, a.D - d, w[j]);
#pragma unroll
            for (int j = 0; j < kTogether; ++j)
#pragma unroll
                for (int e = 0; e < 8; ++e) sum[j] = id[j] < 0 ? sum[j] : fmaf(x[e], w[j][e], sum[j]);
        }
#pragma unroll
        for (int j = 0; j < kTogether; ++j) {
            sum[j] = wave_sum(sum[j]) * a.teacher.scale;
            if (lane == j && k0 + j < K) a.student[row * K + k0 + j] = sum[j];
        }
    }
}

__device__ __forceinline__ float grad_of(const CoefArgs &a, int64_t row)
{
    const float g = a.grad[row * a.grad_step] * a.factor;
    return a.weight != nullptr ? g * *a.weight : g;
}

__device__ __forceinline__ void put_coef(const CoefArgs &a, int64_t row, float c, int &exponent)
{
    exponent = kNoExponent;
    if (a.half) {
        int e = 0;
        if (c != 0.0f && !__builtin_isinf(c) && !__builtin_isnan(c)) {
            c = ldexpf(frexpf(c, &e), kHalfShift);
            exponent = e;
        }
        a.row_scale[row] = ldexpf(1.0f, e - kHalfShift);
        a.exps[row] = e;
    }
    a.coef[row] = c;
}

template <int WAVES>
__device__ __forceinline__ void put_block_max(const CoefArgs &a, int64_t block, int exponent)
{
    if (!a.half) return;
    __shared__ int best[WAVES];
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) exponent = max(exponent, __shfl_xor(exponent, d));
    if ((threadIdx.x & 63) == 0) best[threadIdx.x >> 6] = exponent;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int w = 1; w < WAVES; ++w) exponent = max(exponent, best[w]);
        a.block_max[block] = exponent;
    }
}

__global__ __launch_bounds__(256) void linear_ce_coef_kernel(CoefArgs a)
{
    const int64_t row = (int64_t)blockIdx.x * 256 + threadIdx.x;
    int exponent = kNoExponent;
    if (row < a.T) {
        const int64_t y = a.target[row];
        put_coef(a, row, y == a.ignore ? 0.0f : y < 0 || y >= a.V ? NAN : grad_of(a, row), exponent);
    }
    put_block_max<4>(a, blockIdx.x, exponent);
}

// A wavefront a row.
__global__ __launch_bounds__(1024) void linear_kd_coef_kernel(CoefArgs a, Teacher t)
{
    const int64_t row = (int64_t)blockIdx.x * 16 + (threadIdx.x >> 6);
    const int lane = threadIdx.x & 63;
    int exponent = kNoExponent;
    if (row < a.T) {
        bool any = false, bad = false;
        for (int k = lane; k < t.K; k += 64) {
            const int64_t id = t.ids[row * t.ld_ids + k];
            if (load_as_float(t.logits, row * t.ld_logits + k, t.dtype) == -INFINITY) continue;
            any = true;
            bad |= id < 0 || id >= a.V;
        }
        any = __any(any);
        bad = __any(bad);
        if (lane == 0) put_coef(a, row, !any ? 0.0f : bad ? NAN : grad_of(a, row), exponent);
    }
    put_block_max<16>(a, blockIdx.x, exponent);
}

// A wavefront a row.  An id that comes twice holds the sum of its entries in
// both places; the same value is then written twice.
__global__ __launch_bounds__(64) void linear_scatter_kernel(ScatterArgs a)
{
    extern __shared__ char room[];
    const Teacher &t = a.teacher;
    int64_t *ids = (int64_t *)room;
    float *q = (float *)(ids + t.K);
    const int64_t row = blockIdx.x;
    const int lane = threadIdx.x;
    const float c = a.coef[row];
    if (c == 0.0f) return;
    const TeacherRow r = read_teacher(t, row, INT64_MAX, lane);
    for (int k = lane; k < t.K; k += 64) {
        const float v = load_as_float(t.logits, row * t.ld_logits + k, t.dtype);
        const bool kept = v != -INFINITY;
        ids[k] = kept ? t.ids[row * t.ld_ids + k] : -1;
        q[k] = kept ? expf((v - r.high) * t.scale) / r.sum : 0.0f;
    }
    __syncthreads();
    for (int k = lane; k < t.K; k += 64) {
        const int64_t id = ids[k], at = id - a.v0;
        if (id < 0 || at < 0 || at >= a.cols) continue;
        float sum = 0.0f;
        for (int j = 0; j < t.K; ++j) sum += ids[j] == id ? q[j] : 0.0f;
        float g = c * (expf(a.student[row * t.K + k] - a.lse[row]) - sum);
        uint16_t *to = (uint16_t *)a.G + row * a.ldg + at;
        if (a.half) {
            *to = bits((_Float16)g);
        } else {
            for (int p = 0; p < a.planes; ++p) {
                const __bf16 h = (__bf16)g;
                to[p * a.plane] = bits(h);
                g -= (float)h;
            }
        }
    }
}

__device__ __forceinline__ void store_as(void *p, int64_t at, tgemm_dtype_t dtype, float v)
{
    if (dtype == TGEMM_F32) ((float *)p)[at] = v;
    else if (dtype == TGEMM_BF16) ((__bf16 *)p)[at] = (__bf16)v;
    else ((_Float16 *)p)[at] = (_Float16)v;
}

// Four columns a thread; the parts' rows are padded to a multiple of 64.
__global__ __launch_bounds__(256) void linear_sum_kernel(SumArgs a)
{
    const int64_t per_row = (a.D + 3) / 4, total = a.T * per_row;
    for (int64_t p = (int64_t)blockIdx.x * 256 + threadIdx.x; p < total; p += (int64_t)gridDim.x * 256) {
        const int64_t row = p / per_row, col = (p - row * per_row) * 4;
        const float *part = a.part + row * a.ld + col;
        m16::f32x4 v = *(const m16::f32x4 *)part;
        for (int s = 1; s < a.count; ++s) v += *(const m16::f32x4 *)(part + s * a.stride);
        if (a.row_scale != nullptr) v *= a.row_scale[row];
        const int64_t at = row * a.ldo + col;
        if (a.vec && col + 4 <= a.D) {
            if (a.dtype == TGEMM_F32) {
                *(m16::f32x4 *)((float *)a.out + at) = v;
            } else {
                uint16_t w[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) w[e] = a.dtype == TGEMM_BF16 ? bits((__bf16)v[e]) : bits((_Float16)v[e]);
                *(uint2 *)((uint16_t *)a.out + at) = make_uint2(w[0] | (uint32_t)w[1] << 16, w[2] | (uint32_t)w[3] << 16);
            }
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (col + e < a.D) store_as(a.out, at + e, a.dtype, v[e]);
        }
    }
}

__global__ __launch_bounds__(256) void linear_zero_kernel(void *out, int64_t ldo, tgemm_dtype_t dtype, int64_t rows,
                                                          int64_t cols)
{
    const int64_t total = rows * cols;
    for (int64_t p = (int64_t)blockIdx.x * 256 + threadIdx.x; p < total; p += (int64_t)gridDim.x * 256) {
        const int64_t row = p / cols;
        store_as(out, row * ldo + (p - row * cols), dtype, 0.0f);
    }
}

unsigned blocks_for(int64_t items)
{
    const int64_t b = (items + 255) / 256;
    return (unsigned)(b < 1 ? 1 : b > 16384 ? 16384 : b);
}

}  // namespace

hipError_t launch_copy(const CopyArgs &a, hipStream_t stream)
{
    linear_copy_kernel<<<blocks_for(a.rows_out * (a.ld_out / 8)), 256, 0, stream>>>(a);
    return hipGetLastError();
}

hipError_t launch_join(const JoinArgs &a, hipStream_t stream)
{
    linear_join_kernel<<<(unsigned)((a.T + 3) / 4), 256, 0, stream>>>(a, a.teacher ? *a.teacher : Teacher{},
                                                                      a.teacher != nullptr);
    return hipGetLastError();
}

hipError_t launch_summary(int64_t T, const float *loss, const int *counted, float *summary, hipStream_t stream)
{
    linear_summary_kernel<<<1, 1024, 0, stream>>>(T, loss, counted, summary);
    return hipGetLastError();
}

hipError_t launch_pick(const PickArgs &a, hipStream_t stream)
{
    linear_pick_kernel<<<(unsigned)a.T, 256, 0, stream>>>(a);
    return hipGetLastError();
}

hipError_t launch_coef(const CoefArgs &a, hipStream_t stream)
{
    const unsigned blocks = (unsigned)coef_blocks(a.T, a.teacher != nullptr);
    if (a.teacher == nullptr) linear_ce_coef_kernel<<<blocks, 256, 0, stream>>>(a);
    else linear_kd_coef_kernel<<<blocks, 1024, 0, stream>>>(a, *a.teacher);
    return hipGetLastError();
}

hipError_t launch_scatter(const ScatterArgs &a, hipStream_t stream)
{
    linear_scatter_kernel<<<(unsigned)a.T, 64, (size_t)a.teacher.K * 12, stream>>>(a);
    return hipGetLastError();
}

hipError_t launch_sum(const SumArgs &a, hipStream_t stream)
{
    linear_sum_kernel<<<blocks_for(a.T * ((a.D + 3) / 4)), 256, 0, stream>>>(a);
    return hipGetLastError();
}

hipError_t launch_zero(void *out, int64_t ldo, tgemm_dtype_t dtype, int64_t rows, int64_t cols, hipStream_t stream)
{
    linear_zero_kernel<<<blocks_for(rows * cols), 256, 0, stream>>>(out, ldo, dtype, rows, cols);
    return hipGetLastError();
}

}  // namespace loss
}  // namespace tgemm
