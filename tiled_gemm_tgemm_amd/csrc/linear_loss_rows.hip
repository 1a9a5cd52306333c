// Passes over rows for the loss operators: operands laid out for the matrix
// cores, partial statistics joined into losses, the teacher's entries, the
// rows' gradient factors and the sum of partial gradients.  Each touches its
// data once and is bound by device memory (or, on few rows, by its launch).
#include "linear_loss.h"
#include "mfma16.h"

namespace tgemm {
namespace loss {
namespace {

typedef unsigned short u16x8 __attribute__((ext_vector_type(8)));
typedef float f32x8 __attribute__((ext_vector_type(8)));
// device memory takes 16-byte loads and stores at any address
typedef u16x8 u16x8_anywhere __attribute__((aligned(2)));
typedef f32x8 f32x8_anywhere __attribute__((aligned(4)));
typedef m16::f32x4 f32x4_anywhere __attribute__((aligned(4)));
typedef uint32_t u32x2_anywhere __attribute__((ext_vector_type(2), aligned(2)));

// The exponent of nothing: a row without a factor of its own, or without a
// state that is neither zero nor infinite.  Lower than any other.
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

__device__ __forceinline__ uint16_t bits(__bf16 v) { return __builtin_bit_cast(uint16_t, v); }
__device__ __forceinline__ uint16_t bits(_Float16 v) { return __builtin_bit_cast(uint16_t, v); }

__device__ __forceinline__ float grad_of(const CoefArgs &a, int64_t row)
{
    const float g = a.grad[row * a.grad_step] * a.factor;
    return a.weight != nullptr ? g * *a.weight : g;
}

enum RowKind { kNotCounted, kCounted, kBad };

// Also returns the exponent of an fp16 row's own factor, kNoExponent where there is none.
__device__ __forceinline__ int put_coef(const CoefArgs &a, int64_t row, RowKind kind)
{
    float coef = kind == kBad ? NAN : 0.0f;
    int exponent = kNoExponent;
    if (a.grad_step == 0) {
        const float shift = a.half ? ldexpf(1.0f, kHalfShift) : 1.0f;
        if (kind == kCounted) coef = shift;
        a.row_scale[row] = kind == kNotCounted ? 0.0f : kind == kBad ? NAN : grad_of(a, 0) / shift;
        if (row == 0) *a.all_scale = grad_of(a, 0) / shift;
    } else {
        if (kind == kCounted) coef = grad_of(a, row);
        if (a.half) {
            int e = 0;
            if (coef != 0.0f && !__builtin_isinf(coef) && !__builtin_isnan(coef)) {
                coef = ldexpf(frexpf(coef, &e), kHalfShift);
                exponent = e;
            }
            a.row_scale[row] = ldexpf(1.0f, e - kHalfShift);
            a.exps[row] = exponent;
        }
    }
    a.coef[row] = coef;
    return exponent;
}

__device__ __forceinline__ RowKind ce_kind(const CoefArgs &a, int64_t row)
{
    const int64_t y = a.target[row];
    return y == a.ignore ? kNotCounted : y < 0 || y >= a.V ? kBad : kCounted;
}

__global__ __launch_bounds__(256) void linear_copy_kernel(CopyArgs a, CoefArgs make, bool making)
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
        // no less than float32 holds, so that a NaN in the sums stays one; the least fp16 is far above
        if (blockIdx.x == 0 && threadIdx.x == 0) *a.all_scale = ldexpf(1.0f, max(top - 2 * kHalfShift, -126));
    }
    const int64_t per_row = a.ld_out / 8, total = a.rows_out * per_row;
    for (int64_t p = (int64_t)blockIdx.x * 256 + threadIdx.x; p < total; p += (int64_t)gridDim.x * 256) {
        const int64_t row = p / per_row, col = (p - row * per_row) * 8;
        const int left = row < a.rows ? (int)min((int64_t)8, a.cols - col) : 0;
        uint16_t *to = (uint16_t *)a.dst + row * a.ld_out + col;
        bool counts = left > 0;
        if (making && row < a.rows) {
            const RowKind kind = ce_kind(make, row);
            if (col == 0) put_coef(make, row, kind);
            counts = counts && kind != kNotCounted;
        } else if (a.coef != nullptr && row < a.rows) {
            counts = counts && a.coef[row] != 0.0f;
        }
        u16x8 v[3] = {};
        if (counts && a.dtype == TGEMM_F32) {
            const float *from = (const float *)a.src + row * a.ld + col;
            f32x8 f{};
            if (left == 8) {
                f = *(const f32x8_anywhere *)from;
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e) f[e] = e < left ? from[e] : 0.0f;
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                __bf16 h, m, l;
                m16::split(f[e], h, m, l);
                v[0][e] = bits(h);
                v[1][e] = bits(m);
                v[2][e] = bits(l);
            }
        } else if (counts) {
            const uint16_t *from = (const uint16_t *)a.src + row * a.ld + col;
            if (left == 8) {
                v[0] = *(const u16x8_anywhere *)from;
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e) v[0][e] = e < left ? from[e] : (uint16_t)0;
            }
            if (a.exps != nullptr) {
                const int e = a.exps[row], shift = e == kNoExponent ? 0 : kHalfShift + e - top;
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

constexpr int kSortChunk = 4096;

// A wavefront a row: its entries are counted by column group, the counts are
// summed, and each entry goes to its group's start and its number within the
// group.  That number is whatever the LDS atomic gave: the order within a group
// decides nothing, as each entry is looked up for itself.  `chunk` groups (a
// multiple of 64) at a time have their counts in LDS.  Bound by the latency of
// its loads: 2048 rows of 100 entries in 782 groups 8 µs, 16 rows of 16 5 µs
// (sorting the ids in LDS and searching the groups' starts took 18 and 7).
__global__ __launch_bounds__(64) void linear_sort_kernel(SortArgs a, int chunk)
{
    extern __shared__ uint32_t counts[];
    uint32_t *ids = counts + chunk, *numbers = ids + a.teacher.K;
    const Teacher &t = a.teacher;
    const int64_t row = blockIdx.x;
    const int lane = threadIdx.x;
    const int shift = __builtin_ctz(a.columns);  // a power of two
    constexpr uint32_t kAbsent = ~0u;
    for (int k = lane; k < t.K; k += 64) {
        const float v = load_as_float(t.logits, row * t.ld_logits + k, t.dtype);
        const int64_t id = t.ids[row * t.ld_ids + k];
        ids[k] = kAbsent;
        if (v == -INFINITY) a.student[row * t.K + k] = 0.0f;
        else if (id < 0 || id >= a.V) a.student[row * t.K + k] = NAN;
        else ids[k] = (uint32_t)id;
    }
    uint16_t *starts = a.starts + row * (a.groups + 1);
    uint32_t before = 0;  // entries of earlier chunks
    for (int first = 0; first < a.groups; first += chunk) {
        for (int g = lane; g < chunk; g += 64) counts[g] = 0;
        __syncthreads();
        for (int k = lane; k < t.K; k += 64) {
            const uint32_t group = (ids[k] >> shift) - (uint32_t)first;  // absent: past every chunk
            if (ids[k] != kAbsent && group < (uint32_t)chunk) numbers[k] = atomicAdd(&counts[group], 1u);
        }
        __syncthreads();
        const int each = chunk / 64, from = lane * each;
        uint32_t mine = 0;
        for (int g = from; g < from + each; ++g) mine += counts[g];
        uint32_t upto = mine;
#pragma unroll
        for (int d = 1; d < 64; d *= 2) {
            const uint32_t other = __shfl_up(upto, d);
            if (lane >= d) upto += other;
        }
        uint32_t at = before + upto - mine;
        for (int g = from; g < from + each; ++g) {
            const uint32_t n = counts[g];
            counts[g] = at;
            at += n;
        }
        before += __shfl(upto, 63);
        __syncthreads();
        for (int g = lane; g < chunk && first + g < a.groups; g += 64) starts[first + g] = (uint16_t)counts[g];
        for (int k = lane; k < t.K; k += 64) {
            const uint32_t group = (ids[k] >> shift) - (uint32_t)first;
            if (ids[k] != kAbsent && group < (uint32_t)chunk)
                a.list[row * t.K + counts[group] + numbers[k]] = (ids[k] & (uint32_t)(a.columns - 1)) | (uint32_t)k << 8;
        }
        __syncthreads();
    }
    if (lane == 0) starts[a.groups] = (uint16_t)before;
}

// The sum of the losses and the number of rows that count, by one work-group:
// their order does not depend on timing.
template <int WAVES>
__device__ __forceinline__ void write_summary(int64_t T, const float *loss, const int *counted, float *summary)
{
    __shared__ double sums[WAVES];
    __shared__ int counts[WAVES];
    double sum = 0.0;
    int count = 0;
    for (int64_t i = threadIdx.x; i < T; i += 64 * WAVES) {
        sum += (double)loss[i];
        count += counted[i];
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
        for (int w = 1; w < WAVES; ++w) {
            sum += sums[w];
            count += counts[w];
        }
        const double n = count > 0 ? (double)count : 1.0;
        summary[0] = (float)sum;
        summary[1] = (float)(sum / n);
        summary[2] = (float)(1.0 / n);
    }
}

// A wavefront a row: the pairs (maximum, sum) of its column groups joined,
// eight a lane at once (their way here is what a row waits for), then the
// row's loss.  SUMMARY: one work-group takes all rows, and the summary.
constexpr int kAtOnce = 8;
template <int WAVES, bool SUMMARY>
__global__ __launch_bounds__(64 * WAVES) void linear_join_kernel(JoinArgs a, Teacher t, bool distill)
{
    const int lane = threadIdx.x & 63;
    for (int64_t row = (int64_t)blockIdx.x * WAVES + (threadIdx.x >> 6); row < a.T; row += (int64_t)gridDim.x * WAVES) {
        const float2 *part = a.part + row * a.groups;
        int64_t y = 0;
        float picked = 0.0f;
        if (!distill) {
            y = a.target[row];
            picked = a.picked[row];  // nothing was written there for a target out of range
        }
        float high = -INFINITY, sum = 0.0f;
        for (int g = lane; g < a.groups; g += 64 * kAtOnce) {
            float2 p[kAtOnce];
#pragma unroll
            for (int u = 0; u < kAtOnce; ++u)
                p[u] = g + 64 * u < a.groups ? part[g + 64 * u] : make_float2(-INFINITY, 0.0f);
            float to = high;
#pragma unroll
            for (int u = 0; u < kAtOnce; ++u) to = fmaxf(to, p[u].x);
            const float from = to == -INFINITY ? 0.0f : to;  // nothing yet, or a NaN in the sums
            sum *= __builtin_amdgcn_exp2f(high - from);
#pragma unroll
            for (int u = 0; u < kAtOnce; ++u) sum += p[u].y * __builtin_amdgcn_exp2f(p[u].x - from);
            high = to;
        }
        const float top = wave_max(high);
        sum = wave_sum(top == -INFINITY ? sum : sum * __builtin_amdgcn_exp2f(high - top));
        const float lse = fmaf(top, 0.693147180559945309417f, logf(sum));
        float loss;
        bool counts;
        if (!distill) {
            counts = y != a.ignore;
            loss = !counts ? 0.0f : y < 0 || y >= a.V ? NAN : lse - picked;
        } else {
            const TeacherRow r = read_teacher(t, row, a.V, lane);
            const float log_sum = logf(r.sum);
            loss = 0.0f;
            for (int k = lane; k < t.K; k += 64) {
                const float v = load_as_float(t.logits, row * t.ld_logits + k, t.dtype);
                if (v == -INFINITY) continue;
                const float d = (v - r.high) * t.scale;
                const float q = expf(d) / r.sum;
                // an entry whose probability is below the least float32 adds nothing
                if (q != 0.0f) loss += q * (d - log_sum - (a.student[row * t.K + k] - lse));
            }
            loss = wave_sum(loss) / (t.scale * t.scale);
            counts = r.any;
            loss = !counts ? 0.0f : r.bad ? NAN : loss;
        }
        if (lane == 0) {
            a.lse[row] = lse;
            a.loss[row] = loss;
            if (a.summary != nullptr) a.counted[row] = counts;
        }
    }
    if (!SUMMARY) return;

    // the whole batch is in this work-group
    __syncthreads();
    write_summary<WAVES>(a.T, a.loss, a.counted, a.summary);
}

__global__ __launch_bounds__(1024) void linear_summary_kernel(int64_t T, const float *loss, const int *counted,
                                                              float *summary)
{
    write_summary<16>(T, loss, counted, summary);
}

template <int WAVES>
__device__ __forceinline__ void put_block_max(const CoefArgs &a, int64_t block, int exponent)
{
    if (!a.half || a.grad_step == 0) return;
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

// The exponent of a row's largest finite fp16 state, kNoExponent where all are zero.
__device__ __forceinline__ int state_exponent(const CoefArgs &a, int64_t row, int lane)
{
    const uint16_t *x = (const uint16_t *)a.X + row * a.ldx;
    uint32_t most = 0;
    auto take = [&](uint16_t v) {
        const uint32_t size = v & 0x7FFF;
        if (size < 0x7C00 && size > most) most = size;
    };
    for (int64_t col = lane * 8; col < a.D; col += 512) {
        if (col + 8 <= a.D) {
            const u16x8 v = *(const u16x8_anywhere *)(x + col);
#pragma unroll
            for (int e = 0; e < 8; ++e) take(v[e]);
        } else {
            for (int64_t e = col; e < a.D; ++e) take(x[e]);
        }
    }
    const float high = wave_max((float)__builtin_bit_cast(_Float16, (uint16_t)most));
    int exponent = kNoExponent;
    if (high != 0.0f) frexpf(high, &exponent);
    return exponent;
}

// A wavefront a row: its factor, and where that is an fp16 row's own, the
// exponent of the largest product of factor and state.  Bound by reading X for
// the latter (4096×2048 9 µs; without it, the entries of a teacher read
// instead, 5), about 1% of the products that follow.
__global__ __launch_bounds__(1024) void linear_coef_kernel(CoefArgs a, Teacher t, bool distill)
{
    const int64_t row = (int64_t)blockIdx.x * kCoefRows + (threadIdx.x >> 6);
    const int lane = threadIdx.x & 63;
    int exponent = kNoExponent;
    if (row < a.T) {
        RowKind kind;
        if (distill) {
            bool any = false, bad = false;
            for (int k = lane; k < t.K; k += 64) {
                const int64_t id = t.ids[row * t.ld_ids + k];
                if (load_as_float(t.logits, row * t.ld_logits + k, t.dtype) == -INFINITY) continue;
                any = true;
                bad |= id < 0 || id >= a.V;
            }
            any = __any(any);
            bad = __any(bad);
            kind = !any ? kNotCounted : bad ? kBad : kCounted;
        } else {
            kind = ce_kind(a, row);
        }
        int own = kNoExponent;
        if (lane == 0) own = put_coef(a, row, kind);
        own = __shfl(own, 0);
        if (own != kNoExponent) {
            const int state = state_exponent(a, row, lane);
            if (state != kNoExponent) exponent = own + state;
        }
    }
    put_block_max<kCoefRows>(a, blockIdx.x, exponent);
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
        for (int p = 0; p < a.planes; ++p) {
            if (a.half) {
                const _Float16 h = (_Float16)g;
                to[p * a.plane] = bits(h);
                g -= (float)h;
            } else {
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

// Four columns a thread; the parts' rows are padded to a multiple of 64.  Bound
// by memory where there is much (two parts of 4096×2048 to bf16, 84 MB, 18.7
// µs), by the way there and back where there is little (64 parts of 33×512 7).
__global__ __launch_bounds__(256) void linear_sum_kernel(SumArgs a)
{
    const int64_t per_row = (a.D + 3) / 4, total = a.T * per_row;
    for (int64_t p = (int64_t)blockIdx.x * 256 + threadIdx.x; p < total; p += (int64_t)gridDim.x * 256) {
        const int64_t row = p / per_row, col = (p - row * per_row) * 4;
        const float *part = a.part + row * a.ld + col;
        m16::f32x4 v = *(const m16::f32x4 *)part;
        for (int s = 1; s < a.count; s += 8) {  // eight parts on their way at once
            m16::f32x4 next[8];
#pragma unroll
            for (int u = 0; u < 8; ++u)
                next[u] = s + u < a.count ? *(const m16::f32x4 *)(part + (s + u) * a.stride) : m16::f32x4{};
#pragma unroll
            for (int u = 0; u < 8; ++u) v += next[u];
        }
        const float scale = a.row_scale != nullptr ? a.row_scale[row] : a.all_scale != nullptr ? *a.all_scale : 1.0f;
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = m16::mul_zero(scale, v[e]);
        const int64_t at = row * a.ldo + col;
        if (col + 4 <= a.D) {
            if (a.dtype == TGEMM_F32) {
                *(f32x4_anywhere *)((float *)a.out + at) = v;
            } else {
                uint16_t w[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) w[e] = a.dtype == TGEMM_BF16 ? bits((__bf16)v[e]) : bits((_Float16)v[e]);
                *(u32x2_anywhere *)((uint16_t *)a.out + at) =
                    u32x2_anywhere{w[0] | (uint32_t)w[1] << 16, w[2] | (uint32_t)w[3] << 16};
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
    linear_copy_kernel<<<blocks_for(a.rows_out * (a.ld_out / 8)), 256, 0, stream>>>(a, a.make ? *a.make : CoefArgs{},
                                                                                     a.make != nullptr);
    return hipGetLastError();
}

// Up to this many rows one work-group joins the statistics and writes the
// summary too: two rows a wavefront one after the other.  Three rows each (33
// rows of distillation) take it 11 µs, against 4.6 and 2.1 of two launches.
// (A counter by which the last of many work-groups finds itself needs fences
// that cost more than the launch: 57 against 13 µs for 3000 rows.)
constexpr int64_t kSoloRows = 32;

hipError_t launch_join(const JoinArgs &a, hipStream_t stream)
{
    const Teacher t = a.teacher ? *a.teacher : Teacher{};
    const bool distill = a.teacher != nullptr;
    if (a.summary != nullptr && a.T <= kSoloRows) {
        linear_join_kernel<16, true><<<1, 1024, 0, stream>>>(a, t, distill);
        return hipGetLastError();
    }
    linear_join_kernel<4, false><<<(unsigned)((a.T + 3) / 4), 256, 0, stream>>>(a, t, distill);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || a.summary == nullptr) return e;
    linear_summary_kernel<<<1, 1024, 0, stream>>>(a.T, a.loss, a.counted, a.summary);
    return hipGetLastError();
}

hipError_t launch_summary_none(float *summary, hipStream_t stream)
{
    linear_summary_kernel<<<1, 1024, 0, stream>>>(0, nullptr, nullptr, summary);
    return hipGetLastError();
}

hipError_t launch_sort(const SortArgs &a, hipStream_t stream)
{
    const int groups = (a.groups + 63) / 64 * 64, chunk = groups < kSortChunk ? groups : kSortChunk;
    linear_sort_kernel<<<(unsigned)a.T, 64, (size_t)(chunk + 2 * a.teacher.K) * 4, stream>>>(a, chunk);
    return hipGetLastError();
}

hipError_t launch_coef(const CoefArgs &a, hipStream_t stream)
{
    const unsigned blocks = (unsigned)coef_blocks(a.T, a.teacher != nullptr);
    linear_coef_kernel<<<blocks, 64 * kCoefRows, 0, stream>>>(a, a.teacher ? *a.teacher : Teacher{}, a.teacher != nullptr);
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
