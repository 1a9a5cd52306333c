// The sums of few columns that low-rank adapters take: a token's product with
// its adapter's first matrix, the tokens in the order of their adapters, and
// the gradients of both matrices.
#include "linear_adapters.h"
#include "mfma16.h"
#include "some.h"

namespace tgemm {
namespace adapters {
namespace {

using m16::bf16x8;
using m16::f32x4;
using m16::Frag;
using m16::load_some;

// Eight values of k with eight values of k of 16 rows each, added to acc: one
// instruction for 16-bit values, eight of four k's for float32.
template <class In>
struct Step {
    typedef typename Frag<In>::type type;
    static __device__ __forceinline__ type make(const In (&v)[8])
    {
        type f;
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = v[e];
        return f;
    }
    static __device__ __forceinline__ f32x4 add(const In (&a)[8], const In (&b)[8], f32x4 acc) { return Frag<In>::mfma(make(a), make(b), acc); }
};
template <>
struct Step<float> {
    static __device__ __forceinline__ f32x4 add(const float (&a)[8], const float (&b)[8], f32x4 acc)
    {
#pragma unroll
        for (int e = 0; e < 8; ++e) acc = __builtin_amdgcn_mfma_f32_16x16x4f32(a[e], b[e], acc, 0, 0, 0);
        return acc;
    }
};

// x = high + low to 2^-17 of itself.
__device__ __forceinline__ void halves(float x, __bf16 &high, __bf16 &low)
{
    high = (__bf16)x;
    float rest = x - (float)high;
    if (__builtin_isinf(rest) || __builtin_isnan(rest)) rest = 0.0f;  // all in the high part
    low = (__bf16)rest;
}

// Four hidden values of a row, from rank `at` on, as the products read them.
template <bool WHOLE>
__device__ __forceinline__ void put_planes(void *planes, int64_t row, int at, int rank, const f32x4 &v, float factor)
{
    const int padded = (int)planes_rank(rank);
    if (at >= padded) return;
    float x[4];
#pragma unroll
    for (int r = 0; r < 4; ++r) x[r] = at + r < rank ? v[r] * factor : 0.0f;
    if constexpr (WHOLE) {
        *(f32x4 *)((float *)planes + row * padded + at) = f32x4{x[0], x[1], x[2], x[3]};
    } else {
        typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
        bf16x4 high, low;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            __bf16 h, l;
            halves(x[r], h, l);
            high[r] = h;
            low[r] = l;
        }
        __bf16 *to = (__bf16 *)planes + row * 2 * padded + at;
        *(bf16x4 *)to = high;
        *(bf16x4 *)(to + padded) = low;
    }
}

// A wavefront takes 16·ROWS rows and, for each adapter that they have, 16·BLOCKS
// ranks at a time: tokens of a sequence share theirs.  Rows are read where they
// lie, once for every adapter among them, and the adapters' matrices from the
// caches.  SHARED, for a few rows: the four wavefronts of a work-group take the
// same 16 rows and every fourth step of the sum each.  Either way `slots`
// work-groups share the adapters among the rows.  Bound by the loads' way there
// and back: one row of 4096 with 16 ranks 3 µs, 48 of 2048 with 32 adapters 5.6,
// 256 of 4096 12.
template <class In, int BLOCKS, int ROWS, bool RANK_INNER, bool SHARED>
__global__ __launch_bounds__(256) void shrink_kernel(ShrinkArgs a)
{
    __shared__ f32x4 sums[SHARED ? 3 : 1][SHARED ? BLOCKS : 1][SHARED ? 64 : 1];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, l16 = lane & 15, quarter = lane >> 4;
    const int64_t row0 = ((int64_t)blockIdx.x * (SHARED ? 1 : 4) + (SHARED ? 0 : wave)) * (16 * ROWS);
    int id[ROWS];
    const In *x[ROWS];
    uint32_t left[ROWS];
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
        const int64_t row = row0 + 16 * i + l16;
        id[i] = -1;
        if (row < a.T) {
            const int64_t n = a.ids[row];
            if (n >= 0 && n < a.c.count) id[i] = (int)n;
        }
        x[i] = (const In *)a.rows + (row < a.T ? row : a.T - 1) * a.ld + 16 * quarter;
        left[i] = (uint32_t)__ballot(id[i] >= 0) & 0xFFFF;
    }
    // Steps of 64 values of k, of which a lane takes 16 adjacent ones in two
    // fragments (both operands alike, so their order is free): a row's loads are
    // whole cache lines.
    constexpr int kStep = SHARED ? 256 : 64;
    const int64_t from = blockIdx.z * a.part_k, last = min(from + a.part_k, a.K), first = from + (SHARED ? 64 * wave : 0);
    for (int n = 0;; ++n) {
        int now = -1;
#pragma unroll
        for (int i = 0; i < ROWS; ++i)
            if (now < 0 && left[i] != 0) now = __builtin_amdgcn_readlane(id[i], __builtin_ctz(left[i]));
        if (now < 0) break;
#pragma unroll
        for (int i = 0; i < ROWS; ++i) left[i] &= ~(uint32_t)__ballot(id[i] == now);
        if (n % a.slots != (int)blockIdx.y) continue;
        const In *c = (const In *)a.c.p + now * a.c.stride;
        // (with one block of 16 the padding to 32 is a second turn's)
        for (int rank0 = 0; rank0 < (a.planes != nullptr ? (int)planes_rank(a.c.rank) : a.c.rank); rank0 += 16 * BLOCKS) {
            f32x4 acc[ROWS][BLOCKS];
#pragma unroll
            for (int i = 0; i < ROWS; ++i)
#pragma unroll
                for (int b = 0; b < BLOCKS; ++b) acc[i][b] = f32x4{0, 0, 0, 0};
            const In *cr[BLOCKS];  // past the last rank the last stands in, and is not stored
#pragma unroll
            for (int b = 0; b < BLOCKS; ++b) {
                const int rank = min(rank0 + 16 * b + l16, a.c.rank - 1);
                cr[b] = c + (RANK_INNER ? 16 * quarter * a.c.ld + rank : rank * a.c.ld + 16 * quarter);
            }
            auto step = [&](int64_t k, In (&vx)[ROWS][8], In (&vc)[BLOCKS][8], int64_t there) {
#pragma unroll
                for (int i = 0; i < ROWS; ++i) load_some<In, 8>(x[i] + k, there, vx[i]);
#pragma unroll
                for (int b = 0; b < BLOCKS; ++b) {
                    if constexpr (RANK_INNER) {
#pragma unroll
                        for (int e = 0; e < 8; ++e) vc[b][e] = e < there ? cr[b][(k + e) * a.c.ld] : (In)0.0f;
                    } else {
                        load_some<In, 8>(cr[b] + k, there, vc[b]);
                    }
                }
            };
            auto multiply = [&](const In (&vx)[ROWS][8], const In (&vc)[BLOCKS][8]) {
#pragma unroll
                for (int i = 0; i < ROWS; ++i)
#pragma unroll
                    for (int b = 0; b < BLOCKS; ++b) acc[i][b] = Step<In>::add(vc[b], vx[i], acc[i][b]);
            };
            // two sets of steps: the loads of one are under way while the other is multiplied
            constexpr int kHeld = (ROWS + (RANK_INNER ? 4 : 1) * BLOCKS) * (sizeof(In) == 4 ? 2 : 1);
            constexpr int U = kHeld <= 3 ? 2 : 1;
            In vx[2][2 * U][ROWS][8], vc[2][2 * U][BLOCKS][8];
            auto load = [&](int set, int64_t k) {
#pragma unroll
                for (int u = 0; u < 2 * U; ++u) step(k + kStep * (u / 2) + 8 * (u % 2), vx[set][u], vc[set][u], 8);
            };
            auto use = [&](int set) {
#pragma unroll
                for (int u = 0; u < 2 * U; ++u) multiply(vx[set][u], vc[set][u]);
            };
            int64_t k = first;
            auto whole = [&](int64_t k) { return k + kStep * (U - 1) + 64 <= last; };
            if (whole(k)) {
                load(0, k);
                for (k += kStep * U; whole(k + kStep * U); k += 2 * kStep * U) {
                    load(1, k);
                    use(0);
                    load(0, k + kStep * U);
                    use(1);
                }
                if (whole(k)) {
                    load(1, k);
                    use(0);
                    use(1);
                    k += kStep * U;
                } else {
                    use(0);
                }
            }
            for (; k < last; k += kStep) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    step(k + 8 * h, vx[0][h], vc[0][h], last - (k + 16 * quarter + 8 * h));
                    multiply(vx[0][h], vc[0][h]);
                }
            }
            if constexpr (SHARED) {
                if (wave > 0) {
#pragma unroll
                    for (int b = 0; b < BLOCKS; ++b) sums[wave - 1][b][lane] = acc[0][b];
                }
                __syncthreads();
                if (wave == 0) {
#pragma unroll
                    for (int b = 0; b < BLOCKS; ++b) acc[0][b] += sums[0][b][lane] + sums[1][b][lane] + sums[2][b][lane];
                }
                __syncthreads();
                if (wave > 0) continue;
            }
            const float factor = a.scales != nullptr ? a.scales[now] : 1.0f;
#pragma unroll
            for (int i = 0; i < ROWS; ++i) {
                if (id[i] != now) continue;
                const int64_t row = row0 + 16 * i + l16;
#pragma unroll
                for (int b = 0; b < BLOCKS; ++b) {
                    const int rank = rank0 + 16 * b + 4 * quarter;
                    if (a.part != nullptr) {
                        float *to = a.part + ((int64_t)blockIdx.z * a.T + row) * a.c.rank + rank;
#pragma unroll
                        for (int r = 0; r < 4; ++r)
                            if (rank + r < a.c.rank) to[r] = acc[i][b][r];
                    }
                    if (a.planes != nullptr) put_planes<sizeof(In) == 4>(a.planes, row, rank, a.c.rank, acc[i][b], factor);
                }
            }
        }
    }
}

// The same for many rows of 16-bit values, 16-byte aligned and of whole steps of
// 64, with adapters that lie along the sum: a work-group takes 64 rows and goes
// through LDS, 128 values of k at a time in one of two stages, which makes the
// rows' loads 256 adjacent bytes, and an adapter is read once for 64 rows.  Bound by
// reading the rows once.  (8192 rows of 16384 with 32 ranks straight from device
// memory, where 16 rows that lie a power of two apart meet in few of the memory's channels,
// 115 µs.)
template <class In, int BLOCKS>
__global__ __launch_bounds__(256) void shrink_rows_kernel(ShrinkArgs a)
{
    typedef m16::Slice<64, 1, 256, false, false> SliceX;
    typedef m16::Slice<16 * BLOCKS, BLOCKS, 128 * BLOCKS, false, false> SliceC;  // one round a half
    constexpr int kHalf = SliceX::kBytes, kHalfC = SliceC::kBytes, kStage = 2 * kHalf + 2 * kHalfC;
    static_assert(SliceX::kRounds == 2 && SliceC::kRounds == 1, "rounds");
    __shared__ __align__(1024) char lds[2 * kStage];
    const int thread = threadIdx.x, lane = thread & 63, wave = __builtin_amdgcn_readfirstlane(thread >> 6);
    const int l16 = lane & 15, quarter = lane >> 4;
    const int64_t row0 = (int64_t)blockIdx.x * 64;
    // every wavefront goes through the adapters of all 64 rows
    int all = -1;
    if (row0 + lane < a.T) {
        const int64_t n = a.ids[row0 + lane];
        if (n >= 0 && n < a.c.count) all = (int)n;
    }
    const int id = __shfl(all, wave * 16 + l16);
    const int64_t row = row0 + wave * 16 + l16, from = blockIdx.z * a.part_k, last = min(from + a.part_k, a.K);
    const int last_row = (int)min((int64_t)63, a.T - 1 - row0);
    const char *x = (const char *)((const In *)a.rows + row0 * a.ld);
    m16::Reader<64, 1, false, false> rx;
    m16::Reader<16 * BLOCKS, BLOCKS, false, false> rc;
    rx.place(wave * 16, lane);
    rc.place(0, lane);
    uint64_t left = __ballot(all >= 0);
    while (left != 0) {
        const int now = __builtin_amdgcn_readlane(all, __builtin_ctzll(left));
        left &= ~__ballot(all == now);
        const bool here = __ballot(id == now) != 0;
        for (int rank0 = 0; rank0 < (a.planes != nullptr ? (int)planes_rank(a.c.rank) : a.c.rank); rank0 += 16 * BLOCKS) {
            const int first_rank = min(rank0, a.c.rank - 1), last_rank = a.c.rank - 1 - first_rank;
            const char *c = (const char *)((const In *)a.c.p + now * a.c.stride + first_rank * a.c.ld);
            auto issue = [&](int stage, int64_t k) {
                m16::lds_char *to = (m16::lds_char *)lds + stage * kStage;
                const int64_t half[2] = {k, min(k + 64, last - 64)};  // past the end the last stands in, for nobody
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int r = 0; r < 2; ++r)
                        m16::load_lds(x + half[h] * 2, SliceX::offset(r * 256 + thread, a.ld, last_row, 64), to + h * kHalf + (r * 256 + wave * 64) * 16);
#pragma unroll
                for (int r = 0; r < BLOCKS; ++r) {
                    const int position = r * 256 + thread, h = position / (128 * BLOCKS);
                    m16::load_lds(c, SliceC::offset(position % (128 * BLOCKS), a.c.ld, last_rank, 64) + (uint32_t)half[h] * 2,
                                  to + 2 * kHalf + (r * 256 + wave * 64) * 16);
                }
            };
            f32x4 acc[BLOCKS];
#pragma unroll
            for (int b = 0; b < BLOCKS; ++b) acc[b] = f32x4{0, 0, 0, 0};
            issue(0, from);
            if (from + 128 < last) issue(1, from + 128);
            int stage = 0;
            for (int64_t k = from; k < last; k += 128) {
                if (k + 128 < last) m16::arrive<4 + BLOCKS>();
                else m16::arrive<0>();
                m16::lds_char *at = (m16::lds_char *)lds + stage * kStage;
                if (here) {
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        if (h == 1 && k + 64 >= last) continue;
#pragma unroll
                        for (int s = 0; s < 2; ++s) {
                            const typename Frag<In>::type fx = rx.template read<In>(at + h * kHalf, 0, s);
#pragma unroll
                            for (int b = 0; b < BLOCKS; ++b)
                                acc[b] = Frag<In>::mfma(rc.template read<In>(at + 2 * kHalf + h * kHalfC, b, s), fx, acc[b]);
                        }
                    }
                }
                __syncthreads();
                if (k + 256 < last) issue(stage, k + 256);
                stage ^= 1;
            }
            if (id != now) continue;
            const float factor = a.scales != nullptr ? a.scales[now] : 1.0f;
#pragma unroll
            for (int b = 0; b < BLOCKS; ++b) {
                const int rank = rank0 + 16 * b + 4 * quarter;
                if (a.part != nullptr) {
                    float *to = a.part + ((int64_t)blockIdx.z * a.T + row) * a.c.rank + rank;
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        if (rank + r < a.c.rank) to[r] = acc[b][r];
                }
                if (a.planes != nullptr) put_planes<false>(a.planes, row, rank, a.c.rank, acc[b], factor);
            }
        }
    }
}

template <bool WHOLE>
__global__ __launch_bounds__(256) void finish_kernel(ShrinkArgs a, float *hidden, void *planes)
{
    const int per_row = (int)planes_rank(a.c.rank) / 4;
    const int64_t n = (int64_t)blockIdx.x * 256 + threadIdx.x, row = n / per_row;
    if (row >= a.T) return;
    const int at = (int)(n % per_row) * 4;
    const int64_t id = a.ids[row];
    if (id < 0 || id >= a.c.count) return;
    f32x4 v{0, 0, 0, 0};
    for (int p = 0; p < a.parts; ++p) {
        const float *from = a.part + (p * a.T + row) * a.c.rank + at;
#pragma unroll
        for (int r = 0; r < 4; ++r)
            if (at + r < a.c.rank) v[r] += from[r];
    }
    if (hidden != nullptr) {
#pragma unroll
        for (int r = 0; r < 4; ++r)
            if (at + r < a.c.rank) hidden[row * a.c.rank + at + r] = v[r];
    }
    if (planes != nullptr) put_planes<WHOLE>(planes, row, at, a.c.rank, v, a.scales != nullptr ? a.scales[id] : 1.0f);
}

template <class In, int BLOCKS>
void shrink(const ShrinkArgs &a, hipStream_t stream)
{
    const dim3 grid((unsigned)((a.T + a.rows_each - 1) / a.rows_each), a.slots, a.parts);
    if constexpr (sizeof(In) == 2) {
        if (a.through_lds) {
            shrink_rows_kernel<In, BLOCKS><<<grid, 256, 0, stream>>>(a);
            return;
        }
    }
    if (a.rows_each == 16) {
        if (a.c.rank_inner) shrink_kernel<In, BLOCKS, 1, true, true><<<grid, 256, 0, stream>>>(a);
        else shrink_kernel<In, BLOCKS, 1, false, true><<<grid, 256, 0, stream>>>(a);
    } else if (a.rows_each == 64) {
        if (a.c.rank_inner) shrink_kernel<In, BLOCKS, 1, true, false><<<grid, 256, 0, stream>>>(a);
        else shrink_kernel<In, BLOCKS, 1, false, false><<<grid, 256, 0, stream>>>(a);
    } else {
        if (a.c.rank_inner) shrink_kernel<In, BLOCKS, 2, true, false><<<grid, 256, 0, stream>>>(a);
        else shrink_kernel<In, BLOCKS, 2, false, false><<<grid, 256, 0, stream>>>(a);
    }
}
template <class In>
void shrink(const ShrinkArgs &a, hipStream_t stream)
{
    if (a.c.rank <= 16) shrink<In, 1>(a, stream);
    else if (a.c.rank <= 32) shrink<In, 2>(a, stream);
    else shrink<In, 4>(a, stream);
}

// ---- grouping --------------------------------------------------------------

// The sums over the work-group's threads before this one, and over all.
__device__ __forceinline__ int before(int v, int *room, int &all)
{
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, waves = blockDim.x >> 6;
    int sum = v;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int other = __shfl_up(sum, d);
        if (lane >= d) sum += other;
    }
    if (lane == 63) room[wave] = sum;
    __syncthreads();
    int of = lane < waves ? room[lane] : 0;  // the wavefronts' sums, in every wavefront
    __syncthreads();
#pragma unroll
    for (int d = 1; d < 16; d <<= 1) {
        const int other = __shfl_up(of, d);
        if (lane >= d) of += other;
    }
    all = __shfl(of, waves - 1);
    const int base = __shfl(of, wave > 0 ? wave - 1 : 0);
    return (wave > 0 ? base : 0) + sum - v;
}

// Work-group i counts the tokens of smaller adapters and lists its own in
// their order: the ids are read twice by each adapter's, and nothing is
// counted with atomics.  Bound by the chain of rounds over the ids.
__global__ __launch_bounds__(1024) void group_kernel(GroupArgs a)
{
    __shared__ int room[16];
    const int mine = blockIdx.x;
    int smaller = 0, own = 0;
    for (int t = threadIdx.x; t < a.T; t += 1024) {
        const int64_t id = a.ids[t];
        smaller += id >= 0 && id < mine;
        own += id == mine;
    }
    int start, total;
    before(smaller, room, start);
    before(own, room, total);
    if (threadIdx.x == 0) {
        a.starts[mine] = start;
        if (mine == a.count - 1) a.starts[a.count] = start + total;
    }
    constexpr int kEach = 8;
    for (int t0 = 0; t0 < a.T && total > 0; t0 += 1024 * kEach) {
        const int t = t0 + threadIdx.x * kEach;
        uint32_t is = 0;
#pragma unroll
        for (int e = 0; e < kEach; ++e)
            if (t + e < a.T && a.ids[t + e] == mine) is |= 1u << e;
        int found;
        int at = start + before(__popc(is), room, found);
#pragma unroll
        for (int e = 0; e < kEach; ++e)
            if (is >> e & 1) a.order[at++] = t + e;
        start += found;
    }
}

__device__ __forceinline__ void cut_chunks(const GroupArgs &a, const Cut &cut, int *room)
{
    int chunk0 = 0, slot0 = 0;
    int64_t place0 = 0;
    for (int i0 = 0; i0 < a.count; i0 += blockDim.x) {
        const int i = i0 + threadIdx.x;
        const int from = i < a.count ? a.starts[i] : 0, tokens = i < a.count ? a.starts[i + 1] - from : 0;
        const int chunks = (tokens + cut.tokens - 1) / cut.tokens, slots = chunks > 1 ? chunks : 0;
        int all_chunks, all_slots;
        const int chunk = chunk0 + before(chunks, room, all_chunks), slot = slot0 + before(slots, room, all_slots);
        // in whole 64s; 1024 adapters have 2^24 tokens at most, and 64 more each
        int all_places;
        const int64_t place = place0 + 64 * (int64_t)before((tokens + 63) / 64, room, all_places);
        if (i < a.count) {
            cut.joins[i] = make_int2(slot, chunks);
            // an adapter's tokens are dealt evenly, in whole 64s
            const int each = chunks ? ((tokens + chunks - 1) / chunks + 63) / 64 * 64 : 0;
            for (int n = 0; n < chunks; ++n)
                cut.chunks[chunk + n] = Chunk{i, from + n * each, min(each, tokens - n * each), slots ? slot + n : -1, place + (int64_t)n * each};
        }
        chunk0 += all_chunks;
        slot0 += all_slots;
        place0 += 64 * (int64_t)all_places;
    }
    if (threadIdx.x == 0) *cut.chunk_count = chunk0;
}

__global__ __launch_bounds__(1024) void chunks_kernel(GroupArgs a)
{
    __shared__ int room[16];
    cut_chunks(a, a.cuts[blockIdx.x], room);
}

// All of it by one work-group of THREADS for a few tokens and adapters: a launch
// less, and the adapters' turn goes with it.  A thread takes adjacent tokens,
// whose ids it keeps in registers, and counts them adapter by adapter; one
// round through LDS gives it its places in each adapter's list.
template <int THREADS>
struct AloneRoom {
    int place[kAloneAdapters][THREADS];
    int waves[kAloneAdapters][THREADS / 64];
    int scan[16];
};
template <int THREADS>
__device__ __forceinline__ void group_alone(const GroupArgs &a, AloneRoom<THREADS> &room)
{
    constexpr int kMost = kAloneTokens / THREADS, kWaves = THREADS / 64;
    const int thread = threadIdx.x, lane = thread & 63, wave = thread >> 6;
    const int each = (a.T + THREADS - 1) / THREADS, first = thread * each;
    int id[kMost];
#pragma unroll
    for (int e = 0; e < kMost; ++e) {
        const int64_t n = e < each && first + e < a.T ? a.ids[first + e] : -1;
        id[e] = n >= 0 && n < a.count ? (int)n : -1;
    }
    for (int i = 0; i < a.count; ++i) {
        int own = 0;
#pragma unroll
        for (int e = 0; e < kMost; ++e) own += id[e] == i;
        int sum = own;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const int other = __shfl_up(sum, d);
            if (lane >= d) sum += other;
        }
        if (lane == 63) room.waves[i][wave] = sum;
        room.place[i][thread] = sum - own;  // within the wavefront
    }
    __syncthreads();
    int start = 0;
    for (int i = 0; i < a.count; ++i) {
        int base = start;
#pragma unroll
        for (int w = 0; w < kWaves; ++w) {
            const int n = room.waves[i][w];
            if (w < wave) base += n;
            start += n;
        }
        if (thread == 0) a.starts[i + 1] = start;
        room.place[i][thread] += base;
    }
    if (thread == 0) a.starts[0] = 0;
#pragma unroll
    for (int e = 0; e < kMost; ++e)
        if (id[e] >= 0) a.order[room.place[id[e]][thread]++] = first + e;
    __threadfence_block();
    __syncthreads();
    for (int n = 0; n < 2; ++n) cut_chunks(a, a.cuts[n], room.scan);
}

// ---- gradients -------------------------------------------------------------

// The sum over 32 tokens (8 a lane) of z·v: bf16 values are taken as they are
// and fp16 ones, which bf16's range holds, as two bf16 planes; v in two planes;
// float32 in float32.
template <class In>
struct Outer;
template <>
struct Outer<float> {
    typedef float Z;
    struct F {
        float v[8];
    };
    typedef F Zf;
    typedef F Vf;
    static __device__ __forceinline__ Zf z_of(const float (&v)[8]) { Zf f; 
#pragma unroll
        for (int e = 0; e < 8; ++e) f.v[e] = v[e];
        return f; }
    static __device__ __forceinline__ Vf v_of(const float (&v)[8]) { return z_of(v); }
    template <bool Z_FIRST>
    static __device__ __forceinline__ f32x4 add(const Zf &z, const Vf &v, f32x4 acc)
    {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            if (Z_FIRST) acc = __builtin_amdgcn_mfma_f32_16x16x4f32(z.v[e], v.v[e], acc, 0, 0, 0);
            else acc = __builtin_amdgcn_mfma_f32_16x16x4f32(v.v[e], z.v[e], acc, 0, 0, 0);
        }
        return acc;
    }
};
struct OuterPlanes {
    struct Vf {
        bf16x8 high, low;
    };
    static __device__ __forceinline__ Vf v_of(const float (&v)[8])
    {
        Vf f;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            __bf16 h, l;
            halves(v[e], h, l);
            f.high[e] = h;
            f.low[e] = l;
        }
        return f;
    }
    template <bool Z_FIRST>
    static __device__ __forceinline__ f32x4 one(const bf16x8 &z, const bf16x8 &v, f32x4 acc)
    {
        return Z_FIRST ? Frag<__bf16>::mfma(z, v, acc) : Frag<__bf16>::mfma(v, z, acc);
    }
};
template <>
struct Outer<__bf16> : OuterPlanes {
    typedef bf16x8 Zf;
    static __device__ __forceinline__ Zf z_of(const __bf16 (&v)[8])
    {
        Zf f;
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = v[e];
        return f;
    }
    static __device__ __forceinline__ Zf z_of(const bf16x8 &v) { return v; }
    template <bool Z_FIRST>
    static __device__ __forceinline__ f32x4 add(const Zf &z, const Vf &v, f32x4 acc)
    {
        return one<Z_FIRST>(z, v.high, one<Z_FIRST>(z, v.low, acc));
    }
};
template <>
struct Outer<_Float16> : OuterPlanes {
    typedef Vf Zf;
    static __device__ __forceinline__ Zf z_of(const _Float16 (&v)[8])
    {
        float f[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = (float)v[e];
        return v_of(f);
    }
    static __device__ __forceinline__ Zf z_of(const m16::f16x8 &v)
    {
        float f[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = (float)v[e];
        return v_of(f);
    }
    template <bool Z_FIRST>
    static __device__ __forceinline__ f32x4 add(const Zf &z, const Vf &v, f32x4 acc)
    {
        return one<Z_FIRST>(z.high, v.high, one<Z_FIRST>(z.high, v.low, one<Z_FIRST>(z.low, v.high, acc)));
    }
};

// RANK_INNER: a lane holds column l16, ranks 4·quarter + r; otherwise rank l16,
// columns 4·quarter + r.
template <class In, int BLOCKS, bool RANK_INNER>
__device__ __forceinline__ void put_outer(const OuterArgs &a, const Chunk &chunk, int col0, int rank0, const f32x4 (&acc)[2][BLOCKS])
{
    const int lane = threadIdx.x & 63, l16 = lane & 15, quarter = lane >> 4;
    const bool joined = chunk.slot >= 0;
    const float scale = a.scales != nullptr ? a.scales[chunk.adapter] : 1.0f;
    const int64_t ld = joined ? (RANK_INNER ? a.rank : a.C) : a.ldo;
    const int64_t base = joined ? (int64_t)chunk.slot * a.C * a.rank : chunk.adapter * a.stride_out;
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int b = 0; b < BLOCKS; ++b)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int col = col0 + 16 * j + (RANK_INNER ? l16 : 4 * quarter + r);
                const int rank = rank0 + 16 * b + (RANK_INNER ? 4 * quarter + r : l16);
                if (col >= a.C || rank >= a.rank) continue;
                const int64_t at = base + (RANK_INNER ? col * ld + rank : rank * ld + col);
                if (joined) a.part[at] = acc[j][b][r];
                else ((In *)a.out)[at] = (In)(acc[j][b][r] * scale);
            }
}

// Small values of the chunks' tokens, rank by rank, in two bf16 planes: as the
// matrix cores read a first operand along its sum.  (8192 tokens of 32 ranks for
// both gradients 9.6 µs.)
constexpr int kArranged = 64;  // tokens a work-group
__global__ __launch_bounds__(256) void arrange_kernel(OuterArgs first, OuterArgs second)
{
    const OuterArgs &a = blockIdx.z == 0 ? first : second;
    if (a.out == nullptr || a.arranged == nullptr || (int)blockIdx.x >= *a.cut.chunk_count) return;
    const Chunk chunk = a.cut.chunks[blockIdx.x];
    const int whole = (chunk.tokens + 63) / 64 * 64, t0 = blockIdx.y * kArranged;
    __bf16 *to = (__bf16 *)a.arranged + chunk.place * a.rank;
    // a thread takes two tokens of a rank, a wavefront 16 adjacent ranks of eight tokens' rows
    const int pairs = min(whole - t0, kArranged) / 2, blocks = (a.rank + 15) / 16;
    for (int n = threadIdx.x; n < pairs * 16 * blocks; n += 256) {
        const int block = n / (pairs * 16), in = n - block * (pairs * 16), rank = 16 * block + in % 16, t = t0 + in / 16 * 2;
        if (rank >= a.rank) continue;
        uint32_t high = 0, low = 0;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            if (t + e >= chunk.tokens) continue;
            __bf16 h, l;
            halves(a.small[(int64_t)a.order[chunk.first + t + e] * a.rank + rank], h, l);
            high |= (uint32_t)__builtin_bit_cast(uint16_t, h) << (16 * e);
            low |= (uint32_t)__builtin_bit_cast(uint16_t, l) << (16 * e);
        }
        *(uint32_t *)(to + (int64_t)rank * whole + t) = high;
        *(uint32_t *)(to + a.arranged_plane + (int64_t)rank * whole + t) = low;
    }
}

// 16 bytes a lane from an address of its own to 16 adjacent bytes a lane from
// `to` (as load_lds, which reaches 4 GiB from one base).
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
__device__ __forceinline__ void gather_lds(const void *from, m16::lds_char *to)
{
    const uint32_t at = (uint32_t)(uintptr_t)to;
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off"
                 :
                 : "s"(__builtin_amdgcn_readfirstlane(at)), "v"((uint64_t)(uintptr_t)from)
                 : "memory", "m0");
}
#pragma clang diagnostic pop

template <int BLOCKS>
constexpr int kOuterLds = 2 * (kOuterColumns * 128 + 2 * 16 * BLOCKS * 128);

// A work-group takes 128 columns of the rows, 16·BLOCKS ranks and a chunk of an
// adapter's tokens, 64 at a time: the rows' and the arranged values' slices go
// straight into one of two LDS stages, and the loads of the next 64 are under
// way while these are multiplied.  The rows' fragments come from the transposing
// LDS read.  A wavefront takes 32 columns.  Bound by reading the rows once:
// 8192 tokens of 4096 and 16384 columns (both gradients) with 32 ranks 62 µs,
// 5.4 TB/s.
template <class In, int BLOCKS, bool RANK_INNER>
__device__ __forceinline__ void outer_of(const OuterArgs &a, int rank0, char *lds, int *order)
{
    constexpr int kCols = kOuterColumns, kTokens = kOuterTokens, kRanks = 16 * BLOCKS;
    typedef m16::Slice<kCols, 2, 256, true, false> SliceZ;
    typedef m16::Slice<kRanks, BLOCKS, 128 * BLOCKS, false, false> SliceV;  // one round a plane
    constexpr int kBytesV = SliceV::kBytes, kStage = SliceZ::kBytes + 2 * kBytesV;
    static_assert(SliceZ::kRounds == 4 && SliceV::kRounds == 1, "rounds");
    static_assert(2 * kStage == kOuterLds<BLOCKS>, "room");
    const Chunk chunk = a.cut.chunks[blockIdx.y];
    const int thread = threadIdx.x, lane = thread & 63, wave = __builtin_amdgcn_readfirstlane(thread >> 6);
    const int col0 = blockIdx.x * kCols;
    const int whole = (chunk.tokens + 63) / 64 * 64;
    // tokens past the last meet zeros: the last stands in
    for (int t = thread; t < whole; t += 256) order[t] = a.order[chunk.first + min(t, chunk.tokens - 1)];
    const In *rows = (const In *)a.rows + col0;
    const int last_col = a.C - 8 - col0;
    const __bf16 *small = (const __bf16 *)a.arranged + chunk.place * a.rank + (int64_t)min(rank0, a.rank - 1) * whole;
    const int last_rank = a.rank - 1 - min(rank0, a.rank - 1);
    // the pieces of both planes of V: 2·128·BLOCKS, 256 at a time
    auto issue = [&](int stage, int t0) {
        m16::lds_char *to = (m16::lds_char *)lds + stage * kStage;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int position = r * 256 + thread, row = position / SliceZ::kRowPieces, slot = position % SliceZ::kRowPieces;
            const int col = min((slot ^ m16::flip<kCols, 2, false>(row)) * 8, last_col);
            gather_lds(rows + order[t0 + row] * a.ld + col, to + (r * 256 + wave * 64) * 16);
        }
#pragma unroll
        for (int r = 0; r < BLOCKS; ++r) {
            const int position = r * 256 + thread, plane = position / (128 * BLOCKS), in = position % (128 * BLOCKS);
            gather_lds((const char *)(small + plane * a.arranged_plane + t0) + SliceV::offset(in, whole, last_rank, kTokens),
                       to + SliceZ::kBytes + (r * 256 + wave * 64) * 16);
        }
    };
    m16::Reader<kCols, 2, true, false> rz;
    m16::Reader<kRanks, BLOCKS, false, false> rv;
    rz.place(wave * 32, lane);
    rv.place(0, lane);
    f32x4 acc[2][BLOCKS];
#pragma unroll
    for (int b = 0; b < BLOCKS; ++b) acc[0][b] = acc[1][b] = f32x4{0, 0, 0, 0};
    __syncthreads();  // the order
    issue(0, 0);
    if (kTokens < whole) issue(1, kTokens);
    int stage = 0;
    for (int t0 = 0; t0 < whole; t0 += kTokens) {
        if (t0 + kTokens < whole) m16::arrive<4 + BLOCKS>();
        else m16::arrive<0>();
        m16::lds_char *z = (m16::lds_char *)lds + stage * kStage, *v = z + SliceZ::kBytes;
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            typename Outer<In>::Zf zf[2];
#pragma unroll
            for (int j = 0; j < 2; ++j) zf[j] = Outer<In>::z_of(rz.template read<In>(z, j, s));
#pragma unroll
            for (int b = 0; b < BLOCKS; ++b) {
                OuterPlanes::Vf vf;
                vf.high = rv.template read<__bf16>(v, b, s);
                vf.low = rv.template read<__bf16>(v + kBytesV, b, s);
#pragma unroll
                for (int j = 0; j < 2; ++j) acc[j][b] = Outer<In>::template add<!RANK_INNER>(zf[j], vf, acc[j][b]);
            }
        }
        __syncthreads();
        if (t0 + 2 * kTokens < whole) issue(stage, t0 + 2 * kTokens);
        stage ^= 1;
    }
    put_outer<In, BLOCKS, RANK_INNER>(a, chunk, col0 + 32 * wave, rank0, acc);
}

// Both gradients' in one launch: the first's ranks, then the second's, along z.
template <class In, int BLOCKS>
__global__ __launch_bounds__(256) void outer_kernel(OuterArgs first, OuterArgs second)
{
    __shared__ __align__(1024) char lds[kOuterLds<BLOCKS>];
    __shared__ int order[kMostTokens];
    const int blocks = (first.rank + 16 * BLOCKS - 1) / (16 * BLOCKS);
    const bool other = (int)blockIdx.z >= blocks;
    const OuterArgs &a = other ? second : first;
    if (a.out == nullptr || a.arranged == nullptr || (int)blockIdx.x * kOuterColumns >= a.C || (int)blockIdx.y >= *a.cut.chunk_count) return;
    if (other) outer_of<In, BLOCKS, true>(a, ((int)blockIdx.z - blocks) * 16 * BLOCKS, lds, order);
    else outer_of<In, BLOCKS, false>(a, (int)blockIdx.z * 16 * BLOCKS, lds, order);
}

// The same for float32 rows and rows that start anywhere: through registers into
// LDS, and out of it value by value.
template <class In, int BLOCKS, bool RANK_INNER>
__global__ __launch_bounds__(256) void outer_any_kernel(OuterArgs a)
{
    constexpr int kCols = kOuterColumns, kTokens = kOuterTokens, kRanks = 16 * BLOCKS;
    constexpr int kPiece = 16 / sizeof(In), kPieces = kCols / kPiece * kTokens / 256;
    constexpr int kVals = kRanks * kTokens / 256;
    constexpr int kLdZ = kCols + 16 / sizeof(In), kLdV = kRanks + 1;
    __shared__ __align__(16) In zs[kTokens * kLdZ];
    __shared__ float vs[kTokens * kLdV];
    if ((int)blockIdx.y >= *a.cut.chunk_count) return;
    const Chunk chunk = a.cut.chunks[blockIdx.y];
    const int thread = threadIdx.x, lane = thread & 63, wave = thread >> 6, l16 = lane & 15, quarter = lane >> 4;
    const int col0 = blockIdx.x * kCols, rank0 = blockIdx.z * kRanks;
    const int *order = a.order + chunk.first;
    f32x4 acc[2][BLOCKS];
#pragma unroll
    for (int b = 0; b < BLOCKS; ++b) acc[0][b] = acc[1][b] = f32x4{0, 0, 0, 0};

    In z[kPieces][kPiece];
    float v[kVals];
    auto load = [&](int t0) {
#pragma unroll
        for (int n = 0; n < kPieces; ++n) {
            const int piece = n * 256 + thread, t = t0 + piece / (kCols / kPiece), col = col0 + piece % (kCols / kPiece) * kPiece;
            const bool there = t < chunk.tokens && col < a.C;
            load_some<In, kPiece>((const In *)a.rows + (there ? order[t] * a.ld + col : 0), there ? a.C - col : 0, z[n]);
        }
#pragma unroll
        for (int n = 0; n < kVals; ++n) {
            const int at = n * 256 + thread, t = t0 + at / kRanks, rank = rank0 + at % kRanks;
            v[n] = t < chunk.tokens && rank < a.rank ? a.small[(int64_t)order[t] * a.rank + rank] : 0.0f;
        }
    };
    load(0);
    for (int t0 = 0; t0 < chunk.tokens; t0 += kTokens) {
#pragma unroll
        for (int n = 0; n < kPieces; ++n) {
            const int piece = n * 256 + thread, t = piece / (kCols / kPiece), col = piece % (kCols / kPiece) * kPiece;
            typedef In piece_t __attribute__((ext_vector_type(kPiece)));
            piece_t p;
#pragma unroll
            for (int e = 0; e < kPiece; ++e) p[e] = z[n][e];
            *(piece_t *)(zs + t * kLdZ + col) = p;
        }
#pragma unroll
        for (int n = 0; n < kVals; ++n) {
            const int at = n * 256 + thread;
            vs[at / kRanks * kLdV + at % kRanks] = v[n];
        }
        __syncthreads();
        if (t0 + kTokens < chunk.tokens) load(t0 + kTokens);
#pragma unroll
        for (int s = 0; s < kTokens / 32; ++s) {
            typename Outer<In>::Zf zf[2];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                In e8[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) e8[e] = zs[(32 * s + 8 * quarter + e) * kLdZ + 32 * wave + 16 * j + l16];
                zf[j] = Outer<In>::z_of(e8);
            }
#pragma unroll
            for (int b = 0; b < BLOCKS; ++b) {
                float e8[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) e8[e] = vs[(32 * s + 8 * quarter + e) * kLdV + 16 * b + l16];
                const typename Outer<In>::Vf vf = Outer<In>::v_of(e8);
#pragma unroll
                for (int j = 0; j < 2; ++j) acc[j][b] = Outer<In>::template add<!RANK_INNER>(zf[j], vf, acc[j][b]);
            }
        }
        __syncthreads();
    }

    put_outer<In, BLOCKS, RANK_INNER>(a, chunk, col0 + 32 * wave, rank0, acc);
}

// Adapters without tokens get zeros, those of several chunks their sum, W
// adjacent values a thread (whole rows of W) and eight loads at a time.
template <class In, int W>
__device__ __forceinline__ void join_chunks(const OuterArgs &a, int adapter, int2 join, int64_t inner, int64_t size)
{
    typedef float floats __attribute__((ext_vector_type(W)));
    const float scale = a.scales != nullptr ? a.scales[adapter] : 1.0f;
    for (int64_t n = ((int64_t)blockIdx.x * 256 + threadIdx.x) * W; n < size; n += (int64_t)gridDim.x * 256 * W) {
        const float *from = a.part + join.x * size + n;
        floats sum = 0;
        for (int c = 0; c < join.y; c += 8) {
            floats v[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = c + e < join.y ? *(const floats *)(from + (c + e) * size) : (floats)0;
#pragma unroll
            for (int e = 0; e < 8; ++e) sum += v[e];
        }
        In *to = (In *)a.out + adapter * a.stride_out + n / inner * a.ldo + n % inner;
        typename m16::Some<In, W>::type results;
#pragma unroll
        for (int e = 0; e < W; ++e) results[e] = (In)(join.y ? sum[e] * scale : 0.0f);
        *(typename m16::Some<In, W>::type *)to = results;
    }
}

// Bound by the start of its work-groups and the loads' way there and back (8
// adapters' 32×4096 in two or three chunks, their 32×16384 in one: 9 µs).
template <class In>
__global__ __launch_bounds__(256) void join_kernel(OuterArgs first, OuterArgs second)
{
    const OuterArgs &a = blockIdx.z == 0 ? first : second;
    if (a.out == nullptr) return;
    const int2 join = a.cut.joins[blockIdx.y];
    if (join.y == 1) return;
    const int64_t inner = a.rank_inner ? a.rank : a.C, size = inner * (a.rank_inner ? a.C : a.rank);
    if (inner % 4 == 0) join_chunks<In, 4>(a, blockIdx.y, join, inner, size);
    else join_chunks<In, 1>(a, blockIdx.y, join, inner, size);
}

// The adapters the other way round, 64×64 elements at a time through LDS, four
// adjacent ones a load and store; the last work-group along x of the first
// adapter groups the tokens if `grouping`, which takes longest: 8 adapters of 32
// ranks and 4096 and 16384 columns with 8192 tokens 25 µs, 3 with 777 tokens and
// nothing to turn 10.5.
constexpr int kTurn = 256;
template <class In>
__global__ __launch_bounds__(kTurn) void turn_kernel(TurnArgs first, TurnArgs second, GroupArgs group, bool grouping)
{
    __shared__ In tile[64][65];
    __shared__ AloneRoom<kTurn> room;
    if (grouping && blockIdx.x + 1 == gridDim.x) {
        if (blockIdx.z == 0) group_alone<kTurn>(group, room);
        return;
    }
    const bool other = blockIdx.z >= (unsigned)first.from.count;
    const TurnArgs &a = other ? second : first;
    if (a.to == nullptr) return;
    const int64_t adapter = other ? blockIdx.z - first.from.count : blockIdx.z;
    const int64_t rows = a.from.rank_inner ? a.outer : a.from.rank, cols = a.from.rank_inner ? a.from.rank : a.outer;
    const int64_t across = (cols + 63) / 64, tiles = (rows + 63) / 64 * across;
    const In *from = (const In *)a.from.p + adapter * a.from.stride;
    In *to = (In *)a.to + adapter * a.to_stride;
    for (int64_t n = blockIdx.x; n < tiles; n += gridDim.x - (grouping ? 1 : 0)) {
        const int64_t r0 = n / across * 64, c0 = n % across * 64;
        In v[1024 / kTurn][4];
#pragma unroll
        for (int u = 0; u < 1024 / kTurn; ++u) {
            const int e = u * kTurn + threadIdx.x, r = e / 16, c = e % 16 * 4;
            const bool there = r0 + r < rows && c0 + c < cols;
            m16::load_some<In, 4>(from + (there ? (r0 + r) * a.from.ld + c0 + c : 0), there ? cols - c0 - c : 0, v[u]);
        }
#pragma unroll
        for (int u = 0; u < 1024 / kTurn; ++u) {
            const int e = u * kTurn + threadIdx.x, r = e / 16, c = e % 16 * 4;
#pragma unroll
            for (int x = 0; x < 4; ++x) tile[r][c + x] = v[u][x];
        }
        __syncthreads();
#pragma unroll
        for (int u = 0; u < 1024 / kTurn; ++u) {
            const int e = u * kTurn + threadIdx.x, r = e / 16, c = e % 16 * 4;
            if (c0 + r >= cols || r0 + c >= rows) continue;
            In *at = to + (c0 + r) * a.to_ld + r0 + c;
            typename m16::Some<In, 4>::type four;
#pragma unroll
            for (int x = 0; x < 4; ++x) four[x] = tile[c + x][r];
            // (rows of the copy are whole 8s; past the last of them lies nothing that is read)
            *(typename m16::Some<In, 4>::type *)at = four;
        }
        __syncthreads();
    }
}

template <class In, int BLOCKS>
void outer(const OuterArgs &a, const OuterArgs &b, hipStream_t stream)
{
    const int ranks = (a.rank + 16 * BLOCKS - 1) / (16 * BLOCKS);
    if constexpr (sizeof(In) == 2) {
        const bool first = a.out != nullptr && a.arranged != nullptr, second = b.out != nullptr && b.arranged != nullptr;
        const int C = !second || (first && a.C > b.C) ? a.C : b.C;
        const int chunks = !second || (first && a.most_chunks > b.most_chunks) ? a.most_chunks : b.most_chunks;
        if (first || second)
            outer_kernel<In, BLOCKS><<<dim3((C + kOuterColumns - 1) / kOuterColumns, chunks, 2 * ranks), 256, 0, stream>>>(a, b);
    }
    for (const OuterArgs *o : {&a, &b}) {
        if (o->out == nullptr || (sizeof(In) == 2 && o->arranged != nullptr)) continue;
        const dim3 grid((unsigned)((o->C + kOuterColumns - 1) / kOuterColumns), o->most_chunks, ranks);
        if (o->rank_inner) outer_any_kernel<In, BLOCKS, true><<<grid, 256, 0, stream>>>(*o);
        else outer_any_kernel<In, BLOCKS, false><<<grid, 256, 0, stream>>>(*o);
    }
}
template <class In>
void outer(const OuterArgs &a, const OuterArgs &b, hipStream_t stream)
{
    if (a.rank <= 16) outer<In, 1>(a, b, stream);
    else if (a.rank <= 32) outer<In, 2>(a, b, stream);
    else outer<In, 4>(a, b, stream);
}

}  // namespace

hipError_t launch_shrink(const ShrinkArgs &a, hipStream_t stream)
{
    if (a.dtype == TGEMM_F32) shrink<float>(a, stream);
    else if (a.dtype == TGEMM_BF16) shrink<__bf16>(a, stream);
    else shrink<_Float16>(a, stream);
    return hipGetLastError();
}

hipError_t launch_finish(const ShrinkArgs &a, float *hidden, void *planes, hipStream_t stream)
{
    const unsigned grid = (unsigned)((a.T * (planes_rank(a.c.rank) / 4) + 255) / 256);
    if (a.dtype == TGEMM_F32) finish_kernel<true><<<grid, 256, 0, stream>>>(a, hidden, planes);
    else finish_kernel<false><<<grid, 256, 0, stream>>>(a, hidden, planes);
    return hipGetLastError();
}

hipError_t launch_group(const GroupArgs &a, hipStream_t stream)
{
    group_kernel<<<a.count, 1024, 0, stream>>>(a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    chunks_kernel<<<2, 1024, 0, stream>>>(a);
    return hipGetLastError();
}

hipError_t launch_outer(const OuterArgs &a, const OuterArgs &b, hipStream_t stream)
{
    if (a.dtype == TGEMM_F32) outer<float>(a, b, stream);
    else if (a.dtype == TGEMM_BF16) outer<__bf16>(a, b, stream);
    else outer<_Float16>(a, b, stream);
    return hipGetLastError();
}

hipError_t launch_arrange(const OuterArgs &a, const OuterArgs &b, hipStream_t stream)
{
    const int most = a.most_chunks > b.most_chunks ? a.most_chunks : b.most_chunks;
    const int tokens = a.cut.tokens > b.cut.tokens ? a.cut.tokens : b.cut.tokens;
    arrange_kernel<<<dim3(most, (tokens + kArranged - 1) / kArranged, 2), 256, 0, stream>>>(a, b);
    return hipGetLastError();
}

hipError_t launch_join(const OuterArgs &a, const OuterArgs &b, hipStream_t stream)
{
    const int64_t C = a.C > b.C ? a.C : b.C, each = a.rank % 4 == 0 && a.C % 4 == 0 ? 1024 : 256, blocks = (C * a.rank + each - 1) / each;
    const dim3 grid((unsigned)(blocks < 256 ? blocks : 256), a.count, 2);
    if (a.dtype == TGEMM_F32) join_kernel<float><<<grid, 256, 0, stream>>>(a, b);
    else if (a.dtype == TGEMM_BF16) join_kernel<__bf16><<<grid, 256, 0, stream>>>(a, b);
    else join_kernel<_Float16><<<grid, 256, 0, stream>>>(a, b);
    return hipGetLastError();
}

hipError_t launch_turn(const TurnArgs &a, const TurnArgs &b, const GroupArgs *group, hipStream_t stream)
{
    const bool here = group != nullptr && group->T <= kAloneTokens && group->count <= kAloneAdapters;
    if (group != nullptr && !here) {
        const hipError_t e = launch_group(*group, stream);
        if (e != hipSuccess) return e;
    }
    const bool turning = a.to != nullptr || b.to != nullptr;
    if (!turning && !here) return hipSuccess;
    const int64_t outer = a.outer > b.outer ? a.outer : b.outer, tiles = turning ? (outer + 63) / 64 * ((a.from.rank + 63) / 64) : 0;
    const dim3 grid((unsigned)(tiles < 1024 ? tiles : 1024) + (here ? 1 : 0), 1, turning ? a.from.count + b.from.count : 1);
    const GroupArgs g = here ? *group : GroupArgs{};
    if (a.dtype == TGEMM_F32) turn_kernel<float><<<grid, kTurn, 0, stream>>>(a, b, g, here);
    else turn_kernel<uint16_t><<<grid, kTurn, 0, stream>>>(a, b, g, here);
    return hipGetLastError();
}

}  // namespace adapters
}  // namespace tgemm
