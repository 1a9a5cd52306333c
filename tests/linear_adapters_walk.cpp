// Follows every address of the projection with adapters on the host: the
// library's own entry points (linear_adapters.cpp) with launches that run the
// loads' walk (tile_walk.h) for each thread, or the extents that a pass over
// rows touches, instead of a kernel.  Reads calls from stdin, one a line:
//   need(0 forward, or bits) dtype T N D L r pad_x pad_w pad_y pad_a pad_b shift hidden
// and ends with 1 at the first access that leaves what the call was given.
#include <algorithm>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <vector>

#include "linear_adapters.h"

namespace {

struct Range {
    uintptr_t lo, hi;
    bool written;
    const char *name;
};
std::vector<Range> ranges;
long loads = 0;
char line[256];

void fail(const char *what, uintptr_t a, size_t n)
{
    std::printf("%s of %zu bytes at %#zx fails in: %s", what, n, (size_t)a, line);
    for (const Range &r : ranges) std::printf("  %s %#zx ... %#zx\n", r.name, (size_t)r.lo, (size_t)r.hi);
    std::exit(1);
}

void touch(const void *p, size_t n, bool write, const char *what)
{
    if (n == 0) return;
    const uintptr_t a = (uintptr_t)p;
    for (const Range &r : ranges)
        if (a >= r.lo && a + n <= r.hi && (!write || r.written)) return;
    fail(what, a, n);
}

void rows(const void *p, int64_t n, int64_t cols, int64_t ld, size_t size, bool write, const char *what)
{
    if (n == 0 || cols == 0) return;
    touch(p, cols * size, write, what);
    touch((const char *)p + (n - 1) * ld * (int64_t)size, cols * size, write, what);
}

size_t size_of(tgemm_dtype_t t) { return t == TGEMM_F32 ? 4 : 2; }

using tgemm::adapters::Stack;
using tgemm::m16::Operands;
using tgemm::m16::Slice;

void stack(const Stack &c, int64_t outer, size_t size, const char *what)
{
    const int64_t n = c.rank_inner ? outer : c.rank, cols = c.rank_inner ? c.rank : outer;
    for (int64_t i : {(int64_t)0, (int64_t)c.count - 1}) rows((const char *)c.p + i * c.stride * (int64_t)size, n, cols, c.ld, size, false, what);
}

template <class S>
void slice(const char *base, int64_t ld, int mn_last, int k_last, const char *what)
{
    if (mn_last < 0 || k_last < 0) fail("a clamp below the first row or column", 0, 0);
    for (int position = 0; position < S::kRounds * S::kThreads; ++position) {
        touch(base + S::offset(position, ld, mn_last, k_last), 16, false, what);
        ++loads;
    }
}

template <int BM, int BN, int WM, int WN, bool A_MC, bool B_MC>
void walk(const Operands &p, int wg_per_cu)
{
    typedef Slice<BM, BM / WM / 16, 64 * WM * WN, A_MC, false> A;
    typedef Slice<BN, BN / WN / 16, 64 * WM * WN, B_MC, true> B;
    const int tiles = p.ids(), grid = std::min(tiles, 256 * wg_per_cu);
    for (int group : {0, 1, 7, 8, grid / 2, grid - 9, grid - 2, grid - 1}) {
        if (group < 0 || group >= grid) continue;
        int steps = 2;
        for (int id = group; id < tiles; id += grid) {
            int m0, n0, split, first, last;
            p.tile<BM, BN>(id, m0, n0, split, first, last);
            if (first >= last) fail("a tile without steps", 0, 0);
            steps += (last - first) * p.segments;
        }
        tgemm::m16::Walk<BM, BN, A_MC, B_MC> w;
        w.begin(p, group);
        int a_last = 0, a_k = 0, b_last = 0, b_k = 0;
        for (int n = 0; n < steps; ++n) {
            const auto moved = w.seek(p, grid);
            if (moved.a) a_last = w.a_last, a_k = w.a_k_last;
            if (moved.b) b_last = w.b_last, b_k = w.b_k_last;
            if (n > 8 && n < steps - 8 && !moved.a && !moved.b && n % 61) continue;
            slice<A>(w.from_a, p.lda, a_last, a_k, "A");
            slice<B>(w.from_b, p.ldb, b_last, b_k, "B");
        }
    }
}

template <bool A_MC, bool B_MC>
void walk_tile(int tile, const Operands &p)
{
    switch (tile) {
#define X(I, BM, BN, WM, WN)                                                        \
    case I:                                                                         \
        if ((int64_t)p.tiles_m * BM < p.M || (int64_t)p.tiles_n * BN < p.N) fail("tiles", 0, 0); \
        walk<BM, BN, WM, WN, A_MC, B_MC>(p, tgemm::loss::kTiles[I].wg_per_cu);      \
        break;
        TGEMM_TILES(X)
#undef X
    default:
        fail("an unknown tile", 0, 0);
    }
}

void out(void *p, int64_t M, int64_t N, int64_t ld, tgemm_dtype_t t, int splits, int64_t stride)
{
    for (int s : {0, splits - 1}) rows((char *)p + s * stride * (int64_t)size_of(t), M, N, ld, size_of(t), true, "a product's result");
}

}  // namespace

namespace tgemm {
namespace loss {

hipError_t launch_copy(const CopyArgs &a, hipStream_t)
{
    rows(a.src, a.rows, a.cols, a.ld, size_of(a.dtype), false, "copy's source");
    for (int q = 0; q < a.planes; ++q) rows((char *)a.dst + q * a.plane * 2, a.rows_out, a.ld_out, a.ld_out, 2, true, "copy");
    if (a.rows_out < a.rows || a.ld_out < a.cols) fail("a copy that is too small", 0, 0);
    return hipSuccess;
}
hipError_t launch_dw(bool, int tile, const OutArgs &a, hipStream_t)
{
    walk_tile<true, true>(tile, a.op);
    out(a.out, a.op.M, a.op.N, a.ldo, a.dtype, a.op.splits, a.split_stride);
    return hipSuccess;
}
hipError_t launch_sum(const SumArgs &a, hipStream_t)
{
    for (int s : {0, a.count - 1}) rows(a.part + s * a.stride, a.T, a.D, a.ld, 4, false, "parts of a sum");
    rows(a.out, a.T, a.D, a.ldo, size_of(a.dtype), true, "a sum");
    return hipSuccess;
}
hipError_t launch_zero(void *p, int64_t ldo, tgemm_dtype_t dtype, int64_t n, int64_t cols, hipStream_t)
{
    rows(p, n, cols, ldo, size_of(dtype), true, "zeros");
    return hipSuccess;
}

}  // namespace loss

namespace adapters {

hipError_t launch_shrink(const ShrinkArgs &a, hipStream_t)
{
    if (a.parts < 1 || a.slots < 1 || a.part_k % 256 || a.parts * a.part_k < a.K || (a.parts - 1) * a.part_k >= a.K) fail("parts", 0, 0);
    if (a.parts > 1 && (!a.part || a.planes)) fail("parts without room", 0, 0);
    if (!a.part && !a.planes) fail("hidden values for nobody", 0, 0);
    rows(a.rows, a.T, a.K, a.ld, size_of(a.dtype), false, "shrink's rows");
    if (a.through_lds) {
        if (a.dtype == TGEMM_F32 || a.K % 64 || a.ld % 8 || a.c.ld % 8 || a.c.stride % 8 || (uintptr_t)a.rows % 16 || (uintptr_t)a.c.p % 16 ||
            a.c.rank_inner || a.rows_each != 64 || a.slots != 1 || a.ld > (1 << 22) || a.c.ld > (1 << 22))
            fail("rows through LDS", 0, 0);
        // the offsets of a part's steps, of the first and the last rows and ranks
        typedef Slice<64, 1, 256, false, false> X;
        typedef Slice<64, 4, 512, false, false> C;
        for (int64_t part : {(int64_t)0, (int64_t)a.parts - 1}) {
            const int64_t from = part * a.part_k, last = std::min(from + a.part_k, a.K);
            for (int64_t k : {from, std::min(from + 64, last - 64), last - 64}) {
                for (int64_t row0 : {(int64_t)0, (a.T - 1) / 64 * 64})
                    slice<X>((const char *)a.rows + (row0 * a.ld + k) * 2, a.ld, (int)std::min<int64_t>(63, a.T - 1 - row0), 64, "X");
                for (int64_t i : {(int64_t)0, (int64_t)a.c.count - 1})
                    slice<C>((const char *)a.c.p + (i * a.c.stride + k) * 2, a.c.ld, a.c.rank - 1, 64, "adapters");
            }
        }
    }
    stack(a.c, a.K, size_of(a.dtype), "shrink's adapters");
    rows(a.ids, a.T, 1, 1, 8, false, "ids");
    rows(a.scales, a.scales ? a.c.count : 0, 1, 1, 4, false, "scales");
    if (a.part) rows(a.part, a.parts * a.T, a.c.rank, a.c.rank, 4, true, "hidden parts");
    if (a.planes) rows(a.planes, a.T, planes_rank(a.c.rank), planes_rank(a.c.rank), 4, true, "hidden planes");
    return hipSuccess;
}
hipError_t launch_finish(const ShrinkArgs &a, float *hidden, void *planes, hipStream_t)
{
    rows(a.part, a.parts * a.T, a.c.rank, a.c.rank, 4, false, "hidden parts");
    if (hidden) rows(hidden, a.T, a.c.rank, a.c.rank, 4, true, "hidden");
    if (planes) rows(planes, a.T, planes_rank(a.c.rank), planes_rank(a.c.rank), 4, true, "hidden planes");
    return hipSuccess;
}
hipError_t launch_product(bool, bool b_mc, int tile, const ProductArgs &a, hipStream_t)
{
    if (b_mc) walk_tile<false, true>(tile, a.op);
    else walk_tile<false, false>(tile, a.op);
    out(a.out, a.op.M, a.op.N, a.ldo, a.dtype, a.op.splits, a.split_stride);
    if ((a.e.ids == nullptr) != (a.op.splits > 1)) fail("adapters of a split sum", 0, 0);
    if (a.e.ids == nullptr) return hipSuccess;
    rows(a.e.planes, a.op.M, planes_rank(a.e.c.rank), planes_rank(a.e.c.rank), 4, false, "hidden planes");
    stack(a.e.c, a.op.N, size_of(a.stored), "the product's adapters");
    if (!a.e.c.rank_inner && !b_mc) fail("adapters the other way", 0, 0);
    return hipSuccess;
}
hipError_t launch_add(const AddArgs &a, hipStream_t)
{
    for (int p : {0, a.count - 1}) rows(a.part + p * a.stride, a.T, a.N, a.ld, 4, false, "parts of a sum");
    rows(a.out, a.T, a.N, a.ldo, size_of(a.dtype), true, "a sum");
    rows(a.e.planes, a.T, planes_rank(a.e.c.rank), planes_rank(a.e.c.rank), 4, false, "hidden planes");
    stack(a.e.c, a.N, size_of(a.dtype), "the sum's adapters");
    return hipSuccess;
}
hipError_t launch_few(const FewArgs &a, hipStream_t)
{
    if (a.T > kFewRows) fail("too many rows", 0, 0);
    rows(a.X, a.T, a.D, a.ldx, size_of(a.dtype), false, "X");
    rows(a.W, a.N, a.D, a.ldw, size_of(a.dtype), false, "W");
    rows(a.Y, a.T, a.N, a.ldy, size_of(a.dtype), true, "Y");
    for (int p : {0, a.e.parts - 1}) rows(a.e.hidden + p * a.e.part_stride, a.T, a.e.c.rank, a.e.c.rank, 4, false, "hidden parts");
    stack(a.e.c, a.N, size_of(a.dtype), "the few rows' adapters");
    return hipSuccess;
}
hipError_t launch_group(const GroupArgs &a, hipStream_t)
{
    rows(a.ids, a.T, 1, 1, 8, false, "ids");
    rows(a.order, a.T, 1, 1, 4, true, "order");
    rows(a.starts, a.count + 1, 1, 1, 4, true, "starts");
    for (int n = 0; n < 2; ++n) {
        if (a.cuts[n].tokens % 64 || a.cuts[n].tokens < 64) fail("tokens of a chunk", 0, 0);
        // the most chunks that any ids can come to: all adapters one token more than whole chunks
        const int64_t t = a.cuts[n].tokens, adapters = std::min(a.count, a.T);
        rows(a.cuts[n].chunks, a.T / t + adapters, sizeof(Chunk), sizeof(Chunk), 1, true, "chunks");
        rows(a.cuts[n].joins, a.count, 1, 1, 8, true, "joins");
        rows(a.cuts[n].chunk_count, 1, 1, 1, 4, true, "chunk count");
    }
    return hipSuccess;
}
void check_outer(const OuterArgs &a)
{
    for (int64_t i : {(int64_t)0, (int64_t)a.count - 1})
        rows((char *)a.out + i * a.stride_out * (int64_t)size_of(a.dtype), a.rank_inner ? a.C : a.rank, a.rank_inner ? a.rank : a.C, a.ldo,
             size_of(a.dtype), true, "an adapter's gradient");
    if (a.most_chunks > 65535) fail("a grid", 0, a.most_chunks);
}
int64_t tokens;  // of the call
hipError_t launch_arrange(const OuterArgs &a, const OuterArgs &b, hipStream_t)
{
    for (const OuterArgs *o : {&a, &b}) {
        if (o->out == nullptr || o->arranged == nullptr) continue;
        rows(o->small, tokens, o->rank, o->rank, 4, false, "small");
        if (o->arranged_plane % 64) fail("planes that are not aligned", 0, 0);
        // whole 64s of every chunk
        if (o->arranged_plane < (tokens + 64 * ((int64_t)tokens / o->cut.tokens + std::min<int64_t>(o->count, tokens))) / 64 * 64 * o->rank)
            fail("arranged values' room", 0, 0);
        rows(o->arranged, 2, o->arranged_plane, o->arranged_plane, 2, true, "arranged");
    }
    return hipSuccess;
}
hipError_t launch_outer(const OuterArgs &first, const OuterArgs &second, hipStream_t)
{
    if (first.rank_inner || !second.rank_inner || first.rank != second.rank) fail("which is which", 0, 0);
    for (const OuterArgs *o : {&first, &second}) {
        const OuterArgs &a = *o;
        if (a.out == nullptr) continue;
        check_outer(a);
        rows(a.rows, tokens, a.C, a.ld, size_of(a.dtype), false, "rows");
        rows(a.small, tokens, a.rank, a.rank, 4, false, "small");
        if (a.cut.tokens > kMostTokens) fail("tokens of a chunk", 0, 0);
        if (a.arranged && (a.dtype == TGEMM_F32 || a.C % 8 || a.ld % 8 || (uintptr_t)a.rows % 16)) fail("rows that are not whole pieces", 0, 0);
        rows(a.part, 2 * (tokens / a.cut.tokens), (int64_t)a.C * a.rank, (int64_t)a.C * a.rank, 4, true, "sums of chunks");
    }
    return hipSuccess;
}
hipError_t launch_join(const OuterArgs &a, const OuterArgs &b, hipStream_t)
{
    for (const OuterArgs *o : {&a, &b})
        if (o->out) check_outer(*o);
    return hipSuccess;
}
hipError_t launch_turn(const TurnArgs &a, const TurnArgs &b, const GroupArgs *group, hipStream_t)
{
    if (group && launch_group(*group, nullptr) != hipSuccess) return hipErrorUnknown;
    if (a.from.count + b.from.count > 65535) fail("a grid", 0, 0);
    for (const TurnArgs *t : {&a, &b}) {
        if (t->to == nullptr) continue;
        stack(t->from, t->outer, size_of(t->dtype), "turn's adapters");
        const int64_t n = t->from.rank_inner ? t->from.rank : t->outer, cols = t->from.rank_inner ? t->outer : t->from.rank;
        for (int64_t i : {(int64_t)0, (int64_t)t->from.count - 1})
            rows((char *)t->to + i * t->to_stride * (int64_t)size_of(t->dtype), n, cols, t->to_ld, size_of(t->dtype), true, "turned");
    }
    return hipSuccess;
}

}  // namespace adapters
}  // namespace tgemm

extern "C" {
int tgemm_sgemm_splitk_choose(int64_t M, int64_t N, int64_t K) { return M * N < 512 * 512 && K > 512 ? 4 : 1; }
size_t tgemm_sgemm_splitk_workspace_size(int64_t M, int64_t N, int64_t, int splits) { return splits > 1 ? (size_t)M * N * splits * 4 : 0; }
tgemm_status_t tgemm_sgemm_splitk_ex(tgemm_op_t op_a, tgemm_op_t op_b, int64_t M, int64_t N, int64_t K, const float *A, int64_t lda,
                                     const float *B, int64_t ldb, float *C, int64_t ldc, int splits, void *room, size_t bytes, hipStream_t)
{
    rows(A, op_a ? K : M, op_a ? M : K, lda, 4, false, "A");
    rows(B, op_b ? N : K, op_b ? K : N, ldb, 4, false, "B");
    rows(C, M, N, ldc, 4, true, "C");
    if (bytes != tgemm_sgemm_splitk_workspace_size(M, N, K, splits)) fail("a workspace", 0, bytes);
    touch(room, bytes, true, "the product's workspace");
    return TGEMM_SUCCESS;
}
}

int main()
{
    long calls = 0;
    while (std::fgets(line, sizeof line, stdin)) {
        int need, dtype, hidden;
        long long T, N, D, L, r, px, pw, py, pa, pb, shift;
        if (std::sscanf(line, "%d %d %lld %lld %lld %lld %lld %lld %lld %lld %lld %lld %lld %d", &need, &dtype, &T, &N, &D, &L, &r, &px, &pw, &py,
                        &pa, &pb, &shift, &hidden) != 14)
            return 2;
        const tgemm_dtype_t t = (tgemm_dtype_t)dtype;
        const size_t s = size_of(t);
        uintptr_t next = 0x100000000000ull;
        ranges.clear();
        auto place = [&](size_t bytes, bool written, const char *name, bool shifted = false) {
            const uintptr_t at = next + (shifted ? shift * s : 0);
            ranges.push_back({at, at + bytes, written, name});
            next += 0x40000000000ull;
            return (void *)at;
        };
        tgemm::adapters::tokens = T;
        const long long ldx = D + px, ldw = D + pw, ldy = N + py, lda = D + pa, ldb = r + pb, sa = r * lda + pa, sb = N * ldb + pb;
        void *X = place((T ? (T - 1) * ldx + D : 0) * s, false, "X", true), *W = place(((N - 1) * ldw + D) * s, false, "W", true);
        void *A = place(((L - 1) * sa + (r - 1) * lda + D) * s, false, "A"), *B = place(((L - 1) * sb + (N - 1) * ldb + r) * s, false, "B", true);
        const int64_t *ids = (const int64_t *)place(T * 8, false, "ids");
        const float *scales = (const float *)place(L * 4, false, "scales");
        float *h = (float *)place(T * r * 4, need == 0, "hidden");
        void *Y = place((T ? (T - 1) * ldy + N : 0) * s, need == 0, "Y or dY", true);
        const size_t ws = tgemm_linear_adapters_workspace_size(t, T, N, D, X, ldx, W, ldw, L, r, need ? Y : nullptr, need ? ldy : 0, need);
        void *room = place(ws, true, "workspace");
        tgemm_status_t st;
        if (need == 0) {
            st = tgemm_linear_adapters_forward(t, T, N, D, X, ldx, W, ldw, L, r, A, lda, sa, B, ldb, sb, ids, scales, Y, ldy, hidden ? h : nullptr,
                                               room, ws, nullptr);
        } else {
            void *dX = need & 1 ? place((T ? (T - 1) * ldx + D : 0) * s, true, "dX") : nullptr;
            void *dW = need & 2 ? place(((N - 1) * ldw + D) * s, true, "dW") : nullptr;
            void *dA = need & 4 ? place(((L - 1) * sa + (r - 1) * lda + D) * s, true, "dA") : nullptr;
            void *dB = need & 8 ? place(((L - 1) * sb + (N - 1) * ldb + r) * s, true, "dB") : nullptr;
            st = tgemm_linear_adapters_backward(t, T, N, D, X, ldx, W, ldw, L, r, A, lda, sa, B, ldb, sb, ids, scales, hidden ? h : nullptr, Y, ldy,
                                                dX, ldx, dW, ldw, dA, lda, sa, dB, ldb, sb, room, ws, nullptr);
        }
        if (st != TGEMM_SUCCESS) fail("the call", 0, st);
        ++calls;
    }
    std::printf("%ld calls, %ld loads\n", calls, loads);
    return 0;
}
