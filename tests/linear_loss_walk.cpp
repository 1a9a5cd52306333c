// Follows every address of the loss operators on the host: the library's own
// entry points (linear_loss.cpp) with launches that run the loads' walk
// (tile_walk.h) for each thread, or the extents that a pass over rows touches,
// instead of a kernel.  Reads calls from stdin, one a line:
//   op(0 ce, 1 kd) pass dtype T V D ldx ldw shift_x shift_w K need_x need_w lddx lddw
// and ends with 1 at the first access that leaves what the call was given.
#include <algorithm>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <vector>

#include "linear_loss.h"

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
    std::printf("%s of %zu bytes at %#zx leaves the call's memory in: %s", what, n, (size_t)a, line);
    for (const Range &r : ranges) std::printf("  %s %#zx ... %#zx\n", r.name, (size_t)r.lo, (size_t)r.hi);
    std::exit(1);
}

void touch(const void *p, size_t n, bool write, const char *what)
{
    const uintptr_t a = (uintptr_t)p;
    for (const Range &r : ranges)
        if (a >= r.lo && a + n <= r.hi && (!write || r.written)) return;
    fail(what, a, n);
}

void rows(const void *p, int64_t n, int64_t cols, int64_t ld, size_t size, bool write, const char *what)
{
    if (n <= 0 || cols <= 0) return;
    touch(p, (size_t)cols * size, write, what);
    touch((const char *)p + (n - 1) * ld * (int64_t)size, (size_t)cols * size, write, what);
}

size_t size_of(tgemm_dtype_t t) { return t == TGEMM_F32 ? 4 : 2; }

using namespace tgemm::m16;

template <class S>
void slice(const char *base, int64_t ld, int mn_last, int k_last, const char *what)
{
    for (int position = 0; position < S::kRounds * S::kThreads; ++position) {
        touch(base + S::offset(position, ld, mn_last, k_last), 16, false, what);
        ++loads;
    }
}

// All loads of a few work-groups: the first and last ones, and some between.
template <int BM, int BN, int WM, int WN, bool A_MC, bool B_MC>
void walk(const Operands &p, int wg_per_cu)
{
    typedef Slice<BM, BM / WM / 16, 64 * WM * WN, A_MC, false> A;
    typedef Slice<BN, BN / WN / 16, 64 * WM * WN, B_MC, true> B;
    const int tiles = p.tiles_m * p.tiles_n * p.splits, grid = std::min(tiles, 256 * wg_per_cu);
    for (int group : {0, 1, 7, 8, grid / 2, grid - 9, grid - 2, grid - 1}) {
        if (group < 0 || group >= grid) continue;
        int steps = 2;  // two more than the tiles' own
        for (int id = group; id < tiles; id += grid) {
            int m0, n0, split, first, last;
            tile_at<BM, BN>(p, id, m0, n0, split, first, last);
            if (first >= last) fail("a tile without steps", 0, 0);
            steps += (last - first) * p.segments;
        }
        Walk<BM, BN, A_MC, B_MC> w;
        w.begin(p, group);
        int a_last = 0, a_k = 0, b_last = 0, b_k = 0;  // as the offsets in registers were last worked out
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
        walk<BM, BN, WM, WN, A_MC, B_MC>(p, tgemm::loss::kTiles[I].wg_per_cu);      \
        break;
        TGEMM_TILES(X)
#undef X
    default:
        fail("an unknown tile", 0, 0);
    }
}

}  // namespace

namespace tgemm {
namespace loss {

void read_teacher(const Teacher &t, int64_t T)
{
    rows(t.ids, T, t.K, t.ld_ids, 8, false, "ids");
    rows(t.logits, T, t.K, t.ld_logits, size_of(t.dtype), false, "teacher's logits");
}

void check_stats(const StatsArgs &a, int columns)
{
    if ((int64_t)a.groups * columns < a.op.N) fail("too few column groups", 0, 0);
    rows(a.part, a.op.M, a.groups, a.groups, 8, true, "partial statistics");
    if (a.target) {
        rows(a.target, a.op.M, 1, 1, 8, false, "targets");
        rows(a.picked, a.op.M, 1, 1, 4, true, "picked logits");
    }
    if (a.starts) {
        rows(a.starts, a.op.M, a.groups + 1, a.groups + 1, 2, false, "starts");
        rows(a.list, a.op.M, a.K, a.K, 4, false, "list");
        rows(a.student, a.op.M, a.K, a.K, 4, true, "student");
    }
}

void check_kept(const StatsArgs &a)
{
    if (a.logits) rows(a.logits, a.op.M, a.op.N, a.ldz, 4, true, "kept logits");
}

hipError_t launch_stats(bool, int tile, const StatsArgs &a, hipStream_t)
{
    walk_tile<false, false>(tile, a.op);
    check_stats(a, kTiles[tile].stat_columns);
    check_kept(a);
    return hipSuccess;
}

hipError_t launch_stats_few(const StatsArgs &a, tgemm_dtype_t dtype, int columns, int D, hipStream_t)
{
    const size_t size = size_of(dtype);
    if (a.op.M > kFewRows) fail("too many rows", 0, 0);
    rows(a.op.A, a.op.M, D, a.op.lda, size, false, "X");
    rows(a.op.B, a.op.N, D, a.op.ldb, size, false, "W");
    check_stats(a, columns);
    check_kept(a);
    return hipSuccess;
}

hipError_t launch_grad(bool, int tile, const GradArgs &a, hipStream_t)
{
    walk_tile<false, false>(tile, a.op);
    const TileShape &s = kTiles[tile];
    if (a.op.tiles_m * s.bm < a.rows || a.op.tiles_n * s.bn < (a.op.N + 63) / 64 * 64) fail("rows or columns left out", 0, 0);
    const int64_t cols = std::min<int64_t>(a.ldg, (int64_t)a.op.tiles_n * s.bn);
    if ((uintptr_t)a.G % 16 || a.ldg % 16) fail("rows that are not 16-byte aligned", 0, 0);
    for (int q = 0; q < a.planes; ++q) rows((char *)a.G + q * a.plane * 2, a.rows, cols, a.ldg, 2, true, "G");
    rows(a.coef, a.op.M, 1, 1, 4, false, "coef");
    rows(a.lse, a.op.M, 1, 1, 4, false, "lse");
    if (a.target) rows(a.target, a.op.M, 1, 1, 8, false, "targets");
    return hipSuccess;
}

hipError_t launch_grad_kept(bool, const GradArgs &a, const float *logits, int64_t ldz, hipStream_t)
{
    rows(logits, a.op.M, a.op.N, ldz, 4, false, "kept logits");
    const int64_t cols = (a.op.N + 63) / 64 * 64;
    if (cols > a.ldg || (uintptr_t)a.G % 16 || a.ldg % 16) fail("rows that are not 16-byte aligned", 0, 0);
    for (int q = 0; q < a.planes; ++q) rows((char *)a.G + q * a.plane * 2, a.rows, cols, a.ldg, 2, true, "G");
    rows(a.coef, a.op.M, 1, 1, 4, false, "coef");
    rows(a.lse, a.op.M, 1, 1, 4, false, "lse");
    if (a.target) rows(a.target, a.op.M, 1, 1, 8, false, "targets");
    return hipSuccess;
}

void check_out(const OutArgs &a)
{
    const size_t size = size_of(a.dtype);
    for (int s = 0; s < a.op.splits; ++s)
        rows((char *)a.out + s * a.split_stride * size, a.op.M, a.op.N, a.ldo, size, true, "gradient");
    if (a.row_scale) rows(a.row_scale, a.op.M, 1, 1, 4, false, "row scales");
    if (a.all_scale) touch(a.all_scale, 4, false, "scale");
}

hipError_t launch_dx(bool, int tile, const OutArgs &a, hipStream_t)
{
    walk_tile<false, true>(tile, a.op);
    check_out(a);
    return hipSuccess;
}

hipError_t launch_dw(bool, int tile, const OutArgs &a, hipStream_t)
{
    walk_tile<true, true>(tile, a.op);
    check_out(a);
    return hipSuccess;
}

void check_coef(const CoefArgs &a)
{
    rows(a.grad, a.T, 1, a.grad_step, 4, false, "grad_loss");
    if (a.weight) touch(a.weight, 4, false, "grad_weight");
    if (a.target) rows(a.target, a.T, 1, 1, 8, false, "targets");
    if (a.teacher) read_teacher(*a.teacher, a.T);
    rows(a.coef, a.T, 1, 1, 4, true, "coef");
    if (a.half || a.grad_step == 0) rows(a.row_scale, a.T, 1, 1, 4, true, "row scales");
    if (a.grad_step == 0) touch(a.all_scale, 4, true, "scale");
    else if (a.half) rows(a.exps, a.T, 1, 1, 4, true, "exponents");
}

hipError_t launch_coef(const CoefArgs &a, hipStream_t)
{
    check_coef(a);
    if (a.half && a.grad_step != 0) rows(a.block_max, coef_blocks(a.T, a.teacher != nullptr), 1, 1, 4, true, "largest exponents");
    return hipSuccess;
}

hipError_t launch_copy(const CopyArgs &a, hipStream_t)
{
    rows(a.src, a.rows, a.cols, a.ld, size_of(a.dtype), false, "an operand to copy");
    if ((uintptr_t)a.dst % 16 || a.ld_out % 8) fail("a misaligned copy", 0, 0);
    for (int q = 0; q < a.planes; ++q)
        rows((char *)a.dst + q * a.plane * 2, a.rows_out, a.ld_out, a.ld_out, 2, true, "a copy");
    if (a.make) check_coef(*a.make);
    if (a.coef) rows(a.coef, a.rows, 1, 1, 4, false, "coef");
    if (a.exps) {
        rows(a.exps, a.rows, 1, 1, 4, false, "exponents");
        rows(a.block_max, a.blocks, 1, 1, 4, false, "largest exponents");
    }
    if (a.exps) touch(a.all_scale, 4, true, "scale");
    return hipSuccess;
}

hipError_t launch_sort(const SortArgs &a, hipStream_t)
{
    read_teacher(a.teacher, a.T);
    rows(a.starts, a.T, a.groups + 1, a.groups + 1, 2, true, "starts");
    rows(a.list, a.T, a.teacher.K, a.teacher.K, 4, true, "list");
    rows(a.student, a.T, a.teacher.K, a.teacher.K, 4, true, "student");
    return hipSuccess;
}

hipError_t launch_join(const JoinArgs &a, hipStream_t)
{
    rows(a.part, a.T, a.groups, a.groups, 8, false, "partial statistics");
    if (a.teacher) {
        read_teacher(*a.teacher, a.T);
        rows(a.student, a.T, a.teacher->K, a.teacher->K, 4, false, "student");
    } else {
        rows(a.target, a.T, 1, 1, 8, false, "targets");
        rows(a.picked, a.T, 1, 1, 4, false, "picked logits");
    }
    rows(a.loss, a.T, 1, 1, 4, true, "loss");
    rows(a.lse, a.T, 1, 1, 4, true, "lse");
    if (a.summary) {
        rows(a.counted, a.T, 1, 1, 4, true, "flags");
        touch(a.summary, 12, true, "summary");
    }
    return hipSuccess;
}

hipError_t launch_summary_none(float *summary, hipStream_t)
{
    touch(summary, 12, true, "summary");
    return hipSuccess;
}

hipError_t launch_scatter(const ScatterArgs &a, hipStream_t)
{
    read_teacher(a.teacher, a.T);
    rows(a.student, a.T, a.teacher.K, a.teacher.K, 4, false, "student");
    rows(a.lse, a.T, 1, 1, 4, false, "lse");
    rows(a.coef, a.T, 1, 1, 4, false, "coef");
    for (int q = 0; q < a.planes; ++q) rows((char *)a.G + q * a.plane * 2, a.T, a.cols, a.ldg, 2, true, "G");
    return hipSuccess;
}

hipError_t launch_sum(const SumArgs &a, hipStream_t)
{
    const int64_t padded = (a.D + 3) / 4 * 4;
    for (int s = 0; s < a.count; ++s) rows(a.part + s * a.stride, a.T, padded, a.ld, 4, false, "parts of a sum");
    if ((uintptr_t)a.part % 16 || a.ld % 4 || a.stride % 4) fail("a misaligned read", 0, 0);
    rows(a.out, a.T, a.D, a.ldo, size_of(a.dtype), true, "gradient");
    if (a.row_scale) rows(a.row_scale, a.T, 1, 1, 4, false, "row scales");
    if (a.all_scale) touch(a.all_scale, 4, false, "scale");
    return hipSuccess;
}

hipError_t launch_zero(void *out, int64_t ldo, tgemm_dtype_t dtype, int64_t n, int64_t cols, hipStream_t)
{
    rows(out, n, cols, ldo, size_of(dtype), true, "gradient");
    return hipSuccess;
}

}  // namespace loss
}  // namespace tgemm

int main()
{
    int calls = 0;
    while (std::fgets(line, sizeof line, stdin)) {
        long long op, pass, type, T, V, D, ldx, ldw, sx, sw, K, nx, nw, lddx, lddw;
        if (std::sscanf(line, "%lld %lld %lld %lld %lld %lld %lld %lld %lld %lld %lld %lld %lld %lld %lld", &op, &pass, &type, &T, &V,
                        &D, &ldx, &ldw, &sx, &sw, &K, &nx, &nw, &lddx, &lddw) != 15)
            return 2;
        const tgemm_dtype_t dtype = (tgemm_dtype_t)type;
        const size_t size = size_of(dtype);
        ranges.clear();
        uintptr_t next = (uintptr_t)1 << 40;
        auto give = [&](const char *name, size_t bytes, bool written, size_t shift = 0) {
            const uintptr_t lo = next + shift;
            next += (bytes + shift + ((size_t)1 << 33)) >> 32 << 32;
            ranges.push_back({lo, lo + bytes, written, name});
            return (void *)lo;
        };
        auto matrix = [&](const char *name, long long n, long long cols, long long ld, size_t each, bool written, size_t shift = 0) {
            return give(name, n ? (size_t)((n - 1) * ld + cols) * each : 0, written, shift);
        };
        void *X = matrix("X", T, D, ldx, size, false, sx * size), *W = matrix("W", V, D, ldw, size, false, sw * size);
        int64_t *target = (int64_t *)matrix("target", op ? 0 : T, 1, 1, 8, false);
        int64_t *ids = (int64_t *)matrix("ids", op ? T : 0, K, K + 1, 8, false);
        void *logits = matrix("logits", op ? T : 0, K, K + 3, size, false);
        float *lse = (float *)matrix("lse", T, 1, 1, 4, !pass), *loss = (float *)matrix("loss", T, 1, 1, 4, true);
        float *student = (float *)matrix("student", op ? T : 0, K, K, 4, !pass);
        float *summary = (float *)give("summary", 12, !pass), *grad = (float *)matrix("grad", T, 1, nx ? 0 : 1, 4, false);
        void *dX = nx ? matrix("dX", T, D, lddx, size, true, sx * size) : nullptr;
        void *dW = nw ? matrix("dW", V, D, lddw, size, true, sw * size) : nullptr;
        const int64_t ldz = V + 3;
        float *z = (T + V) % 2 ? (float *)matrix("kept logits", T, V, ldz, 4, !pass) : nullptr;
        const size_t need = tgemm_linear_loss_workspace_size(dtype, T, V, D, X, ldx, W, ldw, op ? K : 0, (int)pass);
        void *ws = give("workspace", need, true);
        tgemm_status_t st;
        const int64_t step = nx ? 0 : 1;
        if (!op && !pass)
            st = tgemm_linear_ce_forward(dtype, T, V, D, X, ldx, W, ldw, target, -100, loss, lse, z, ldz, summary, ws, need, nullptr);
        else if (!op)
            st = tgemm_linear_ce_backward(dtype, T, V, D, X, ldx, W, ldw, target, -100, lse, z, ldz, grad, step, summary + 2, dX, lddx, dW,
                                          lddw, ws, need, nullptr);
        else if (!pass)
            st = tgemm_linear_kd_forward(dtype, T, V, D, X, ldx, W, ldw, K, ids, K + 1, dtype, logits, K + 3, 2.0f, loss, lse,
                                         student, z, ldz, summary, ws, need, nullptr);
        else
            st = tgemm_linear_kd_backward(dtype, T, V, D, X, ldx, W, ldw, K, ids, K + 1, dtype, logits, K + 3, 2.0f, lse, student,
                                          z, ldz, grad, step, nullptr, dX, lddx, dW, lddw, ws, need, nullptr);
        if (st != TGEMM_SUCCESS) {
            std::printf("status %d for: %s", (int)st, line);
            return 1;
        }
        ++calls;
    }
    std::printf("%d calls, %ld loads\n", calls, loads);
    return 0;
}
