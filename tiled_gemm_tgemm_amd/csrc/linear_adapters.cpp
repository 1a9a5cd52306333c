// C entry points of the projection with low-rank adapters: argument checks, the
// plan of a call (operand copies, tiles, parts, workspace) and its launches on
// the caller's stream.  The declarations, with the meaning of every argument,
// are in tgemm.h.
#include "linear_adapters.h"
#include "entry.h"
#include "product_plan.h"

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace {

using namespace tgemm::entry;
using namespace tgemm::adapters;
using tgemm::loss::Choice;
using tgemm::loss::choose_tile;
using tgemm::loss::CopyArgs;
using tgemm::loss::fits;
using tgemm::loss::kTiles;
using tgemm::loss::launch_copy;
using tgemm::loss::launch_dw;
using tgemm::loss::launch_sum;
using tgemm::loss::launch_zero;
using tgemm::loss::OutArgs;
using tgemm::loss::parts_of;
using tgemm::loss::SumArgs;
using tgemm::m16::kStepK;

constexpr int64_t kMaxT = ((int64_t)1 << 24) - 1;
constexpr int64_t kMaxSide = (int64_t)1 << 22;  // 256 rows of 16-bit values stay within 32-bit offsets
constexpr int64_t kMaxRank = 1024, kMaxCount = ((int64_t)1 << 15) - 1;  // twice that is a launch's z
constexpr int64_t kMaxLd = (int64_t)1 << 40;
constexpr int64_t kMaxLdA = (int64_t)1 << 26;   // 32 ranks of float32 stay within 32-bit offsets

struct Layer {
    tgemm_dtype_t dtype;
    int64_t T, N, D;
    const void *X;
    int64_t ldx;
    const void *W;
    int64_t ldw;
    int64_t count, rank;
    const void *A;
    int64_t lda, stride_a;
    const void *B;
    int64_t ldb, stride_b;
    const int64_t *ids;
    const float *scales;
};

tgemm_status_t check(const Layer &l)
{
    if (l.T < 0 || l.N < 1 || l.D < 1 || l.count < 1 || l.rank < 1 || l.ldx < l.D || l.ldw < l.D || l.lda < l.D ||
        l.ldb < l.rank || l.stride_a < 0 || l.stride_b < 0)
        return TGEMM_ERROR_INVALID_VALUE;
    if (!known(l.dtype) || l.T > kMaxT || l.N > kMaxSide || l.D > kMaxSide || l.count > kMaxCount || l.rank > kMaxRank ||
        l.ldx > kMaxLd || l.ldw > kMaxLd || l.lda > kMaxLdA || l.ldb > kMaxLd || l.stride_a > kMaxLd || l.stride_b > kMaxLd)
        return TGEMM_ERROR_NOT_SUPPORTED;
    return TGEMM_SUCCESS;
}

// What every call reads of the adapters lies in memory.
bool there(const Layer &l, Range *r)
{
    const size_t size = size_of(l.dtype);
    return at(l.X, l.T, l.D, l.ldx, size, r[0]) && at(l.W, l.N, l.D, l.ldw, size, r[1]) &&
           at(l.A, l.count, (l.rank - 1) * l.lda + l.D, l.stride_a, size, r[2]) &&
           at(l.B, l.count, (l.N - 1) * l.ldb + l.rank, l.stride_b, size, r[3]) && at(l.ids, l.T, 1, 1, 8, r[4]) &&
           at(l.scales, l.scales ? l.count : 0, 1, 1, 4, r[5]);
}
constexpr int kRead = 6;

// The matrix cores take a 16-bit operand as it is stored if its rows start
// 16-byte aligned and hold whole pieces of 16 bytes (an operand that comes
// first and lies along K: whole steps) and a tile's offsets fit 32 bits.
bool as_stored(tgemm_dtype_t dtype, const void *p, int64_t ld, int64_t cols, int64_t whole)
{
    return dtype != TGEMM_F32 && cols % whole == 0 && ld % 8 == 0 && ld <= kMaxSide && reinterpret_cast<uintptr_t>(p) % 16 == 0;
}

Stack stack_a(const Layer &l) { return Stack{l.A, l.lda, l.stride_a, false, (int)l.count, (int)l.rank}; }
Stack stack_b(const Layer &l) { return Stack{l.B, l.ldb, l.stride_b, true, (int)l.count, (int)l.rank}; }

// Whether the rows and the adapters' sums over them go through LDS as they lie.
bool along_k(const Layer &l, const void *rows, int64_t ld, int64_t K, const Stack &c)
{
    return as_stored(l.dtype, rows, ld, K, kStepK) && !c.rank_inner && c.ld % 8 == 0 && c.ld <= kMaxSide && c.stride % 8 == 0 &&
           reinterpret_cast<uintptr_t>(c.p) % 16 == 0;
}

// How the sums over K of the tokens' hidden values are cut: in parts while there
// are fewer wavefronts than keep the memory busy.  (With 8 parts at 16 to 64 row
// blocks of 16 slots, as few rows take, 256, 512 and 1024 rows of 4096 of 32
// adapters in random order 15, 24 and 44 µs, with 4, 2 and 2 12, 17 and 31.)
struct Shrink {
    int64_t part_k = 0;
    int parts = 1, slots = 1, rows_each = 16;
    bool through_lds = false;
};
Shrink shrink_of(int64_t T, int64_t K, int64_t count, bool through_lds)
{
    Shrink s;
    s.through_lds = through_lds && T > 1024;
    s.rows_each = T <= 1024 ? 16 : T < 4096 || s.through_lds ? 64 : 128;
    s.slots = T <= 1024 ? 16 : 1;
    if (s.slots > count) s.slots = (int)count;
    // (the workspace does not depend on how the adapters lie)
    int64_t parts = T <= 1024 ? 1024 / (ceil_div(T, 16) * s.slots) : 1024 / ceil_div(T, T < 4096 ? 64 : 128);
    if (T <= 1024 && parts < 2) parts = 2;  // rows in runs leave all but one slot idle
    if (parts > ceil_div(K, 512)) parts = ceil_div(K, 512);
    if (K <= 1024 && T > kFewRows) parts = 1;  // not worth the launch that adds them up
    if (parts > (T <= 1024 ? 8 : 16)) parts = T <= 1024 ? 8 : 16;
    if (parts < 1) parts = 1;
    s.part_k = round_up(ceil_div(K, parts), 256);
    s.parts = (int)ceil_div(K, s.part_k);
    return s;
}

// How a product with the weight is taken: on the tiles, or, float32 ones, on the
// library's float32 product, which needs no planes.  Six products of planes are
// 1.4 times faster than one in float32 where there are many tiles; with few of
// them, or short sums, the planes' copies and the steps' own time take that
// back.
struct Route {
    bool plain = false;
    Choice tile;
    int splits = 1;  // of the plain product
};
Route route_of(tgemm_dtype_t dtype, int64_t M, int64_t N, int64_t K, int64_t k_steps, int64_t copied, int64_t most_ld)
{
    Route r;
    r.tile = choose_tile(M, N, k_steps * (dtype == TGEMM_F32 ? 6 : 1), true);
    r.tile.splits = parts_of(k_steps, r.tile.splits);
    if (dtype != TGEMM_F32 || most_ld >= (int64_t)1 << 21) return r;
    // the planes are read and written once, 10 bytes a value, by launches of their own
    const double planes = r.tile.time + 10.0 + (double)copied * 10.0 / 4e6;
    const double plain = 10.0 + 2.0 * (double)M * (double)N * (double)K / 125e6;
    r.plain = plain < planes;
    if (r.plain) r.splits = tgemm_sgemm_splitk_choose(M, N, K);
    return r;
}

// Where a call's buffers lie in its workspace.
struct Plan {
    bool half = false;
    int planes = 1, segments = 1;
    int64_t Tp = 0, Np = 0, Dp = 0;
    int64_t total = 0;
    int64_t x = -1, w = -1, dy = -1;         // operands laid out for the matrix cores
    int64_t parts = -1, hidden_planes = -1;  // of the hidden values
    Shrink shrink;
    // forward
    bool few = false;
    Route main;
    int64_t out_part = -1;
    // backward
    Shrink shrink_x;
    int64_t u = -1, hidden = -1, parts_x = -1;
    Route dw;
    int64_t dw_part = -1;
    int64_t order = -1, starts = -1, chunks[2] = {-1, -1}, joins[2] = {-1, -1}, counts = -1, sums[2] = {-1, -1};
    int64_t arranged[2] = {-1, -1}, arranged_plane[2] = {0, 0};
    // the adapters the other way round
    int64_t turned_a = -1, turned_b = -1;
    int cut[2] = {64, 64}, most_chunks[2] = {0, 0};

    int64_t take(int64_t bytes)
    {
        const int64_t at = total;
        total += round_up(bytes, 256);
        return at;
    }
};

void plan_types(Plan &p, const Layer &l)
{
    p.half = l.dtype == TGEMM_F16;
    p.planes = l.dtype == TGEMM_F32 ? 3 : 1;
    p.segments = l.dtype == TGEMM_F32 ? 6 : 1;
    p.Tp = round_up(l.T, kStepK);
    p.Np = round_up(l.N, kStepK);
    p.Dp = round_up(l.D, kStepK);
}

int64_t planes_bytes(const Layer &l) { return l.T * planes_rank(l.rank) * 4; }

bool plan_forward(Plan &p, const Layer &l)
{
    plan_types(p, l);
    p.few = l.T <= kFewRows;
    p.shrink = shrink_of(l.T, l.D, l.count, along_k(l, l.X, l.ldx, l.D, stack_a(l)));
    if (p.few || p.shrink.parts > 1) p.parts = p.take(p.shrink.parts * l.T * l.rank * 4);
    if (p.few) return true;
    p.hidden_planes = p.take(planes_bytes(l));
    p.main = route_of(l.dtype, l.T, l.N, l.D, p.Dp / kStepK, (l.T + l.N) * l.D, l.ldx > l.ldw ? l.ldx : l.ldw);
    if (p.main.plain) {
        p.out_part = p.take((int64_t)tgemm_sgemm_splitk_workspace_size(l.T, l.N, l.D, p.main.splits));
        return true;
    }
    if (!as_stored(l.dtype, l.X, l.ldx, l.D, kStepK)) p.x = p.take(l.T * p.Dp * 2 * p.planes);
    if (!as_stored(l.dtype, l.W, l.ldw, l.D, 8)) p.w = p.take(l.N * p.Dp * 2 * p.planes);
    if (p.main.tile.splits > 1) p.out_part = p.take(p.main.tile.splits * l.T * p.Np * 4);
    return fits(l.T, l.N, p.main.tile.tile, p.main.tile.splits);
}

struct Need {
    bool x, w, a, b;
};

bool plan_backward(Plan &p, const Layer &l, const void *dY, int64_t lddy, Need need, bool have_hidden)
{
    plan_types(p, l);
    if (need.a || need.b) {
        const int64_t C[2] = {l.D, l.N}, most_adapters = l.count < l.T ? l.count : l.T;
        p.order = p.take(l.T * 4);
        p.starts = p.take((l.count + 1) * 4);
        p.counts = p.take(8);
        for (int n = 0; n < 2; ++n) {
            // 512 work-groups or more, of 64 tokens or more
            const int64_t columns = ceil_div(C[n], kOuterColumns);
            int64_t tokens = round_up(ceil_div(l.T * columns, 512), 64);
            if (tokens < 64) tokens = 64;
            if (tokens > kMostTokens) tokens = kMostTokens;
            p.cut[n] = (int)tokens;
            p.most_chunks[n] = (int)(l.T / tokens + most_adapters);
            p.chunks[n] = p.take(((int64_t)p.most_chunks[n] + 1) * (int64_t)sizeof(Chunk));
            p.joins[n] = p.take(l.count * 8);
            if (!(n == 0 ? need.a : need.b)) continue;
            // an adapter of several chunks has more than `tokens` tokens, and at most twice as many chunks as whole ones
            p.sums[n] = p.take(2 * (l.T / tokens) * C[n] * l.rank * 4);
            // a chunk's small values are whole 64s
            const bool direct = n == 0 ? as_stored(l.dtype, l.X, l.ldx, l.D, 8) : as_stored(l.dtype, dY, lddy, l.N, 8);
            if (direct) {
                p.arranged_plane[n] = (l.T + 64 * (l.T / tokens + most_adapters)) / 64 * 64 * l.rank;
                p.arranged[n] = p.take(2 * p.arranged_plane[n] * 2);
            }
        }
    }
    if (l.T == 0) return true;
    // A copy of the adapters the other way round is read 16 bytes at a time (hidden values of 8192×16384 with 8 adapters
    // of 32 ranks 75 µs, against 280 with B as it lies).  It is worth its launch, 7 to 20 µs, where the adapters have
    // fewer ranks together than there are tokens, and those are many: from 1025 on they go through LDS.
    if ((need.x || need.a) && l.T > 1024 && 4 * l.count * l.rank <= l.T) {
        p.turned_b = p.take(l.count * l.rank * round_up(l.N, 8) * (int64_t)size_of(l.dtype));
        if (need.x) p.turned_a = p.take(l.count * l.D * round_up(l.rank, 8) * (int64_t)size_of(l.dtype));
    }
    if (need.x || need.a) {
        // (turned, B lies along the sum)
        const Stack b{nullptr, round_up(l.N, 8), 0, false, (int)l.count, (int)l.rank};
        p.shrink = shrink_of(l.T, l.N, l.count, p.turned_b >= 0 && along_k(l, dY, lddy, l.N, b));
        if (p.shrink.parts > 1) p.parts = p.take(p.shrink.parts * l.T * l.rank * 4);
        if (need.a) p.u = p.take(l.T * l.rank * 4);
        if (need.x) p.hidden_planes = p.take(planes_bytes(l));
    }
    if (need.b && !have_hidden) {
        p.shrink_x = shrink_of(l.T, l.D, l.count, along_k(l, l.X, l.ldx, l.D, stack_a(l)));
        if (p.shrink_x.parts > 1) p.parts_x = p.take(p.shrink_x.parts * l.T * l.rank * 4);
        p.hidden = p.take(l.T * l.rank * 4);
    }
    const int64_t widest = l.ldx > lddy ? l.ldx > l.ldw ? l.ldx : l.ldw : lddy > l.ldw ? lddy : l.ldw;
    if (need.x) p.main = route_of(l.dtype, l.T, l.D, l.N, p.Np / kStepK, (l.T + l.D) * l.N, widest);
    if (need.w) p.dw = route_of(l.dtype, l.N, l.D, l.T, p.Tp / kStepK, (l.N + l.D) * l.T, widest);
    // dY comes first in either product: along K for dX, across for dW, whose sum has whole steps of tokens
    if ((need.x && !p.main.plain && !as_stored(l.dtype, dY, lddy, l.N, kStepK)) ||
        (need.w && !p.dw.plain && (!as_stored(l.dtype, dY, lddy, l.N, 8) || l.T % kStepK != 0)))
        p.dy = p.take(p.Tp * p.Np * 2 * p.planes);
    bool fit = true;
    if (need.x && p.main.plain) {
        p.out_part = p.take((int64_t)tgemm_sgemm_splitk_workspace_size(l.T, l.D, l.N, p.main.splits));
    } else if (need.x) {
        if (!as_stored(l.dtype, l.W, l.ldw, l.D, 8)) p.w = p.take(l.N * p.Dp * 2 * p.planes);
        if (p.main.tile.splits > 1) p.out_part = p.take(p.main.tile.splits * l.T * p.Dp * 4);
        fit = fits(l.T, l.D, p.main.tile.tile, p.main.tile.splits);
    }
    if (need.w && p.dw.plain) {
        p.dw_part = p.take((int64_t)tgemm_sgemm_splitk_workspace_size(l.N, l.D, l.T, p.dw.splits));
    } else if (need.w) {
        if (!as_stored(l.dtype, l.X, l.ldx, l.D, 8)) p.x = p.take(l.T * p.Dp * 2 * p.planes);
        if (p.dw.tile.splits > 1) p.dw_part = p.take(p.dw.tile.splits * l.N * p.Dp * 4);
        fit = fit && fits(l.N, l.D, p.dw.tile.tile, p.dw.tile.splits);
    }
    return fit;
}

// An operand as the matrix cores read it.
struct Stored {
    const void *p;
    int64_t ld, plane;
};

// The operand as stored, or copied to `room` (offset -1: as stored).
hipError_t lay_out(const Plan &p, const Layer &l, const void *src, int64_t ld, int64_t rows, int64_t cols, int64_t room,
                   int64_t rows_out, void *ws, Stored &s, hipStream_t stream)
{
    s = Stored{src, ld, 0};
    if (room < 0) return hipSuccess;
    CopyArgs c{};
    c.src = src;
    c.ld = ld;
    c.dtype = l.dtype;
    c.rows = rows;
    c.cols = cols;
    c.dst = in<void>(ws, room);
    c.rows_out = rows_out;
    c.ld_out = round_up(cols, kStepK);
    c.plane = rows_out * c.ld_out;
    c.planes = p.planes;
    s = Stored{c.dst, c.ld_out, c.plane};
    return launch_copy(c, stream);
}

ShrinkArgs shrink_args(const Layer &l, const Shrink &s, const void *rows, int64_t ld, int64_t K, const Stack &c)
{
    ShrinkArgs a{};
    a.dtype = l.dtype;
    a.T = l.T;
    a.K = K;
    a.rows = rows;
    a.ld = ld;
    a.c = c;
    a.ids = l.ids;
    a.scales = l.scales;
    a.part_k = s.part_k;
    a.parts = s.parts;
    a.slots = s.slots;
    a.rows_each = s.rows_each;
    a.through_lds = s.through_lds;
    return a;
}

// Hidden values to `hidden` and `planes`, either of which may be NULL.
hipError_t make_hidden(ShrinkArgs a, float *parts, float *hidden, void *planes, hipStream_t stream)
{
    if (a.parts == 1) {
        a.part = hidden;
        a.planes = planes;
        return launch_shrink(a, stream);
    }
    a.part = parts;
    const hipError_t e = launch_shrink(a, stream);
    return e != hipSuccess ? e : launch_finish(a, hidden, planes, stream);
}

// The product on the tiles with its adapters' part.
hipError_t run_product(const Plan &p, const Layer &l, ProductArgs a, bool b_mc, int64_t steps, int64_t ld_part, void *out,
                       int64_t ldo, void *ws, hipStream_t stream)
{
    const Choice &tile = p.main.tile;
    const Expand e = a.e;
    a.stored = l.dtype;
    a.out = out;
    a.ldo = ldo;
    a.dtype = l.dtype;
    if (tile.splits == 1) return launch_product(p.half, b_mc, tile.tile, a, stream);
    a.op.splits = tile.splits;
    a.op.steps_per_split = (int)ceil_div(steps, tile.splits);
    a.out = in<float>(ws, p.out_part);
    a.ldo = ld_part;
    a.dtype = TGEMM_F32;
    a.split_stride = l.T * ld_part;
    a.e.ids = nullptr;
    const hipError_t st = launch_product(p.half, b_mc, tile.tile, a, stream);
    if (st != hipSuccess) return st;
    return launch_add(AddArgs{l.T, a.op.N, in<float>(ws, p.out_part), ld_part, a.split_stride, tile.splits, out, ldo, l.dtype, e}, stream);
}

// A float32 product as it is.
tgemm_status_t run_plain(const Route &r, tgemm_op_t op_a, tgemm_op_t op_b, int64_t M, int64_t N, int64_t K, const void *A, int64_t lda,
                         const void *B, int64_t ldb, void *C, int64_t ldc, void *room, hipStream_t stream)
{
    return tgemm_sgemm_splitk_ex(op_a, op_b, M, N, K, (const float *)A, lda, (const float *)B, ldb, (float *)C, ldc, r.splits, room,
                                 tgemm_sgemm_splitk_workspace_size(M, N, K, r.splits), stream);
}

tgemm_status_t forward(const Plan &p, const Layer &l, void *Y, int64_t ldy, float *hidden, void *ws, hipStream_t stream)
{
    ShrinkArgs s = shrink_args(l, p.shrink, l.X, l.ldx, l.D, stack_a(l));
    if (p.few) {
        s.part = in<float>(ws, p.parts);
        hipError_t e = launch_shrink(s, stream);
        if (e == hipSuccess && hidden != nullptr) e = launch_finish(s, hidden, nullptr, stream);
        if (e != hipSuccess) return from_hip(e);
        const FewArgs f{l.dtype, (int)l.T, (int)l.N, (int)l.D, l.X, l.ldx, l.W, l.ldw, Y, ldy,
                        Expand{l.ids, l.scales, s.part, l.T * l.rank, s.parts, nullptr, stack_b(l)},
                        as_stored(l.dtype, l.X, l.ldx, l.D, kStepK) && as_stored(l.dtype, l.W, l.ldw, l.D, kStepK)};
        return from_hip(launch_few(f, stream));
    }
    void *planes = in<void>(ws, p.hidden_planes);
    hipError_t e = make_hidden(s, in<float>(ws, p.parts), hidden, planes, stream);
    const Expand expand{l.ids, l.scales, nullptr, 0, 1, planes, stack_b(l)};
    if (p.main.plain) {
        if (e != hipSuccess) return from_hip(e);
        const tgemm_status_t st = run_plain(p.main, TGEMM_OP_N, TGEMM_OP_T, l.T, l.N, l.D, l.X, l.ldx, l.W, l.ldw, Y, ldy,
                                            in<void>(ws, p.out_part), stream);
        if (st != TGEMM_SUCCESS) return st;
        return from_hip(launch_add(AddArgs{l.T, l.N, (const float *)Y, ldy, 0, 1, Y, ldy, l.dtype, expand}, stream));
    }
    Stored x, w;
    if (e == hipSuccess) e = lay_out(p, l, l.X, l.ldx, l.T, l.D, p.x, l.T, ws, x, stream);
    if (e == hipSuccess) e = lay_out(p, l, l.W, l.ldw, l.N, l.D, p.w, l.N, ws, w, stream);
    if (e != hipSuccess) return from_hip(e);
    ProductArgs a{};
    const int64_t steps = p.Dp / kStepK;
    a.op = tgemm::loss::operands(p.segments, l.T, l.N, steps, p.main.tile.tile);
    a.op.A = x.p;
    a.op.lda = x.ld;
    a.op.plane_a = x.plane;
    a.op.mn_a = (int)l.T;
    a.op.B = w.p;
    a.op.ldb = w.ld;
    a.op.plane_b = w.plane;
    a.op.mn_b = (int)l.N;
    a.op.k_b = (int)(p.w >= 0 ? p.Dp : l.D);
    a.e = expand;
    return from_hip(run_product(p, l, a, false, steps, p.Np, Y, ldy, ws, stream));
}

struct Gradients {
    void *dX;
    int64_t lddx;
    void *dW;
    int64_t lddw;
    void *dA;
    int64_t ldda, stride_da;
    void *dB;
    int64_t lddb, stride_db;
};

tgemm_status_t backward(const Plan &p, const Layer &l, const void *dY, int64_t lddy, const float *hidden, const Gradients &g,
                        void *ws, hipStream_t stream)
{
    hipError_t e = hipSuccess;
    GroupArgs o{};
    const bool grouped = g.dA != nullptr || g.dB != nullptr;
    if (grouped) {
        o.ids = l.ids;
        o.T = (int)l.T;
        o.count = (int)l.count;
        o.order = in<int>(ws, p.order);
        o.starts = in<int>(ws, p.starts);
        for (int n = 0; n < 2; ++n)
            o.cuts[n] = Cut{p.cut[n], in<Chunk>(ws, p.chunks[n]), in<int2>(ws, p.joins[n]), in<int>(ws, p.counts) + n};
    }
    Stack a_stack = stack_a(l), b_stack = stack_b(l);
    const int64_t ld_a = round_up(l.rank, 8), ld_b = round_up(l.N, 8);
    const TurnArgs turn_b{l.dtype, b_stack, l.N, in<void>(ws, p.turned_b), ld_b, l.rank * ld_b};
    const TurnArgs turn_a{l.dtype, a_stack, l.D, in<void>(ws, p.turned_a), ld_a, l.D * ld_a};
    e = launch_turn(turn_b, turn_a, grouped ? &o : nullptr, stream);
    if (e != hipSuccess) return from_hip(e);
    if (turn_b.to != nullptr) b_stack = Stack{turn_b.to, ld_b, turn_b.to_stride, false, (int)l.count, (int)l.rank};
    if (turn_a.to != nullptr) a_stack = Stack{turn_a.to, ld_a, turn_a.to_stride, true, (int)l.count, (int)l.rank};
    float *u = in<float>(ws, p.u);
    void *planes = in<void>(ws, p.hidden_planes);
    if (l.T > 0 && (g.dX != nullptr || g.dA != nullptr))
        e = make_hidden(shrink_args(l, p.shrink, dY, lddy, l.N, b_stack), in<float>(ws, p.parts), u, planes, stream);
    if (e == hipSuccess && p.hidden >= 0) {
        hidden = in<float>(ws, p.hidden);
        e = make_hidden(shrink_args(l, p.shrink_x, l.X, l.ldx, l.D, stack_a(l)), in<float>(ws, p.parts_x),
                        in<float>(ws, p.hidden), nullptr, stream);
    }
    if (e != hipSuccess) return from_hip(e);

    if (g.dA != nullptr || g.dB != nullptr) {
        OuterArgs r[2] = {};
        for (int n = 0; n < 2; ++n) {
            r[n].dtype = l.dtype;
            r[n].scales = l.scales;
            r[n].order = o.order;
            r[n].part = in<float>(ws, p.sums[n]);
            r[n].count = (int)l.count;
            r[n].rank = (int)l.rank;
            r[n].C = (int)(n == 0 ? l.D : l.N);
            r[n].rows = n == 0 ? l.X : dY;
            r[n].ld = n == 0 ? l.ldx : lddy;
            r[n].small = n == 0 ? u : hidden;
            r[n].arranged = in<void>(ws, p.arranged[n]);
            r[n].arranged_plane = p.arranged_plane[n];
            r[n].cut = o.cuts[n];
            r[n].most_chunks = p.most_chunks[n];
            r[n].out = n == 0 ? g.dA : g.dB;
            r[n].ldo = n == 0 ? g.ldda : g.lddb;
            r[n].stride_out = n == 0 ? g.stride_da : g.stride_db;
            r[n].rank_inner = n == 1;
        }
        if (l.T > 0 && (r[0].arranged != nullptr || r[1].arranged != nullptr)) e = launch_arrange(r[0], r[1], stream);
        if (e == hipSuccess && l.T > 0) e = launch_outer(r[0], r[1], stream);
        if (e == hipSuccess) e = launch_join(r[0], r[1], stream);
        if (e != hipSuccess) return from_hip(e);
    }
    if (l.T == 0) return g.dW ? from_hip(launch_zero(g.dW, g.lddw, l.dtype, l.N, l.D, stream)) : TGEMM_SUCCESS;

    const Expand expand{l.ids, l.scales, nullptr, 0, 1, planes, a_stack};
    if (g.dX != nullptr && p.main.plain) {
        const tgemm_status_t st = run_plain(p.main, TGEMM_OP_N, TGEMM_OP_N, l.T, l.D, l.N, dY, lddy, l.W, l.ldw, g.dX, g.lddx,
                                            in<void>(ws, p.out_part), stream);
        if (st != TGEMM_SUCCESS) return st;
        e = launch_add(AddArgs{l.T, l.D, (const float *)g.dX, g.lddx, 0, 1, g.dX, g.lddx, l.dtype, expand}, stream);
        if (e != hipSuccess) return from_hip(e);
    }
    if (g.dW != nullptr && p.dw.plain) {
        const tgemm_status_t st = run_plain(p.dw, TGEMM_OP_T, TGEMM_OP_N, l.N, l.D, l.T, dY, lddy, l.X, l.ldx, g.dW, g.lddw,
                                            in<void>(ws, p.dw_part), stream);
        if (st != TGEMM_SUCCESS) return st;
    }
    const bool tiled_x = g.dX != nullptr && !p.main.plain, tiled_w = g.dW != nullptr && !p.dw.plain;
    Stored dy, w, x;
    if (tiled_x || tiled_w) e = lay_out(p, l, dY, lddy, l.T, l.N, p.dy, p.Tp, ws, dy, stream);
    if (e == hipSuccess && tiled_x) {
        e = lay_out(p, l, l.W, l.ldw, l.N, l.D, p.w, l.N, ws, w, stream);
        if (e != hipSuccess) return from_hip(e);
        ProductArgs a{};
        const int64_t steps = p.Np / kStepK;
        a.op = tgemm::loss::operands(p.segments, l.T, l.D, steps, p.main.tile.tile);
        a.op.A = dy.p;
        a.op.lda = dy.ld;
        a.op.plane_a = dy.plane;
        a.op.mn_a = (int)l.T;
        a.op.B = w.p;
        a.op.ldb = w.ld;
        a.op.plane_b = w.plane;
        a.op.mn_b = (int)(p.w >= 0 ? p.Dp : l.D);
        a.op.k_b = (int)l.N;
        a.e = expand;
        e = run_product(p, l, a, true, steps, p.Dp, g.dX, g.lddx, ws, stream);
    }
    if (e == hipSuccess && tiled_w) {
        e = lay_out(p, l, l.X, l.ldx, l.T, l.D, p.x, l.T, ws, x, stream);
        if (e != hipSuccess) return from_hip(e);
        OutArgs d{};
        const int64_t steps = p.Tp / kStepK;
        d.op = tgemm::loss::operands(p.segments, l.N, l.D, steps, p.dw.tile.tile);
        d.op.A = dy.p;
        d.op.lda = dy.ld;
        d.op.plane_a = dy.plane;
        d.op.mn_a = (int)(p.dy >= 0 ? p.Np : l.N);
        d.op.k_a = (int)p.Tp;
        d.op.B = x.p;
        d.op.ldb = x.ld;
        d.op.plane_b = x.plane;
        d.op.mn_b = (int)(p.x >= 0 ? p.Dp : l.D);
        d.op.k_b = (int)l.T;
        d.out = g.dW;
        d.ldo = g.lddw;
        d.dtype = l.dtype;
        if (p.dw.tile.splits > 1) {
            d.op.splits = p.dw.tile.splits;
            d.op.steps_per_split = (int)ceil_div(steps, p.dw.tile.splits);
            d.out = in<float>(ws, p.dw_part);
            d.ldo = p.Dp;
            d.dtype = TGEMM_F32;
            d.split_stride = l.N * p.Dp;
        }
        e = launch_dw(p.half, p.dw.tile.tile, d, stream);
        if (e == hipSuccess && p.dw.tile.splits > 1) {
            const SumArgs s{l.N, l.D, in<float>(ws, p.dw_part), p.Dp, d.split_stride, p.dw.tile.splits, nullptr, nullptr, g.dW, g.lddw, l.dtype};
            e = launch_sum(s, stream);
        }
    }
    return from_hip(e);
}

}  // namespace

extern "C" {

size_t tgemm_linear_adapters_workspace_size(tgemm_dtype_t dtype, int64_t T, int64_t N, int64_t D, const void *X, int64_t ldx,
                                            const void *W, int64_t ldw, int64_t count, int64_t rank, const void *dY, int64_t lddy,
                                            int need)
{
    const Layer l{dtype, T, N, D, X, ldx, W, ldw, count, rank, nullptr, D, 0, nullptr, rank, 0, nullptr, nullptr};
    if (check(l) != TGEMM_SUCCESS || need < 0 || need > 15) return 0;
    Plan p;
    if (need == 0) return T > 0 && plan_forward(p, l) ? (size_t)p.total : 0;
    if (lddy < N || lddy > kMaxLd) return 0;
    const Need n{(need & 1) != 0, (need & 2) != 0, (need & 4) != 0, (need & 8) != 0};
    return plan_backward(p, l, dY, lddy, n, false) ? (size_t)p.total : 0;
}

tgemm_status_t tgemm_linear_adapters_forward(tgemm_dtype_t dtype, int64_t T, int64_t N, int64_t D, const void *X, int64_t ldx,
                                             const void *W, int64_t ldw, int64_t count, int64_t rank,
                                             const void *A, int64_t lda, int64_t stride_a,
                                             const void *B, int64_t ldb, int64_t stride_b,
                                             const int64_t *ids, const float *scales,
                                             void *Y, int64_t ldy, float *hidden,
                                             void *workspace, size_t workspace_bytes, hipStream_t stream)
{
    const Layer l{dtype, T, N, D, X, ldx, W, ldw, count, rank, A, lda, stride_a, B, ldb, stride_b, ids, scales};
    const tgemm_status_t st = check(l);
    if (st != TGEMM_SUCCESS) return st;
    if (ldy < N) return TGEMM_ERROR_INVALID_VALUE;
    if (ldy > kMaxLd) return TGEMM_ERROR_NOT_SUPPORTED;
    if (T == 0) return TGEMM_SUCCESS;
    Plan p;
    if (!plan_forward(p, l)) return TGEMM_ERROR_NOT_SUPPORTED;
    Range r[kRead], w[3];
    if (!there(l, r) || !at(Y, T, N, ldy, size_of(dtype), w[0]) || !at(hidden, hidden ? T : 0, rank, rank, 4, w[1]) ||
        !room_at(workspace, workspace_bytes, p.total, w[2]) || !disjoint(w, 3, r, kRead))
        return TGEMM_ERROR_INVALID_VALUE;
    return forward(p, l, Y, ldy, hidden, workspace, stream);
}

tgemm_status_t tgemm_linear_adapters_backward(tgemm_dtype_t dtype, int64_t T, int64_t N, int64_t D, const void *X, int64_t ldx,
                                              const void *W, int64_t ldw, int64_t count, int64_t rank,
                                              const void *A, int64_t lda, int64_t stride_a,
                                              const void *B, int64_t ldb, int64_t stride_b,
                                              const int64_t *ids, const float *scales,
                                              const float *hidden, const void *dY, int64_t lddy,
                                              void *dX, int64_t lddx, void *dW, int64_t lddw,
                                              void *dA, int64_t ldda, int64_t stride_da,
                                              void *dB, int64_t lddb, int64_t stride_db,
                                              void *workspace, size_t workspace_bytes, hipStream_t stream)
{
    const Layer l{dtype, T, N, D, X, ldx, W, ldw, count, rank, A, lda, stride_a, B, ldb, stride_b, ids, scales};
    const tgemm_status_t st = check(l);
    if (st != TGEMM_SUCCESS) return st;
    if (lddy < N || (dX && lddx < D) || (dW && lddw < D) || (dA && (ldda < D || stride_da < 0)) ||
        (dB && (lddb < rank || stride_db < 0)))
        return TGEMM_ERROR_INVALID_VALUE;
    if (lddy > kMaxLd || lddx > kMaxLd || lddw > kMaxLd || ldda > kMaxLd || stride_da > kMaxLd || lddb > kMaxLd || stride_db > kMaxLd)
        return TGEMM_ERROR_NOT_SUPPORTED;
    const Need need{dX != nullptr && T > 0, dW != nullptr, dA != nullptr, dB != nullptr};
    if (!need.x && !need.w && !need.a && !need.b) return TGEMM_SUCCESS;
    Plan p;
    if (!plan_backward(p, l, dY, lddy, need, hidden != nullptr)) return TGEMM_ERROR_NOT_SUPPORTED;
    const size_t size = size_of(dtype);
    const int64_t span_a = (rank - 1) * ldda + D, span_b = (N - 1) * lddb + rank;
    Range r[kRead + 2], w[5];
    if (!there(l, r) || !at(hidden, hidden ? T : 0, rank, rank, 4, r[kRead]) || !at(dY, T, N, lddy, size, r[kRead + 1]) ||
        !at(dX, dX ? T : 0, D, lddx, size, w[0]) || !at(dW, dW ? N : 0, D, lddw, size, w[1]) ||
        (dA && !separate(count, rank, D, ldda, stride_da)) || !at(dA, dA ? count : 0, span_a, stride_da, size, w[2]) ||
        (dB && !separate(count, N, rank, lddb, stride_db)) || !at(dB, dB ? count : 0, span_b, stride_db, size, w[3]) ||
        !room_at(workspace, workspace_bytes, p.total, w[4]) || !disjoint(w, 5, r, kRead + 2))
        return TGEMM_ERROR_INVALID_VALUE;
    const Gradients g{need.x ? dX : nullptr, lddx, dW, lddw, dA, ldda, stride_da, dB, lddb, stride_db};
    return backward(p, l, dY, lddy, hidden, g, workspace, stream);
}

}  // extern "C"
