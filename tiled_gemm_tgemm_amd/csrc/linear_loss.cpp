// C entry points of the loss operators on an output head's product: argument
// checks, the plan of a call (operand copies, pieces of the vocabulary, tiles,
// workspace) and its launches on the caller's stream.  The declarations, with
// the meaning of every argument, are in tgemm.h.
#include "entry.h"
#include "linear_loss.h"
#include "product_plan.h"

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace {

using namespace tgemm::entry;
using namespace tgemm::loss;
using tgemm::m16::kStepK;
using tgemm::m16::Operands;

constexpr int64_t kMaxT = ((int64_t)1 << 24) - 1;  // a launch of 256 threads a row stays below 2^32 threads
constexpr int64_t kMaxV = (int64_t)1 << 24;
constexpr int64_t kMaxD = (int64_t)1 << 22;   // 256 rows of 16-bit values stay within 32-bit offsets
constexpr int64_t kMaxK = 1024;
constexpr int64_t kMaxLd = (int64_t)1 << 40;
// Bytes of one piece of the logits' gradient: large enough that the products
// of a piece fill the GPU for several rounds, small enough to stay near the
// 256 MiB last-level cache between the product that writes it and the two
// that read it.  It has 2048 words at least, however many rows there are, so
// from 65536 rows (float32 21845) on a piece takes T·2048 values: dX's sums are
// read and written once a piece, which fewer words do not cover (2048, 1024 and
// 512 words at 262144×32768×2048 bf16 110, 138 and 189 ms, 1048576×32768×256
// 79, 96 and 128, 100000×32768×1024 float32 107, 115 and 129).
constexpr int64_t kPieceBytes = (int64_t)256 << 20;
constexpr int64_t kMinPiece = 2048, kMaxPiece = (int64_t)1 << 22;

// Up to this many rows the logits' gradient is held as two 16-bit planes.  One
// plane's roundings are as large as those of the results, so the two together
// are sqrt(2) times the latter, which a sum over many rows' entries comes close
// to; a few rows' gradients hang on a few entries, whose rounding may be the
// largest there is (3 rows of distillation 1.8 times the results' own rounding,
// 128 rows 1.47).  A second plane takes little time while W's way from memory
// is what takes it (distillation backward at 32000×2048 with 8, 33 and 128
// rows 115 -> 113, 114 -> 122 and 138 -> 159 µs; 512 rows would be 244 -> 350).
constexpr int64_t kTwoPlaneRows = 128;

struct Head {
    tgemm_dtype_t dtype;
    int64_t T, V, D;
    const void *X;
    int64_t ldx;
    const void *W;
    int64_t ldw;
};

tgemm_status_t check_head(const Head &h)
{
    if (h.T < 0 || h.V < 1 || h.D < 1 || h.ldx < h.D || h.ldw < h.D) return TGEMM_ERROR_INVALID_VALUE;
    if (!known(h.dtype) || h.T > kMaxT || h.V > kMaxV || h.D > kMaxD || h.ldx > kMaxLd || h.ldw > kMaxLd)
        return TGEMM_ERROR_NOT_SUPPORTED;
    return TGEMM_SUCCESS;
}

// The matrix cores take an operand as it is stored if it is 16-bit, its rows
// start 16-byte aligned and hold whole pieces of 16 bytes, and a tile's
// offsets fit 32 bits; otherwise the call lays a copy out first.  X has to
// end in whole steps of K besides, so that what stands in for W's last step
// meets zeros.
bool as_stored(const void *p, int64_t ld, const Head &h, int64_t whole = 8)
{
    return h.dtype != TGEMM_F32 && h.D % whole == 0 && ld % 8 == 0 && ld <= kMaxD &&
           reinterpret_cast<uintptr_t>(p) % 16 == 0;
}

// Where a call's buffers lie in its workspace.
struct Plan {
    bool half = false;
    int planes = 1, segments = 1;      // of X and W, and of their product
    int g_planes = 1;                  // of the logits' gradient
    int dw_segments = 1;
    int64_t dx_rows = 0;
    int64_t Tp = 0, Dp = 0;
    bool copy_x = false, copy_w = false;
    int64_t total = 0;
    int64_t x = -1, w = -1, xs = -1;  // operands laid out for the matrix cores
    // forward
    bool few = false;
    int stat_tile = 0, groups = 0, group_columns = 0;
    int64_t part = -1, picked = -1, counted = -1, starts = -1, list = -1;
    // backward
    int64_t piece = 0, pieces = 0, ldg = 0;
    int grad_tile = 0, dx_tile = 0, dw_tile = 0, dx_splits = 1, dw_splits = 1;
    bool dx_direct = false;
    int64_t coef = -1, row_scale = -1, exps = -1, block_max = -1, all_scale = -1, g = -1, dx_part = -1, dw_part = -1;

    int64_t take(int64_t bytes)
    {
        const int64_t at = total;
        total += round_up(bytes, 256);
        return at;
    }
};

void plan_operands(Plan &p, const Head &h, bool backward)
{
    p.half = h.dtype == TGEMM_F16;
    p.planes = h.dtype == TGEMM_F32 ? 3 : 1;
    p.segments = h.dtype == TGEMM_F32 ? 6 : 1;
    p.Tp = round_up(h.T, kStepK);
    p.Dp = round_up(h.D, kStepK);
    p.copy_w = !as_stored(h.W, h.ldw, h);
    if (p.copy_w) p.w = p.take(h.V * p.Dp * 2 * p.planes);
    // the backward pass holds X with its rows that do not count cleared (`xs`);
    // only fp16, where `xs` is scaled too, may need another copy
    p.copy_x = !as_stored(h.X, h.ldx, h, kStepK) && (!backward || p.half);
    if (p.copy_x) p.x = p.take(h.T * p.Dp * 2 * p.planes);
    if (backward) p.xs = p.take(p.Tp * p.Dp * 2 * p.planes);
}

bool plan_forward(Plan &p, const Head &h, int64_t teacher_k)
{
    // The rows of X come from the caches once for every 16 words, which is as
    // much again as W from 16 rows on: tiles take more than 8 rows sooner
    // where they need no copy of W and the vocabulary gives every compute unit
    // one (µs, tiles against few rows' kernel: 16×32000×2048 bf16 28, 35 and
    // 16×128256×1024 50, 65; 16×16384×2048 25, 21, 32×8192×512 13, 10 and
    // 32×5000×4096 39, 28; with a copy 20×32000×1001 55, 45, 32 of them 55, 55;
    // the same W call after call, part of which stays in the last-level cache).
    const bool stored = as_stored(h.X, h.ldx, h, kStepK) && as_stored(h.W, h.ldw, h);
    p.few = h.T <= (stored && h.V > kFewBelow ? 8 : kFewRows);
    if (p.few) {
        p.group_columns = few_columns(h.V);
    } else {
        plan_operands(p, h, false);
        p.stat_tile = choose_tile(h.T, h.V, p.Dp / kStepK * p.segments).tile;
        p.group_columns = kTiles[p.stat_tile].stat_columns;
    }
    p.groups = (int)ceil_div(h.V, p.group_columns);
    p.part = p.take(h.T * p.groups * 8);
    if (teacher_k > 0) {
        p.starts = p.take(h.T * (p.groups + 1) * 2);
        p.list = p.take(h.T * teacher_k * 4);
    } else {
        p.picked = p.take(h.T * 4);
    }
    p.counted = p.take(h.T * 4);
    return p.few || fits(h.T, h.V, p.stat_tile, 1);
}

bool plan_backward(Plan &p, const Head &h)
{
    plan_operands(p, h, true);
    p.g_planes = h.dtype == TGEMM_F32 ? 3 : h.T <= kTwoPlaneRows ? 2 : 1;
    // dW meets both of two planes one after the other; dX has them as rows, so
    // that W is read once, and adds the two rows' sums up with the parts'
    p.dw_segments = h.dtype == TGEMM_F32 ? 6 : p.g_planes;
    p.dx_rows = p.g_planes == 2 ? 2 * p.Tp : h.T;
    int64_t cols = kPieceBytes / (p.Tp * 2 * p.g_planes) / 256 * 256;
    cols = cols < kMinPiece ? kMinPiece : cols > kMaxPiece ? kMaxPiece : cols;
    p.pieces = ceil_div(h.V, cols);
    p.piece = round_up(ceil_div(h.V, p.pieces), 256);
    p.pieces = ceil_div(h.V, p.piece);
    p.ldg = p.piece + 128;
    p.grad_tile = choose_tile(p.Tp, p.piece, p.Dp / kStepK * p.segments).tile;
    const Choice dw = choose_tile(p.piece, h.D, p.Tp / kStepK * p.dw_segments, true);
    p.dw_tile = dw.tile;
    p.dw_splits = parts_of(p.Tp / kStepK, dw.splits);
    const Choice dx = choose_tile(p.dx_rows, h.D, p.piece / kStepK * p.segments, true);
    p.dx_tile = dx.tile;
    p.dx_splits = parts_of(ceil_div(h.V < p.piece ? h.V : p.piece, kStepK), dx.splits);
    p.dx_direct = p.pieces == 1 && p.dx_splits == 1 && p.dx_rows == h.T;
    p.coef = p.take(h.T * 4);
    p.row_scale = p.take(h.T * 4);
    p.all_scale = p.take(4);
    if (p.half) {
        p.exps = p.take(h.T * 4);
        p.block_max = p.take(coef_blocks(h.T, true) * 4);
    }
    p.g = p.take(p.Tp * p.ldg * 2 * p.g_planes);
    if (!p.dx_direct) p.dx_part = p.take(p.dx_splits * p.dx_rows * p.Dp * 4);
    if (p.dw_splits > 1) p.dw_part = p.take(p.dw_splits * p.piece * p.Dp * 4);
    return fits(p.Tp, p.piece, p.grad_tile, 1) && fits(p.piece, h.D, p.dw_tile, p.dw_splits) &&
           fits(p.dx_rows, h.D, p.dx_tile, p.dx_splits);
}

// Lays out `rows` rows of an operand at dst.
CopyArgs copy_of(const Plan &p, const Head &h, const void *src, int64_t ld, int64_t rows, void *dst, int64_t rows_out)
{
    CopyArgs c{};
    c.src = src;
    c.ld = ld;
    c.dtype = h.dtype;
    c.rows = rows;
    c.cols = h.D;
    c.dst = dst;
    c.rows_out = rows_out;
    c.ld_out = p.Dp;
    c.plane = rows_out * p.Dp;
    c.planes = p.planes;
    return c;
}

// The products that the forward pass may leave for the backward pass.
struct Logits {
    float *p = nullptr;
    int64_t ld = 0;
};

struct Labels {
    const int64_t *target = nullptr;
    int64_t ignore = 0;
    const Teacher *teacher = nullptr;
};

// An operand of the head's product as the matrix cores read it.  plane: 0 if
// it is not split, so that its only plane meets both of the logits' gradient.
struct Stored {
    const void *p;
    int64_t ld, plane;
};

tgemm_status_t forward(const Plan &p, const Head &h, const Labels &l, float *loss, float *lse, float *student,
                       const Logits &z, float *summary, void *ws, hipStream_t stream)
{
    hipError_t e = hipSuccess;
    Stored x{h.X, h.ldx, 0}, w{h.W, h.ldw, 0};
    if (p.copy_x) {
        x = Stored{in<void>(ws, p.x), p.Dp, h.T * p.Dp};
        e = launch_copy(copy_of(p, h, h.X, h.ldx, h.T, in<void>(ws, p.x), h.T), stream);
        if (e != hipSuccess) return from_hip(e);
    }
    if (p.copy_w) {
        w = Stored{in<void>(ws, p.w), p.Dp, p.planes > 1 ? h.V * p.Dp : 0};
        e = launch_copy(copy_of(p, h, h.W, h.ldw, h.V, in<void>(ws, p.w), h.V), stream);
        if (e != hipSuccess) return from_hip(e);
    }
    StatsArgs s{};
    s.op = operands(p.segments, h.T, h.V, p.Dp / kStepK, p.stat_tile);
    s.op.A = x.p;
    s.op.lda = x.ld;
    s.op.plane_a = x.plane;
    s.op.mn_a = (int)h.T;
    s.op.B = w.p;
    s.op.ldb = w.ld;
    s.op.plane_b = w.plane;
    s.op.mn_b = (int)h.V;
    s.op.k_b = (int)(p.copy_w ? p.Dp : h.D);
    s.scale = l.teacher ? l.teacher->scale : 1.0f;
    s.part = in<float2>(ws, p.part);
    s.groups = p.groups;
    s.target = l.target;
    s.picked = in<float>(ws, p.picked);
    s.logits = z.p;
    s.ldz = z.ld;
    if (l.teacher != nullptr) {
        const SortArgs k{h.T, h.V, p.groups, p.group_columns, *l.teacher, in<uint16_t>(ws, p.starts),
                         in<uint32_t>(ws, p.list), student};
        e = launch_sort(k, stream);
        if (e != hipSuccess) return from_hip(e);
        s.starts = k.starts;
        s.list = k.list;
        s.K = l.teacher->K;
        s.student = student;
    }
    e = p.few ? launch_stats_few(s, h.dtype, p.group_columns, (int)h.D, stream) : launch_stats(p.half, p.stat_tile, s, stream);
    if (e != hipSuccess) return from_hip(e);
    JoinArgs j{h.T, h.V, p.groups, s.part, l.target, l.ignore, s.picked, l.teacher, student, loss, lse, summary,
               in<int>(ws, p.counted)};
    return from_hip(launch_join(j, stream));
}

tgemm_status_t backward(const Plan &p, const Head &h, const Labels &l, const float *grad, int64_t grad_step,
                        const float *weight, const float *lse, const float *student, const Logits &z, void *dX, int64_t lddx,
                        void *dW, int64_t lddw, void *ws, hipStream_t stream)
{
    // d loss / d (x·w) = grad·(1/τ)·τ² (p - q) for distillation
    const float scale = l.teacher ? l.teacher->scale : 1.0f;
    CoefArgs c{};
    c.T = h.T;
    c.V = h.V;
    c.grad = grad;
    c.grad_step = grad_step;
    c.weight = weight;
    c.factor = 1.0f / scale;
    c.target = l.target;
    c.ignore = l.ignore;
    c.teacher = l.teacher;
    c.half = p.half;
    c.X = h.X;
    c.ldx = h.ldx;
    c.D = h.D;
    c.coef = in<float>(ws, p.coef);
    const bool scaled = p.half || grad_step == 0;
    float *row_scale = scaled ? in<float>(ws, p.row_scale) : nullptr;
    float *all_scale = scaled ? in<float>(ws, p.all_scale) : nullptr;
    c.row_scale = row_scale;
    c.all_scale = all_scale;
    c.exps = in<int>(ws, p.exps);
    c.block_max = in<int>(ws, p.block_max);
    hipError_t e = coef_in_copy(c) ? hipSuccess : launch_coef(c, stream);
    if (e != hipSuccess) return from_hip(e);

    // Rows that do not count may hold anything: they are cleared where they
    // would meet a zero of the logits' gradient.
    void *xs = in<void>(ws, p.xs);
    CopyArgs clear = copy_of(p, h, h.X, h.ldx, h.T, xs, p.Tp);
    if (coef_in_copy(c)) {
        clear.make = &c;
    } else {
        clear.coef = c.coef;
        if (p.half && grad_step != 0) {
            clear.exps = c.exps;
            clear.block_max = c.block_max;
            clear.blocks = (int)coef_blocks(h.T, l.teacher != nullptr);
            clear.all_scale = all_scale;
        }
    }
    e = launch_copy(clear, stream);
    if (e != hipSuccess) return from_hip(e);
    const Stored cleared{xs, p.Dp, p.planes > 1 ? p.Tp * p.Dp : 0};
    Stored x = cleared, w{h.W, h.ldw, 0};
    if (p.half) x = Stored{h.X, h.ldx, 0};
    if (p.copy_x && z.p == nullptr) {
        x = Stored{in<void>(ws, p.x), p.Dp, h.T * p.Dp};
        e = launch_copy(copy_of(p, h, h.X, h.ldx, h.T, in<void>(ws, p.x), h.T), stream);
        if (e != hipSuccess) return from_hip(e);
    }
    if (p.copy_w && (z.p == nullptr || dX != nullptr)) {
        w = Stored{in<void>(ws, p.w), p.Dp, p.planes > 1 ? h.V * p.Dp : 0};
        e = launch_copy(copy_of(p, h, h.W, h.ldw, h.V, in<void>(ws, p.w), h.V), stream);
        if (e != hipSuccess) return from_hip(e);
    }

    void *g = in<void>(ws, p.g);
    const int64_t plane_g = p.Tp * p.ldg;
    for (int64_t n = 0; n < p.pieces; ++n) {
        const int64_t v0 = n * p.piece, cols = h.V - v0 < p.piece ? h.V - v0 : p.piece;
        const int64_t cols_steps = ceil_div(cols, kStepK);
        const char *wn = (const char *)w.p + v0 * w.ld * 2;

        GradArgs a{};
        a.op = operands(p.segments, h.T, cols, p.Dp / kStepK, p.grad_tile);
        a.op.tiles_m = (int)ceil_div(p.Tp, kTiles[p.grad_tile].bm);
        a.op.A = x.p;
        a.op.lda = x.ld;
        a.op.plane_a = x.plane;
        a.op.mn_a = (int)h.T;
        a.op.B = wn;
        a.op.ldb = w.ld;
        a.op.plane_b = w.plane;
        a.op.mn_b = (int)(h.V - v0);
        a.op.k_b = (int)(p.copy_w ? p.Dp : h.D);
        a.scale = scale;
        a.lse = lse;
        a.coef = c.coef;
        a.target = l.target;
        a.v0 = v0;
        a.rows = (int)p.Tp;
        a.G = g;
        a.ldg = p.ldg;
        a.plane = plane_g;
        a.planes = p.g_planes;
        e = z.p ? launch_grad_kept(p.half, a, z.p + v0, z.ld, stream) : launch_grad(p.half, p.grad_tile, a, stream);
        if (e != hipSuccess) return from_hip(e);
        if (l.teacher != nullptr) {
            ScatterArgs s{h.T, v0, cols, *l.teacher, student, lse, c.coef, g, p.ldg, plane_g, p.g_planes, p.half};
            e = launch_scatter(s, stream);
            if (e != hipSuccess) return from_hip(e);
        }
        if (dX != nullptr) {
            OutArgs o{};
            o.op = operands(p.segments, p.dx_rows, h.D, cols_steps, p.dx_tile);
            // the last piece may take fewer parts; the others' sums stand
            o.op.splits = parts_of(cols_steps, p.dx_splits);
            o.op.steps_per_split = (int)ceil_div(cols_steps, o.op.splits);
            o.op.A = g;
            o.op.lda = p.ldg;
            o.op.plane_a = plane_g;
            o.op.mn_a = (int)(p.dx_rows > p.Tp ? p.dx_rows : p.Tp);
            o.op.B = wn;
            o.op.ldb = w.ld;
            o.op.plane_b = w.plane;
            o.op.mn_b = (int)(p.copy_w ? p.Dp : h.D);
            o.op.k_b = (int)(h.V - v0);
            if (p.dx_direct) {
                o.out = dX;
                o.ldo = lddx;
                o.dtype = h.dtype;
                o.row_scale = row_scale;
            } else {
                o.out = in<float>(ws, p.dx_part);
                o.ldo = p.Dp;
                o.dtype = TGEMM_F32;
                o.add = n > 0;
                o.split_stride = p.dx_rows * p.Dp;
                if (p.dx_rows > p.Tp) {  // two planes' rows
                    o.period = (int)p.Tp;
                    o.kept = (int)h.T;
                }
            }
            e = launch_dx(p.half, p.dx_tile, o, stream);
            if (e != hipSuccess) return from_hip(e);
        }
        if (dW != nullptr) {
            OutArgs o{};
            o.op = operands(p.dw_segments, cols, h.D, p.Tp / kStepK, p.dw_tile);
            o.op.A = g;
            o.op.lda = p.ldg;
            o.op.plane_a = plane_g;
            o.op.mn_a = (int)p.piece;
            o.op.k_a = (int)p.Tp;
            o.op.B = cleared.p;
            o.op.ldb = cleared.ld;
            o.op.plane_b = cleared.plane;
            o.op.mn_b = (int)p.Dp;
            o.op.k_b = (int)p.Tp;
            void *to = (char *)dW + v0 * lddw * (int64_t)size_of(h.dtype);
            if (p.dw_splits == 1) {
                o.out = to;
                o.ldo = lddw;
                o.dtype = h.dtype;
                o.all_scale = all_scale;
            } else {
                o.op.splits = p.dw_splits;
                o.op.steps_per_split = (int)ceil_div(p.Tp / kStepK, p.dw_splits);
                o.out = in<float>(ws, p.dw_part);
                o.ldo = p.Dp;
                o.dtype = TGEMM_F32;
                o.split_stride = p.piece * p.Dp;
            }
            e = launch_dw(p.half, p.dw_tile, o, stream);
            if (e != hipSuccess) return from_hip(e);
            if (p.dw_splits > 1) {
                SumArgs s{cols, h.D, in<float>(ws, p.dw_part), p.Dp, o.split_stride, p.dw_splits, nullptr,
                          all_scale, to, lddw, h.dtype};
                e = launch_sum(s, stream);
                if (e != hipSuccess) return from_hip(e);
            }
        }
    }
    if (dX != nullptr && !p.dx_direct) {
        const int planes = p.dx_rows > p.Tp ? 2 : 1;
        SumArgs s{h.T, h.D, in<float>(ws, p.dx_part), p.Dp, p.dx_rows / planes * p.Dp, p.dx_splits * planes, row_scale, nullptr,
                  dX, lddx, h.dtype};
        e = launch_sum(s, stream);
        if (e != hipSuccess) return from_hip(e);
    }
    return TGEMM_SUCCESS;
}

// The kept products' rows.
tgemm_status_t check_kept(const Head &h, const float *logits, int64_t ldz)
{
    if (logits == nullptr) return TGEMM_SUCCESS;
    return ldz < h.V ? TGEMM_ERROR_INVALID_VALUE : ldz > kMaxLd ? TGEMM_ERROR_NOT_SUPPORTED : TGEMM_SUCCESS;
}

tgemm_status_t no_rows(float *summary, hipStream_t stream)
{
    Range r;
    if (!at(summary, summary ? 1 : 0, 3, 3, 4, r)) return TGEMM_ERROR_INVALID_VALUE;
    return summary ? from_hip(launch_summary_none(summary, stream)) : TGEMM_SUCCESS;
}

tgemm_status_t check_teacher(const Head &h, int64_t K, int64_t ld_ids, tgemm_dtype_t dtype, int64_t ld_logits,
                             float temperature)
{
    if (K < 1 || ld_ids < K || ld_logits < K || !(temperature > 0.0f) || __builtin_isinf(temperature) ||
        __builtin_isinf(1.0f / temperature))
        return TGEMM_ERROR_INVALID_VALUE;
    if (!known(dtype) || K > kMaxK || ld_ids > kMaxLd || ld_logits > kMaxLd) return TGEMM_ERROR_NOT_SUPPORTED;
    return TGEMM_SUCCESS;
}

}  // namespace

extern "C" {

size_t tgemm_linear_loss_workspace_size(tgemm_dtype_t dtype, int64_t T, int64_t V, int64_t D, const void *X, int64_t ldx,
                                        const void *W, int64_t ldw, int64_t teacher_k, int backward_pass)
{
    const Head h{dtype, T, V, D, X, ldx, W, ldw};
    if (check_head(h) != TGEMM_SUCCESS || T == 0 || teacher_k < 0 || teacher_k > kMaxK) return 0;
    Plan p;
    if (!(backward_pass ? plan_backward(p, h) : plan_forward(p, h, teacher_k))) return 0;
    return (size_t)p.total;
}

tgemm_status_t tgemm_linear_ce_forward(tgemm_dtype_t dtype, int64_t T, int64_t V, int64_t D, const void *X, int64_t ldx,
                                       const void *W, int64_t ldw, const int64_t *target, int64_t ignore_index,
                                       float *loss, float *lse, float *logits, int64_t ldz, float *summary,
                                       void *workspace, size_t workspace_bytes, hipStream_t stream)
{
    const Head h{dtype, T, V, D, X, ldx, W, ldw};
    tgemm_status_t st = check_head(h);
    if (st == TGEMM_SUCCESS) st = check_kept(h, logits, ldz);
    if (st != TGEMM_SUCCESS) return st;
    if (T == 0) return no_rows(summary, stream);
    Plan p;
    if (!plan_forward(p, h, 0)) return TGEMM_ERROR_NOT_SUPPORTED;
    const Logits z{logits, ldz};
    Range r[3], w[5];
    if (!at(X, T, D, ldx, size_of(dtype), r[0]) || !at(W, V, D, ldw, size_of(dtype), r[1]) ||
        !at(target, T, 1, 1, 8, r[2]) || !at(loss, T, 1, 1, 4, w[0]) || !at(lse, T, 1, 1, 4, w[1]) ||
        !at(summary, summary ? 1 : 0, 3, 3, 4, w[2]) || !room_at(workspace, workspace_bytes, p.total, w[3]) ||
        !at(logits, logits ? T : 0, V, ldz, 4, w[4]) || !disjoint(w, 5, r, 3))
        return TGEMM_ERROR_INVALID_VALUE;
    return forward(p, h, Labels{target, ignore_index, nullptr}, loss, lse, nullptr, z, summary, workspace, stream);
}

tgemm_status_t tgemm_linear_ce_backward(tgemm_dtype_t dtype, int64_t T, int64_t V, int64_t D, const void *X, int64_t ldx,
                                        const void *W, int64_t ldw, const int64_t *target, int64_t ignore_index,
                                        const float *lse, const float *logits, int64_t ldz,
                                        const float *grad_loss, int64_t grad_step, const float *grad_weight,
                                        void *dX, int64_t lddx, void *dW, int64_t lddw,
                                        void *workspace, size_t workspace_bytes, hipStream_t stream)
{
    const Head h{dtype, T, V, D, X, ldx, W, ldw};
    tgemm_status_t st = check_head(h);
    if (st == TGEMM_SUCCESS) st = check_kept(h, logits, ldz);
    if (st != TGEMM_SUCCESS) return st;
    if (grad_step < 0 || (dX != nullptr && lddx < D) || (dW != nullptr && lddw < D)) return TGEMM_ERROR_INVALID_VALUE;
    if (lddx > kMaxLd || lddw > kMaxLd || grad_step > kMaxLd) return TGEMM_ERROR_NOT_SUPPORTED;
    if (dX == nullptr && dW == nullptr) return TGEMM_SUCCESS;
    Plan p;
    if (T > 0 && !plan_backward(p, h)) return TGEMM_ERROR_NOT_SUPPORTED;
    const Logits z{const_cast<float *>(logits), ldz};
    Range r[7], w[3];
    if (!at(X, T, D, ldx, size_of(dtype), r[0]) || !at(W, T == 0 ? 0 : V, D, ldw, size_of(dtype), r[1]) ||
        !at(target, T, 1, 1, 8, r[2]) || !at(lse, T, 1, 1, 4, r[3]) ||
        !at(grad_loss, T, 1, grad_step, 4, r[4]) || !at(grad_weight, T && grad_weight ? 1 : 0, 1, 1, 4, r[5]) ||
        !at(dX, dX ? T : 0, D, lddx, size_of(dtype), w[0]) || !at(dW, dW ? V : 0, D, lddw, size_of(dtype), w[1]) ||
        !room_at(workspace, workspace_bytes, p.total, w[2]) || !at(logits, logits ? T : 0, V, ldz, 4, r[6]) || !disjoint(w, 3, r, 7))
        return TGEMM_ERROR_INVALID_VALUE;
    if (T == 0) return dW ? from_hip(launch_zero(dW, lddw, dtype, V, D, stream)) : TGEMM_SUCCESS;
    return backward(p, h, Labels{target, ignore_index, nullptr}, grad_loss, grad_step, grad_weight, lse, nullptr, z, dX,
                    lddx, dW, lddw, workspace, stream);
}

tgemm_status_t tgemm_linear_kd_forward(tgemm_dtype_t dtype, int64_t T, int64_t V, int64_t D, const void *X, int64_t ldx,
                                       const void *W, int64_t ldw, int64_t K, const int64_t *teacher_ids,
                                       int64_t ld_ids, tgemm_dtype_t teacher_dtype, const void *teacher_logits,
                                       int64_t ld_logits, float temperature, float *loss, float *lse, float *student,
                                       float *logits, int64_t ldz, float *summary, void *workspace,
                                       size_t workspace_bytes, hipStream_t stream)
{
    const Head h{dtype, T, V, D, X, ldx, W, ldw};
    tgemm_status_t st = check_head(h);
    if (st == TGEMM_SUCCESS) st = check_teacher(h, K, ld_ids, teacher_dtype, ld_logits, temperature);
    if (st == TGEMM_SUCCESS) st = check_kept(h, logits, ldz);
    if (st != TGEMM_SUCCESS) return st;
    if (T == 0) return no_rows(summary, stream);
    Plan p;
    if (!plan_forward(p, h, K)) return TGEMM_ERROR_NOT_SUPPORTED;
    const Logits z{logits, ldz};
    Range r[4], w[6];
    if (!at(X, T, D, ldx, size_of(dtype), r[0]) || !at(W, V, D, ldw, size_of(dtype), r[1]) ||
        !at(teacher_ids, T, K, ld_ids, 8, r[2]) || !at(teacher_logits, T, K, ld_logits, size_of(teacher_dtype), r[3]) ||
        !at(loss, T, 1, 1, 4, w[0]) || !at(lse, T, 1, 1, 4, w[1]) || !at(student, T, K, K, 4, w[2]) ||
        !at(summary, summary ? 1 : 0, 3, 3, 4, w[3]) || !room_at(workspace, workspace_bytes, p.total, w[4]) ||
        !at(logits, logits ? T : 0, V, ldz, 4, w[5]) || !disjoint(w, 6, r, 4))
        return TGEMM_ERROR_INVALID_VALUE;
    const Teacher t{(int)K, teacher_ids, ld_ids, teacher_logits, ld_logits, teacher_dtype, 1.0f / temperature};
    return forward(p, h, Labels{nullptr, 0, &t}, loss, lse, student, z, summary, workspace, stream);
}

tgemm_status_t tgemm_linear_kd_backward(tgemm_dtype_t dtype, int64_t T, int64_t V, int64_t D, const void *X, int64_t ldx,
                                        const void *W, int64_t ldw, int64_t K, const int64_t *teacher_ids,
                                        int64_t ld_ids, tgemm_dtype_t teacher_dtype, const void *teacher_logits,
                                        int64_t ld_logits, float temperature, const float *lse, const float *student,
                                        const float *logits, int64_t ldz, const float *grad_loss, int64_t grad_step,
                                        const float *grad_weight, void *dX,
                                        int64_t lddx, void *dW, int64_t lddw,
                                        void *workspace, size_t workspace_bytes, hipStream_t stream)
{
    const Head h{dtype, T, V, D, X, ldx, W, ldw};
    tgemm_status_t st = check_head(h);
    if (st == TGEMM_SUCCESS) st = check_teacher(h, K, ld_ids, teacher_dtype, ld_logits, temperature);
    if (st == TGEMM_SUCCESS) st = check_kept(h, logits, ldz);
    if (st != TGEMM_SUCCESS) return st;
    if (grad_step < 0 || (dX != nullptr && lddx < D) || (dW != nullptr && lddw < D)) return TGEMM_ERROR_INVALID_VALUE;
    if (lddx > kMaxLd || lddw > kMaxLd || grad_step > kMaxLd) return TGEMM_ERROR_NOT_SUPPORTED;
    if (dX == nullptr && dW == nullptr) return TGEMM_SUCCESS;
    Plan p;
    if (T > 0 && !plan_backward(p, h)) return TGEMM_ERROR_NOT_SUPPORTED;
    const Logits z{const_cast<float *>(logits), ldz};
    Range r[9], w[3];
    if (!at(X, T, D, ldx, size_of(dtype), r[0]) || !at(W, T == 0 ? 0 : V, D, ldw, size_of(dtype), r[1]) ||
        !at(teacher_ids, T, K, ld_ids, 8, r[2]) || !at(teacher_logits, T, K, ld_logits, size_of(teacher_dtype), r[3]) ||
        !at(lse, T, 1, 1, 4, r[4]) || !at(student, T, K, K, 4, r[5]) ||
        !at(grad_loss, T, 1, grad_step, 4, r[6]) || !at(grad_weight, T && grad_weight ? 1 : 0, 1, 1, 4, r[7]) ||
        !at(dX, dX ? T : 0, D, lddx, size_of(dtype), w[0]) || !at(dW, dW ? V : 0, D, lddw, size_of(dtype), w[1]) ||
        !room_at(workspace, workspace_bytes, p.total, w[2]) || !at(logits, logits ? T : 0, V, ldz, 4, r[8]) || !disjoint(w, 3, r, 9))
        return TGEMM_ERROR_INVALID_VALUE;
    if (T == 0) return dW ? from_hip(launch_zero(dW, lddw, dtype, V, D, stream)) : TGEMM_SUCCESS;
    const Teacher t{(int)K, teacher_ids, ld_ids, teacher_logits, ld_logits, teacher_dtype, 1.0f / temperature};
    return backward(p, h, Labels{nullptr, 0, &t}, grad_loss, grad_step, grad_weight, lse, student, z, dX,
                    lddx, dW, lddw, workspace, stream);
}

}  // extern "C"
