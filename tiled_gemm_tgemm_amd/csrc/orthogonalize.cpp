// C entry points of the Newton-Schulz operator: argument checks, the plan of a
// call and its launches on the caller's stream.  The declarations, with the
// meaning of every argument, are in tgemm.h.
#include "entry.h"
#include "orthogonalize.h"

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace {

using namespace tgemm::entry;
using namespace tgemm::ortho;
using tgemm::m16::kStepK;

constexpr int64_t kMaxSide = (int64_t)1 << 20;   // a tile's offsets fit 32 bits
constexpr int64_t kMaxBatch = 65535;             // a launch's y
constexpr int64_t kMaxLd = (int64_t)1 << 40;
constexpr int64_t kMaxTiles = INT32_MAX - 1024;
constexpr float kMostFolded = 16.0f;             // a larger a stays out of Q's planes, which hold up to 64

struct Stack {
    tgemm_dtype_t dtype;
    int64_t batch, M, N;
    int steps;
};

// Every product takes three of planes, in every step and for every type.  A
// bf16 result's own rounding is 1.7e-3 (norms over norm), but one plane left out
// anywhere can show beside it: values that are alike are rounded alike, and what
// that changes in a dominant direction the polynomial makes several times as
// large.  Of the rounding's error, the roundings followed on the host: with one
// plane for S alone, from the third step on, 256×1024 of one large value a row
// 2.7 times and an orthogonal 384×384 1.4; with one in the first two steps 1 +
// 0.001·normal values of 384×384 1.4 to 3.9, by the coefficients, and 70×300 of
// rank 1 with noise of a thousandth up to 340; with three 1.0 in all of these.
// Two of the three cost bf16 8192×8192 26.8 ms instead of 17.2, 8×1024×4096 2.05
// instead of 1.40 and 256×1024 0.20 instead of 0.16.
constexpr int kSegments = 3;

// The tile for `batch` M×N products of `steps` steps (of kSegments each), whether
// only the tiles on and below the diagonal are formed, and into how many
// parts the sums of the tiles are split that do not fill the GPU a last time:
// the least estimated time, in µs.
//
// A compute unit that holds 1 ... 4 tiles takes kStep for a step of all of them
// and kBegin for what comes before and after, most of which is the planes' way;
// across the diagonal a tile's takes kAcross more.  The whole GPU multiplies no
// more than 1.3 PFLOP/s, and runs the faster the less of it is at work (a tenth
// of the time at that rate is added).  Parts are written and read once more, by another
// launch.  Measured (µs; tiles of 256, 128 and 64): S and Q of 256×1024 with 16
// and 12 steps 31 and 33, 16 and 16, 11 and 10; Q of 2048×2048, 96 steps, 135,
// 66 and 56; of 4096×4096, 192 steps, 268 below the diagonal and 341, 288 and
// 406; S of 3000×1000, 141 steps, 128 and below the diagonal 91, in 7 parts 34.
struct Choice {
    int tile = -1;
    bool lower = false;
    int whole = 0, rest = 0, splits = 1;  // tiles in whole sums, and those in parts
};
constexpr double kStep[kTileCount][4] = {{1.2}, {0.57, 0.95}, {0.33, 0.45, 0.62, 0.8}};
constexpr double kBegin[kTileCount] = {22.0, 10.0, 6.5}, kBeginPart[kTileCount] = {15.0, 8.0, 5.0}, kAcross[kTileCount] = {8.0, 1.5, 0.7};
Choice choose(int64_t M, int64_t N, int64_t steps, int64_t batch, bool symmetric)
{
    Choice best;
    double least = -1;
    for (int i = 0; i < kTileCount; ++i) {
        const TileShape &s = kTiles[i];
        const int64_t m = ceil_div(M, s.side), n = ceil_div(N, s.side);
        for (int lower = 0; lower <= (symmetric ? 1 : 0); ++lower) {
            if (m * n > kMaxTiles / batch / 64) continue;
            const int64_t tiles = (lower ? m * (m + 1) / 2 : m * n) * batch, most = (int64_t)256 * s.wg_per_cu;
            auto rounds = [&](int64_t tiles, int64_t steps, double begin) {
                const int64_t on_one = ceil_div(tiles, 256), rest = on_one % s.wg_per_cu;
                auto round = [&](int64_t held) { return (double)(steps * kSegments) * kStep[i][held - 1] + begin; };
                const double time = (double)(on_one / s.wg_per_cu) * round(s.wg_per_cu) + (rest ? round(rest) : 0.0);
                const double area = (double)(tiles * s.side) * s.side;
                const double power = area * (double)(steps * kSegments * kStepK) * 2.0 / 1.3e9 + begin;
                return tiles == 0 ? 0.0 : (time > power ? time : power) + 0.1 * power;
            };
            for (int64_t whole : {tiles, tiles / most * most}) {
                const int64_t rest = tiles - whole;
                for (int64_t parts = rest ? 2 : 1; parts == 1 || (parts <= 32 && parts <= steps); ++parts) {
                    double time = rounds(whole, steps, kBegin[i] + (lower ? kAcross[i] : 0.0));
                    if (rest)
                        time += rounds(rest * parts, ceil_div(steps, parts), kBeginPart[i]) + (whole ? 9.0 : 6.0) +
                                (double)(rest * parts * s.side * s.side) * 8.0 / 4e6;
                    if (least < 0 || time < least) {
                        least = time;
                        best.tile = i;
                        best.lower = lower != 0;
                        best.whole = (int)whole;
                        best.rest = (int)rest;
                        best.splits = (int)ceil_div(steps, ceil_div(steps, parts));
                    }
                    if (rest == 0) break;
                }
            }
        }
    }
    return best;
}

// Where a call's buffers lie in its workspace, and the sizes of its matrices.
struct Plan {
    bool small = false, tall = false;
    int64_t side = 0, length = 0;              // the smaller and the larger of M and N
    int64_t side_p = 0, length_p = 0;          // in whole steps of K
    int64_t total = 0;
    // the chain
    int parts = 0;
    int64_t x_rows = 0, x_ld = 0;
    int64_t squares = -1, x[2] = {-1, -1}, s = -1, q = -1, parts_room = -1;
    Choice product_s, product_q, product_x;  // of every step
    // the small side's
    int64_t part_length = 0, grams = -1, factor = -1;

    int64_t take(int64_t bytes)
    {
        const int64_t at = total;
        total += round_up(bytes, 256);
        return at;
    }
};

int64_t parts_bytes(const Choice &c) { return (int64_t)c.rest * c.splits * kTiles[c.tile].side * kTiles[c.tile].side * 4; }

bool make_plan(Plan &p, const Stack &g)
{
    p.tall = g.M > g.N;
    p.side = p.tall ? g.N : g.M;
    p.length = p.tall ? g.M : g.N;
    p.side_p = round_up(p.side, kStepK);
    p.length_p = round_up(p.length, kStepK);
    p.small = p.side <= kSmallSide;
    if (p.small) {
        const int64_t blocks = blocks_of((int)p.side), most = 16;
        p.part_length = round_up(ceil_div(p.length, most), 128);
        if (p.part_length < 256) p.part_length = 256;
        p.parts = (int)ceil_div(p.length, p.part_length);
        p.grams = p.take(g.batch * p.parts * (blocks * (blocks + 1) / 2) * 256 * 8);
        p.factor = p.take(g.batch * 256 * blocks * blocks * 8);
        return true;
    }
    const int64_t pieces = g.M * ceil_div(g.N, 8);
    p.parts = (int)(pieces / 1024 + 1 < kMaxSquares ? pieces / 1024 + 1 : kMaxSquares);
    // S = Xᵀ·X of a tall X sums over its rows, in whole steps
    p.x_rows = p.tall ? p.length_p : p.side;
    p.x_ld = p.tall ? p.side_p : p.length_p;
    p.squares = p.take(g.batch * p.parts * 8);
    const int64_t x = g.batch * 2 * p.x_rows * p.x_ld * 2, s = g.batch * 2 * p.side * p.side_p * 2;
    p.x[0] = p.take(x);
    if (g.steps > 1) p.x[1] = p.take(x);
    p.s = p.take(s);
    p.q = p.take(s);
    p.product_s = choose(p.side, p.side, p.length_p / kStepK, g.batch, true);
    p.product_q = choose(p.side, p.side, p.side_p / kStepK, g.batch, true);
    p.product_x = choose(g.M, g.N, p.side_p / kStepK, g.batch, false);
    int64_t room = 0;
    for (const Choice *one : {&p.product_s, &p.product_q, &p.product_x}) {
        if (one->tile < 0) return false;
        if (parts_bytes(*one) > room) room = parts_bytes(*one);
    }
    p.parts_room = p.take(room);
    return true;
}

tgemm_status_t check(const Stack &g, float eps)
{
    if (g.batch < 0 || g.M < 0 || g.N < 0 || g.steps < 1 || !(eps >= 0.0f) || __builtin_isinf(eps))
        return TGEMM_ERROR_INVALID_VALUE;
    if (!known(g.dtype) || g.batch > kMaxBatch || g.M > kMaxSide || g.N > kMaxSide || g.steps > kMaxSteps)
        return TGEMM_ERROR_NOT_SUPPORTED;
    return TGEMM_SUCCESS;
}

Chain product(int64_t M, int64_t N, int64_t steps, const Choice &c)
{
    Chain o{};
    o.segments = kSegments;
    o.M = (int)M;
    o.N = (int)N;
    o.steps = (int)steps;
    o.tiles_m = (int)ceil_div(M, kTiles[c.tile].side);
    o.tiles_n = (int)ceil_div(N, kTiles[c.tile].side);
    o.lower = c.lower;
    return o;
}

// The tiles with whole sums, then those in parts.
hipError_t run(Order order, const Choice &c, ChainArgs a, hipStream_t stream)
{
    hipError_t e = hipSuccess;
    if (c.whole > 0) {
        a.op.count = c.whole;
        a.op.splits = 1;
        a.op.steps_per_split = a.op.steps;
        e = launch_chain(order, c.tile, a, stream);
    }
    if (e != hipSuccess || c.rest == 0) return e;
    a.op.from = c.whole;
    a.op.count = c.rest;
    a.op.splits = c.splits;
    a.op.steps_per_split = (int)ceil_div(a.op.steps, c.splits);
    e = launch_chain(order, c.tile, a, stream);
    return e != hipSuccess ? e : launch_join(c.tile, a, stream);
}

tgemm_status_t run_small(const Plan &p, const Stack &g, const void *G, int64_t ldg, int64_t batch_g, const float *coefficients,
                         float eps, void *out, int64_t ldo, int64_t batch_o, void *ws, hipStream_t stream)
{
    SmallArgs a{};
    a.G = G;
    a.ld = ldg;
    a.batch_g = batch_g;
    a.dtype = g.dtype;
    a.batch = (int)g.batch;
    a.side = (int)p.side;
    a.length = p.length;
    a.tall = p.tall;
    a.grams = in<double>(ws, p.grams);
    a.part_length = p.part_length;
    a.parts = p.parts;
    a.steps = g.steps;
    for (int n = 0; n < 3 * g.steps; ++n) a.coefficients[n] = coefficients[n];
    a.eps = eps;
    a.factor = in<double>(ws, p.factor);
    a.out = out;
    a.ldo = ldo;
    a.batch_o = batch_o;
    hipError_t e = launch_grams(a, stream);
    if (e == hipSuccess) e = launch_iterate(a, stream);
    if (e == hipSuccess) e = launch_apply(a, stream);
    return from_hip(e);
}

tgemm_status_t run_chain(const Plan &p, const Stack &g, const void *G, int64_t ldg, int64_t batch_g, const float *coefficients,
                         float eps, void *out, int64_t ldo, int64_t batch_o, void *ws, hipStream_t stream)
{
    const int64_t x_plane = p.x_rows * p.x_ld, s_plane = p.side * p.side_p;
    SplitArgs c{};
    c.G = G;
    c.ld = ldg;
    c.batch_g = batch_g;
    c.dtype = g.dtype;
    c.batch = (int)g.batch;
    c.rows = g.M;
    c.cols = g.N;
    c.squares = in<double>(ws, p.squares);
    c.parts = p.parts;
    c.eps = eps;
    c.planes = in<void>(ws, p.x[0]);
    c.rows_out = p.x_rows;
    c.ldo = p.x_ld;
    c.plane = x_plane;
    c.batch_out = 2 * x_plane;
    hipError_t e = launch_squares(c, stream);
    if (e == hipSuccess) e = launch_split(c, stream);
    if (e != hipSuccess) return from_hip(e);

    const float one = 1.0f / (1 << kShift);
    void *s = in<void>(ws, p.s), *q = in<void>(ws, p.q);
    for (int step = 0; step < g.steps; ++step) {
        const float *k = coefficients + 3 * step;
        void *x = in<void>(ws, p.x[step & 1]);

        const int64_t s_steps = p.length_p / kStepK, q_steps = p.side_p / kStepK;
        ChainArgs a{};
        a.parts = in<float>(ws, p.parts_room);
        a.op = product(p.side, p.side, s_steps, p.product_s);
        a.op.A = a.op.B = x;
        a.op.lda = a.op.ldb = p.x_ld;
        a.op.plane_a = a.op.plane_b = x_plane;
        a.op.batch_a = a.op.batch_b = 2 * x_plane;
        a.op.mn_a = a.op.mn_b = (int)(p.tall ? p.x_ld : p.side);
        a.op.k_a = a.op.k_b = (int)p.length_p;
        a.beta = one;
        a.planes = s;
        a.ldo = p.side_p;
        a.plane_out = s_plane;
        a.batch_out = 2 * s_plane;
        a.rows = (int)p.side;
        e = run(p.tall ? kColumns : kRows, p.product_s, a, stream);
        if (e != hipSuccess) return from_hip(e);

        a.op = product(p.side, p.side, q_steps, p.product_q);
        a.op.A = a.op.B = s;
        a.op.lda = a.op.ldb = p.side_p;
        a.op.plane_a = a.op.plane_b = s_plane;
        a.op.batch_a = a.op.batch_b = 2 * s_plane;
        a.op.mn_a = a.op.mn_b = (int)p.side;
        a.op.k_a = a.op.k_b = (int)p.side_p;
        a.add = s;
        a.ld_add = p.side_p;
        a.plane_add = s_plane;
        a.batch_add = 2 * s_plane;
        a.alpha = k[1];
        a.beta = k[2] * one;
        // Q's planes hold as much of a·X as X's do, while a is no more than what else they hold
        const bool folded = k[0] >= -kMostFolded && k[0] <= kMostFolded;
        a.diagonal = folded ? k[0] * (1 << kShift) : 0.0f;
        a.planes = q;
        e = run(kRows, p.product_q, a, stream);
        if (e != hipSuccess) return from_hip(e);

        a.op = product(g.M, g.N, q_steps, p.product_x);
        a.op.A = p.tall ? x : q;
        a.op.lda = p.tall ? p.x_ld : p.side_p;
        a.op.plane_a = p.tall ? x_plane : s_plane;
        a.op.batch_a = 2 * a.op.plane_a;
        a.op.mn_a = (int)g.M;
        a.op.k_a = (int)p.side_p;
        a.op.B = p.tall ? q : x;
        a.op.ldb = p.tall ? p.side_p : p.x_ld;
        a.op.plane_b = p.tall ? s_plane : x_plane;
        a.op.batch_b = 2 * a.op.plane_b;
        a.op.mn_b = (int)(p.tall ? p.side : p.x_ld);
        a.op.k_b = (int)(p.tall ? p.side_p : p.side);
        a.diagonal = 0.0f;
        a.add = folded ? nullptr : x;
        a.ld_add = p.x_ld;
        a.plane_add = x_plane;
        a.batch_add = 2 * x_plane;
        a.alpha = k[0];
        a.beta = one;
        if (step + 1 < g.steps) {
            a.planes = in<void>(ws, p.x[(step + 1) & 1]);
            a.ldo = p.x_ld;
            a.plane_out = x_plane;
            a.batch_out = 2 * x_plane;
            a.rows = (int)p.x_rows;
        } else {
            a.planes = nullptr;
            a.result = out;
            a.ldr = ldo;
            a.batch_r = batch_o;
            a.dtype = g.dtype;
        }
        e = run(p.tall ? kRows : kMixed, p.product_x, a, stream);
        if (e != hipSuccess) return from_hip(e);
    }
    return TGEMM_SUCCESS;
}

}  // namespace

extern "C" {

size_t tgemm_orthogonalize_workspace_size(tgemm_dtype_t dtype, int64_t batch, int64_t M, int64_t N, int steps)
{
    const Stack g{dtype, batch, M, N, steps};
    Plan p;
    if (check(g, 0.0f) != TGEMM_SUCCESS || batch == 0 || M == 0 || N == 0 || !make_plan(p, g)) return 0;
    return (size_t)p.total;
}

tgemm_status_t tgemm_orthogonalize(tgemm_dtype_t dtype, int64_t batch, int64_t M, int64_t N,
                                   const void *G, int64_t ldg, int64_t stride_g,
                                   int steps, const float *coefficients, float eps,
                                   void *out, int64_t ldo, int64_t stride_out,
                                   void *workspace, size_t workspace_bytes, hipStream_t stream)
{
    const Stack g{dtype, batch, M, N, steps};
    const tgemm_status_t st = check(g, eps);
    if (st != TGEMM_SUCCESS) return st;
    if (coefficients == nullptr || ldg < N || ldo < N || stride_g < 0 || stride_out < 0) return TGEMM_ERROR_INVALID_VALUE;
    if (ldg > kMaxLd || ldo > kMaxLd || stride_g > kMaxLd || stride_out > kMaxLd) return TGEMM_ERROR_NOT_SUPPORTED;
    if (batch == 0 || M == 0 || N == 0) return TGEMM_SUCCESS;
    Plan p;
    if (!make_plan(p, g)) return TGEMM_ERROR_NOT_SUPPORTED;
    // a matrix's elements, from its first to its last
    const int64_t span_g = (M - 1) * ldg + N, span_out = (M - 1) * ldo + N;
    Range r[1], w[2];
    if (!separate(batch, M, N, ldo, stride_out) || !at(G, batch, span_g, stride_g, size_of(dtype), r[0]) ||
        !at(out, batch, span_out, stride_out, size_of(dtype), w[0]) || !room_at(workspace, workspace_bytes, p.total, w[1]) ||
        !disjoint(w, 2, r, 1))
        return TGEMM_ERROR_INVALID_VALUE;
    return (p.small ? run_small : run_chain)(p, g, G, ldg, stride_g, coefficients, eps, out, ldo, stride_out, workspace, stream);
}

}  // extern "C"
