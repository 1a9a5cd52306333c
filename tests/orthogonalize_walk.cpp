// Follows every address of the Newton-Schulz operator on the host: the
// library's own entry point (orthogonalize.cpp) with launches that run the
// loads' walk (tile_walk.h) for each thread, or the extents that a pass over
// rows touches, instead of a kernel.  Reads calls from stdin, one a line:
//   dtype batch M N steps ldg stride_g shift_g ldo stride_o
// and ends with 1 at the first access that leaves what the call was given, or
// where the products' tiles do not cover their results once.
#include <algorithm>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <vector>

#include "orthogonalize.h"

namespace {

struct Range {
    uintptr_t lo, hi;
    bool written;
    const char *name;
};
std::vector<Range> ranges;
long loads = 0;
int64_t matrices = 0;  // of the call
char line[256];

void fail(const char *what, uintptr_t a, size_t n)
{
    std::printf("%s of %zu bytes at %#zx fails in: %s", what, n, (size_t)a, line);
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

void span(const void *p, int64_t batch, int64_t stride, int64_t rows, int64_t cols, int64_t ld, size_t size, bool write, const char *what)
{
    if (rows == 0 || cols == 0) return;
    for (int64_t b : {(int64_t)0, batch - 1}) {
        touch((const char *)p + b * stride * (int64_t)size, cols * size, write, what);
        touch((const char *)p + (b * stride + (rows - 1) * ld) * (int64_t)size, cols * size, write, what);
    }
}

size_t size_of(tgemm_dtype_t t) { return t == TGEMM_F32 ? 4 : 2; }

using tgemm::ortho::Chain;
using tgemm::m16::Slice;

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
void walk(const Chain &p, int wg_per_cu)
{
    typedef Slice<BM, BM / WM / 16, 64 * WM * WN, A_MC, false> A;
    typedef Slice<BN, BN / WN / 16, 64 * WM * WN, B_MC, true> B;
    const int tiles = p.ids(), grid = std::min(tiles, 256 * wg_per_cu);
    if (tiles <= 4096) {  // every part of every tile of the launch once
        std::vector<int> seen((size_t)tiles, 0), where((size_t)p.tiles_m * p.tiles_n, -1);
        for (int id = 0; id < tiles; ++id) {
            int m0, n0, split, first, last;
            p.tile<BM, BN>(id, m0, n0, split, first, last);
            const int at = split - p.from * p.splits;
            if (m0 % BM || n0 % BN || m0 / BM >= p.tiles_m || n0 / BN >= p.tiles_n || m0 < 0 || n0 < 0 || at < 0 || at >= tiles)
                fail("a tile outside", 0, 0);
            if (first >= last || first != split % p.splits * p.steps_per_split) fail("a tile's steps", 0, 0);
            if (p.lower && n0 > m0) fail("a tile above the diagonal", 0, 0);
            ++seen[at];
            // numbers and places of a matrix's tiles go together
            int &place = where[(size_t)(m0 / BM) * p.tiles_n + n0 / BN];
            const int number = split / p.splits % p.tiles();
            if (place >= 0 && place != number) fail("a tile in two places", 0, 0);
            place = number;
        }
        for (int n : seen)
            if (n != 1) fail("a tile that is not taken once", 0, n);
        std::vector<int> numbers;
        for (int n : where)
            if (n >= 0) numbers.push_back(n);
        std::sort(numbers.begin(), numbers.end());
        for (size_t n = 1; n < numbers.size(); ++n)
            if (numbers[n] == numbers[n - 1]) fail("two tiles in a place", 0, 0);
    }
    for (int group : {0, 1, 7, 8, grid / 2, grid - 9, grid - 2, grid - 1}) {
        if (group < 0 || group >= grid) continue;
        int steps = 2;
        for (int id = group; id < tiles; id += grid) {
            int m0, n0, split, first, last;
            p.tile<BM, BN>(id, m0, n0, split, first, last);
            steps += (last - first) * p.segments;
        }
        tgemm::m16::Walk<BM, BN, A_MC, B_MC, Chain> w;
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

}  // namespace

namespace tgemm {
namespace ortho {

int64_t covered = 0;  // tiles of the product that is being launched
void check_rest(const ChainArgs &a, int64_t batch)
{
    if (a.add)
        for (int q = 0; q < 2; ++q)
            span((const char *)a.add + q * a.plane_add * 2, batch, a.batch_add, a.op.M, a.ld_add, a.ld_add, 2, false, "add");
    if (a.planes) {
        for (int q = 0; q < 2; ++q)
            span((char *)a.planes + q * a.plane_out * 2, batch, a.batch_out, a.rows, a.ldo, a.ldo, 2, true, "planes");
        if (a.planes == a.op.A || a.planes == a.op.B || a.planes == a.add) fail("planes in place", 0, 0);
    } else {
        span(a.result, batch, a.batch_r, a.op.M, a.op.N, a.ldr, size_of(a.dtype), true, "result");
    }
}
hipError_t launch_chain(Order order, int tile, const ChainArgs &a, hipStream_t)
{
    if (a.op.lower && (a.op.tiles_m != a.op.tiles_n || a.op.M != a.op.N)) fail("a triangle that is not square", 0, 0);
    const int64_t batch = (a.op.from + a.op.count - 1) / a.op.tiles() + 1;
    if (a.op.from != covered) fail("tiles that were left out", 0, covered);
    covered = a.op.from + a.op.count;
    if (a.op.splits > 1 || covered == (int64_t)a.op.tiles() * matrices) {
        if (covered != (int64_t)a.op.tiles() * matrices) fail("tiles that were left out", 0, covered);
        covered = 0;
    }
    switch (tile) {
#define X(I, BM, BN, WM, WN)                                                                                      \
    case I:                                                                                                       \
        if ((int64_t)a.op.tiles_m * BM < a.op.M || (int64_t)a.op.tiles_n * BN < a.op.N) fail("tiles", 0, 0);      \
        if (a.planes && (int64_t)a.op.tiles_n * BN < a.ldo) fail("columns that no tile clears", 0, 0);            \
        if (a.planes && !a.op.lower && (int64_t)a.op.tiles_m * BM < a.rows) fail("rows that no tile clears", 0, 0); \
        if (order == kRows) walk<BM, BN, WM, WN, false, false>(a.op, kTiles[I].wg_per_cu);                        \
        else if (order == kColumns) walk<BM, BN, WM, WN, true, true>(a.op, kTiles[I].wg_per_cu);                  \
        else walk<BM, BN, WM, WN, false, true>(a.op, kTiles[I].wg_per_cu);                                        \
        if (a.op.splits > 1) touch(a.parts, (size_t)a.op.count * a.op.splits * BM * BN * 4, true, "parts");       \
        break;
        TGEMM_CHAIN_TILES(X)
#undef X
    default:
        fail("an unknown tile", 0, 0);
    }
    if (a.op.splits == 1) check_rest(a, batch);
    return hipSuccess;
}
hipError_t launch_join(int, const ChainArgs &a, hipStream_t)
{
    if (a.op.splits < 2) fail("a join of nothing", 0, 0);
    check_rest(a, (a.op.from + a.op.count - 1) / a.op.tiles() + 1);
    return hipSuccess;
}

hipError_t launch_squares(const SplitArgs &a, hipStream_t)
{
    span(a.G, a.batch, a.batch_g, a.rows, a.cols, a.ld, size_of(a.dtype), false, "G");
    span(a.squares, 1, 0, a.batch, a.parts, a.parts, 8, true, "squares");
    return hipSuccess;
}

hipError_t launch_split(const SplitArgs &a, hipStream_t)
{
    if (launch_squares(a, nullptr) != hipSuccess) return hipErrorUnknown;
    if (a.rows_out < a.rows || a.ldo < a.cols || a.ldo % 64) fail("planes' sizes", 0, 0);
    for (int q = 0; q < 2; ++q)
        span((char *)a.planes + q * a.plane * 2, a.batch, a.batch_out, a.rows_out, a.ldo, a.ldo, 2, true, "planes");
    return hipSuccess;
}

hipError_t launch_grams(const SmallArgs &a, hipStream_t)
{
    const int64_t rows = a.tall ? a.length : a.side, cols = a.tall ? a.side : a.length, b = blocks_of(a.side);
    if (a.side > 16 * b || (int64_t)a.parts * a.part_length < a.length || (int64_t)(a.parts - 1) * a.part_length >= a.length) fail("parts", 0, 0);
    span(a.G, a.batch, a.batch_g, rows, cols, a.ld, size_of(a.dtype), false, "G");
    span(a.grams, a.batch, a.parts * b * (b + 1) / 2 * 256, a.parts, b * (b + 1) / 2 * 256, b * (b + 1) / 2 * 256, 8, true, "grams");
    return hipSuccess;
}

hipError_t launch_iterate(const SmallArgs &a, hipStream_t)
{
    const int64_t b = blocks_of(a.side);
    span(a.factor, a.batch, 256 * b * b, 16 * b, 16 * b, 16 * b, 8, true, "factor");
    return hipSuccess;
}

hipError_t launch_apply(const SmallArgs &a, hipStream_t)
{
    const int64_t rows = a.tall ? a.length : a.side, cols = a.tall ? a.side : a.length;
    span(a.out, a.batch, a.batch_o, rows, cols, a.ldo, size_of(a.dtype), true, "out");
    return hipSuccess;
}

}  // namespace ortho
}  // namespace tgemm

int main()
{
    long calls = 0;
    while (std::fgets(line, sizeof line, stdin)) {
        int dtype, steps;
        long long batch, M, N, ldg, sg, shift, ldo, so;
        if (std::sscanf(line, "%d %lld %lld %lld %d %lld %lld %lld %lld %lld", &dtype, &batch, &M, &N, &steps, &ldg, &sg, &shift, &ldo, &so) != 10) return 2;
        const tgemm_dtype_t t = (tgemm_dtype_t)dtype;
        const size_t size = size_of(t);
        matrices = batch;
        const uintptr_t G = 0x100000000000ull + shift * size, O = 0x300000000000ull, W = 0x500000000000ull;
        const size_t ws = tgemm_orthogonalize_workspace_size(t, batch, M, N, steps);
        ranges = {{G, G + ((batch - 1) * sg + (M - 1) * ldg + N) * size, false, "G"},
                  {O, O + ((batch - 1) * so + (M - 1) * ldo + N) * size, true, "out"},
                  {W, W + ws, true, "workspace"}};
        std::vector<float> c(3 * steps, 1.0f);
        const tgemm_status_t st = tgemm_orthogonalize(t, batch, M, N, (void *)G, ldg, sg, steps, c.data(), 1e-7f, (void *)O, ldo, so,
                                                      (void *)W, ws, nullptr);
        if (st != TGEMM_SUCCESS) fail("the call", 0, st);
        ++calls;
    }
    std::printf("%ld calls, %ld loads\n", calls, loads);
    return 0;
}
