// How the products of the loss operators and of the adapters are laid out:
// tiles, parts of a sum, operands.
#pragma once

#include <stdint.h>

#include "entry.h"
#include "linear_loss.h"

namespace tgemm {
namespace loss {

using entry::ceil_div;

// A launch has as many work-groups as the GPU holds at most; they count their
// tiles in 32 bits, and a tile's number plus a step of the grid has to fit.
constexpr int64_t kMaxTiles = INT32_MAX - 1024;

// The tile for an M×N product of `steps` steps, and into how many parts its
// sum is split (1 where `split` is false): the least estimated time, in µs.  A
// compute unit holds up to wg_per_cu tiles at once; their step takes as long
// as their area at the rate that the shape sustains (a 256×256 tile 1.5 µs,
// 1.37 PFLOP/s on 256 compute units), but not less than the loads' way there
// and back, and a tile takes 4 µs to begin and to end.  Measured at 32 steps
// with 256, 128 and 32 rows a tile: 512×16384 40, 29 and 58 µs; 64×32000 43,
// 23 and 22; 4096×32768 with 8 steps 127, 162 and 275.
struct Choice {
    int tile = 0, splits = 1;
    double time = 0;
};
inline Choice choose_tile(int64_t M, int64_t N, int64_t steps, bool split = false)
{
    static const double rate[] = {1.0, 0.83, 0.375};
    Choice best;
    double least = -1;
    for (int i = 0; i < kTileCount; ++i) {
        const TileShape &s = kTiles[i];
        const int64_t tiles = ceil_div(M, s.bm) * ceil_div(N, s.bn);
        for (int64_t parts = 1; parts == 1 || (split && parts <= 64 && steps / parts >= 4); ++parts) {
            const int64_t on_one = ceil_div(tiles * parts, 256);
            auto round = [&](int64_t held) {
                const double step = (double)held * s.bm * s.bn / 65536.0 / rate[i] * 1.5;
                return (double)ceil_div(steps, parts) * (step > 0.75 ? step : 0.75) + 4.0;
            };
            double time = (double)(on_one / s.wg_per_cu) * round(s.wg_per_cu);
            if (on_one % s.wg_per_cu != 0) time += round(on_one % s.wg_per_cu);
            // the parts are written and read once more, by another launch
            if (parts > 1) time += 6.0 + (double)M * (double)N * 8.0 * (double)parts / 5e6;
            if (least < 0 || time < least) {
                least = time;
                best.tile = i;
                best.splits = (int)parts;
                best.time = time;
            }
        }
    }
    return best;
}

// The parts of a sum of `steps` steps, at most `most`, none of them empty.
inline int parts_of(int64_t steps, int64_t most) { return (int)ceil_div(steps, ceil_div(steps, most)); }

// False where a product would have too many tiles.
inline bool fits(int64_t M, int64_t N, int tile, int64_t splits)
{
    const TileShape &s = kTiles[tile];
    return ceil_div(M, s.bm) * ceil_div(N, s.bn) <= kMaxTiles / splits;
}

inline m16::Operands operands(int segments, int64_t M, int64_t N, int64_t steps, int tile)
{
    const TileShape &s = kTiles[tile];
    m16::Operands o{};
    o.segments = segments;
    o.M = (int)M;
    o.N = (int)N;
    o.steps = o.steps_per_split = (int)steps;
    o.tiles_m = (int)ceil_div(M, s.bm);
    o.tiles_n = (int)ceil_div(N, s.bn);
    o.splits = 1;
    return o;
}

}  // namespace loss
}  // namespace tgemm
