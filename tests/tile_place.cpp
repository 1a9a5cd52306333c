// The tiles that numbers stand for (tile_walk.h), at tile counts up to the
// largest that the entry points take.  Reads rows and columns of tiles and the
// parts of the sum, one product a line; built to end at an overflow.
#include <cstdio>
#include <cstdlib>
#include <set>
#include <tuple>

#include "tile_walk.h"

int main()
{
    int tiles_m, tiles_n, splits, products = 0;
    while (std::scanf("%d %d %d", &tiles_m, &tiles_n, &splits) == 3) {
        const int tiles = tiles_m * tiles_n * splits;
        for (int grid : {256, 768}) {
            std::set<std::tuple<int, int, int>> seen;
            std::set<int> ids;
            const int far = tiles / 7 + 1;
            for (int k = 0; k < 8; ++k) {
                const int at = k < 7 ? k * far : tiles - 1;
                for (int id = at < 2000 ? 0 : at - 2000; id < tiles && id <= at; ++id) {
                    int tm, tn, split;
                    tgemm::m16::place_tile(id, tiles, tiles_m, tiles_n, tm, tn, split);
                    if (tm < 0 || tm >= tiles_m || tn < 0 || tn >= tiles_n || split < 0 || split >= splits) return 1;
                    ids.insert(id), seen.emplace(tm, tn, split);
                }
                if (ids.size() != seen.size()) return 2;  // two numbers, two tiles
            }
            // a work-group's way past its last tile
            tgemm::m16::Operands p{};
            p.segments = p.steps = p.steps_per_split = 1;
            p.tiles_m = tiles_m, p.tiles_n = tiles_n, p.splits = splits;
            p.mn_a = p.mn_b = p.k_a = p.k_b = 64;
            tgemm::m16::Walk<256, 256, false, false> w;
            w.begin(p, tiles - 1);
            for (int n = 0; n < 4; ++n) w.seek(p, grid);
            if (w.id != tiles - 1) return 3;
        }
        ++products;
    }
    std::printf("%d products\n", products);
    return 0;
}
