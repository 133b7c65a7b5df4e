// window_harness.cu -- host program that prints the position tiles of the
// window kernels (window.cuh) for one problem, so that a CPU test can check
// them against the oracle's placement.  Built and run by
// tests/test_window_host.py; no GPU needed.
//
// usage: window_harness LAYOUT S N W
// prints "T t r has row pos" for every row of every tile, "B t row stripe R N"
// (its copy box) and "W t lo hi" for every tile.
#include <stdio.h>
#include <stdlib.h>

#include "window.cuh"

int main(int argc, char **argv) {
    if (argc != 5) return 2;
    striped::PosGeom g;
    if (!striped::pos_geom(&g, atol(argv[2]), atoi(argv[3]), atoi(argv[1]))) return 3;
    for (int t = 0; t < g.nt; ++t) {
        for (int r = 0; r < 128; ++r)
            printf("T %d %d %d %ld %d\n", t, r, (int)striped::tile_has(g, t, r), (long)striped::tile_row(g, t, r),
                   t * g.P + striped::tile_pos(g, r));
        const striped::TileAt a = striped::tile_at(g, t);
        printf("B %d %d %d %d %d %d\n", t, a.row, a.stripe, g.R, g.layout == STRIPED_LAYOUT_STRIPED ? g.N : 1, g.L);
        printf("W %d %d %d\n", t, striped::window_lo(g, t, atoi(argv[4])), striped::window_hi(g, t, atoi(argv[4])));
    }
    return 0;
}
