// window_harness.cu -- host program that prints the position tiles of the
// window kernels (window.cuh) for one problem, so that a CPU test can check
// them against the oracle's placement.  Built and run by
// tests/test_window_host.py; no GPU needed.
//
// usage: window_harness LAYOUT S N W
// prints "T t r has row pos" for every row of every tile, "B t row stripe R N L"
// (its copy box: N stripes inside R rows) and "W t lo hi" for every tile, and
// "K base hi lo sk bits" for ranges of kept columns.
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
                   t * g.P + r);
        const striped::TileAt a = striped::tile_at(g, t);
        const bool st = g.layout == STRIPED_LAYOUT_STRIPED;
        printf("B %d %d %d %d %d %d\n", t, st ? a.c2 : a.c1, st ? a.c1 : a.c2, g.R, st ? g.N : 1, g.L);
        printf("W %d %d %d\n", t, striped::window_lo(g, t, atoi(argv[4])), striped::window_hi(g, t, atoi(argv[4])));
    }
    for (int base = 0; base < 128; base += 32)
        for (int hi = -2; hi < 130; hi += 11)
            for (int lo = -3; lo < 131; lo += 13)
                for (int sk = -1; sk < 129; sk += 10)
                    printf("K %d %d %d %d %u\n", base, hi, lo, sk, striped::kept_bits(base, hi, lo, sk));
    return 0;
}
