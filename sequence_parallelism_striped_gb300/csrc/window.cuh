// window.cuh -- geometry shared by the attention kernels that see a sliding
// window and a few first tokens (sinks): tiles of consecutive POSITIONS.
//
// A window of W positions is one band of the causal triangle in position
// order, but N bands (one per stripe) in striped rows: tiles of 128 rows of
// one stripe would visit N * (W / (128 N) + 2) key tiles instead of
// W / 128 + 2.  All stripes are in one GPU's memory here, so a tile is
// formed from positions instead: a TMA box of {64 columns, R rows, N
// stripes}, R = 128 / N, brings rows d*L + i for R consecutive i and all d,
// which are the P = N * R consecutive positions i*N + d, in one copy of the
// same size.  Row r of such a tile holds position (r % R) * N + r / R of the
// tile.  The zig-zag and contiguous placements hold 128 consecutive
// positions in 128 consecutive rows.
#pragma once

#include <stdint.h>

#include "striped.h"

namespace striped {

// Positions are 32-bit in the kernels (a tile may reach 127 past the last),
// and the sink tiles' gradients are kept as shares: both bounded.
constexpr int64_t kMaxPositions = (1ll << 31) - 256;
constexpr int64_t kMaxSinks = 1024;

struct PosGeom {
    int layout;   // contiguous sequences are carried as one stripe of S rows
    int N;        // stripes
    int L;        // rows of a stripe
    int S;        // positions
    int R, P;     // rows per stripe and positions of a tile
    int nt;       // tiles of the sequence
};

// False if the placement has no position tiles (more than 128 stripes).
static inline bool pos_geom(PosGeom *g, int64_t S, int N, int layout) {
    if (layout == STRIPED_LAYOUT_CONTIGUOUS || N == 1) {
        layout = STRIPED_LAYOUT_STRIPED;
        N = 1;
    }
    g->layout = layout;
    g->N = N;
    g->S = (int)S;
    g->L = (int)(S / N);
    if (layout == STRIPED_LAYOUT_STRIPED) {
        if (N > 128) return false;
        g->R = 128 / N;
        g->P = g->R * N;
    } else {
        g->R = g->P = 128;
    }
    g->nt = (int)((S + g->P - 1) / g->P);
    return true;
}

// Tensor-map coordinates of position tile t: first row inside a stripe's
// slice and (first) stripe.  Zig-zag chunks are whole tiles.
struct TileAt {
    int row, stripe;
};
__host__ __device__ __forceinline__ TileAt tile_at(const PosGeom &g, int t) {
    if (g.layout == STRIPED_LAYOUT_STRIPED) return TileAt{t * g.R, 0};
    const int per = g.L / 256;  // tiles of a chunk
    const int c = t / per, in = (t - c * per) * 128;
    return c < g.N ? TileAt{in, c} : TileAt{g.L / 2 + in, 2 * g.N - 1 - c};
}

// Position (inside the tile) of row r, and the row of the [S] tensors that
// holds row r of tile t.
__host__ __device__ __forceinline__ int tile_pos(const PosGeom &g, int r) {
    return (r % g.R) * g.N * (g.layout == STRIPED_LAYOUT_STRIPED) + (g.layout == STRIPED_LAYOUT_STRIPED ? r / g.R : r);
}
__host__ __device__ __forceinline__ int64_t tile_row(const PosGeom &g, int t, int r) {
    const TileAt a = tile_at(g, t);
    if (g.layout == STRIPED_LAYOUT_STRIPED) return (int64_t)(r / g.R) * g.L + a.row + r % g.R;
    return (int64_t)a.stripe * g.L + a.row + r;
}
// Row r of tile t holds a position of the sequence.
__host__ __device__ __forceinline__ bool tile_has(const PosGeom &g, int t, int r) {
    return r < g.P && t * (int64_t)g.P + tile_pos(g, r) < g.S;
}

// Lowest key tile inside the window of query tile t, and highest query tile
// whose window reaches key tile t.
__host__ __device__ __forceinline__ int window_lo(const PosGeom &g, int t, int W) {
    const int64_t first = (int64_t)t * g.P - W + 1;
    return first <= 0 ? 0 : (int)(first / g.P);
}
__host__ __device__ __forceinline__ int window_hi(const PosGeom &g, int t, int W) {
    const int64_t last = ((int64_t)t * g.P + g.P - 1 + W - 1) / g.P;
    return last < g.nt ? (int)last : g.nt - 1;
}

}  // namespace striped
