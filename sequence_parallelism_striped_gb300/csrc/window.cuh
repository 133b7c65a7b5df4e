// window.cuh -- geometry shared by the attention kernels that see a sliding
// window and a few first tokens (sinks): tiles of consecutive POSITIONS.
//
// A window of W positions is one band of the causal triangle in position
// order, but N bands (one per stripe) in striped rows: tiles of 128 rows of
// one stripe would visit N * (W / (128 N) + 2) key tiles instead of
// W / 128 + 2.  All stripes are in one GPU's memory here, so a tile is
// formed from positions instead: the tensor map puts the stripe dimension
// inside the row dimension, and a box of {64 columns, N stripes, R rows}, R =
// 128 / N, brings the P = N * R consecutive positions i*N + d of R
// consecutive i, in order, in one copy of the same size (measured: the same
// time as from contiguous rows).  The zig-zag and contiguous placements hold
// 128 consecutive positions in 128 consecutive rows.  Row r of tile t
// always holds position t * P + r.
//
// N that does not divide 128 leaves 128 - P rows of every tile empty, in
// products of the same size, and the forward masks every tile: H = 16 + 4, S =
// 32768, D = 128, window 1024, forward / backward: 282 / 1006 us at P = 128 (N
// = 1, 8, 32, 64, 128), 330 / 1090 at 126 (N = 42, 63), 475 / 1539 at 99 (N =
// 33), 576 / 1799 at 86 (N = 43), 939 / 2853 at 65 (N = 65), 472 / 1532 at 96
// (N = 96).
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

// Tensor-map coordinates of position tile t between the column and the head:
// {stripe, row} in the striped placement, {row, device} in the zig-zag one,
// whose chunks are whole tiles.
struct TileAt {
    int c1, c2;
};
__host__ __device__ __forceinline__ TileAt tile_at(const PosGeom &g, int t) {
    if (g.layout == STRIPED_LAYOUT_STRIPED) return TileAt{0, t * g.R};
    const int per = g.L / 256;  // tiles of a chunk
    const int c = t / per, in = (t - c * per) * 128;
    return c < g.N ? TileAt{in, c} : TileAt{g.L / 2 + in, 2 * g.N - 1 - c};
}

// The row of the [S] tensors that holds row r of tile t.
__host__ __device__ __forceinline__ int64_t tile_row(const PosGeom &g, int t, int r) {
    const TileAt a = tile_at(g, t);
    if (g.layout == STRIPED_LAYOUT_STRIPED) return (int64_t)(r % g.N) * g.L + a.c2 + r / g.N;
    return (int64_t)a.c2 * g.L + a.c1 + r;
}
// Row r of tile t holds a position of the sequence.
__host__ __device__ __forceinline__ bool tile_has(const PosGeom &g, int t, int r) {
    return r < g.P && t * (int64_t)g.P + r < g.S;
}

// Bits 0 .. 31 for columns base .. base + 31: column <= hi and (column >= lo
// or column < sk).
__host__ __device__ __forceinline__ uint32_t kept_bits(int base, int hi, int lo, int sk) {
    hi -= base, lo -= base, sk -= base;
    const uint32_t below = hi >= 31 ? ~0u : hi < 0 ? 0u : (2u << hi) - 1u;
    const uint32_t above = lo <= 0 ? ~0u : lo > 31 ? 0u : ~0u << lo;
    const uint32_t sink = sk >= 32 ? ~0u : sk <= 0 ? 0u : (1u << sk) - 1u;
    return below & (above | sink);
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
