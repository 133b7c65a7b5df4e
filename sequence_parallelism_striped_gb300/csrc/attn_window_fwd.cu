// attn_window_fwd.cu -- bf16 causal attention over a sliding window and a few
// first tokens (sinks), forward, on tcgen05.
//
// Query position p keeps key position t iff t <= p and (p - t < W or
// t < sinks); the placement of the rows is that of the full attention
// (research.elamur.ai summary page, §Summary "every N-th token").  Tiles are
// 128 (or N * (128 / N)) consecutive positions, see window.cuh; query tile a
// visits the sink tiles 0 .. and the tiles from its window's lower edge to
// its own.
//
// A work item is query tiles A = 2u and B = 2u + 1 of one head on one K/V
// stream: their windows differ by one tile.  The K/V tiles of the pair are
//   [0, ns) (sink tiles below the window), [lo(A), B];
// group A takes all but the last (key tile B lies after it), group B all but
// tile lo(A) when that is below its own window and holds no sink.  An item is
// short (W/128 + 3 tiles), so the kernel is persistent: one CTA per
// multiprocessor takes every gridDim-th item, and the next item's Q, K and V
// load, and its first S is formed, while the softmax groups still write out
// the last one's O.
//   warp 0      TMA producer: Q_A, Q_B of an item, then its K/V tiles
//   warp 1      TMEM allocator + tcgen05.mma issuer: the whole warp waits and
//               one elected lane issues (a product of 128 x 128 x 16 in less
//               than the 64 clocks that it runs; from a branch of a single
//               thread in about 90)
//   warps 2..5  softmax group A, thread t owns query row t
//   warps 6..9  softmax group B
// Tensor memory: S_A [0,128), S_B [128,256), O_A [256,256+HD), O_B
// [384,384+HD); P is written back over S as bf16 pairs, the A operand of
// O += P V.  The running max moves lazily (by more than 2^8), which is exact
// because the final division uses the same reference.  P is rounded to bf16
// as a tensor-core operand (tf32 would run at half the rate, with V converted);
// the row sum adds the unrounded values, which lse needs.  o is 2.3e-3 off in
// the root mean square then, 1.6e-3 of it the rounding of o itself.
//
// The kept columns of a row in a partly kept tile (the diagonal one, at most
// two at the window's lower edge, the last sink tile) are a few bit ranges;
// a warp skips the 32-column words that all its rows keep whole.
//
// Bound by the chain S -> softmax -> P -> O of a query tile: the tensor pipe is
// 53% active, DRAM 17%.  Measured (H = 32 + 8, S = 65536, D = 128, N = 8): a
// 128 x 128 tile takes 0.77 us of a multiprocessor at a window of 16384, 1.00
// us at 1024, where an item's ends (its first S, its last O) are 20% of it.
// With 4 sinks, whose tile is one of the ten that a query tile issues for
// eight kept: 1093 us in a graph (1090 .. 1105 over boxes), 1000 TFLOP/s of
// kept pairs; D = 64, H = 32: 857 us.  Slower: 32-column products
// for the sink tile, K and V in places of their own, two issuing warps, two
// threads a row, the maximum off the chain.
#include <math.h>

#include "common.cuh"
#include "internal.h"
#include "window.cuh"

namespace striped {

namespace {

constexpr int WB = 128;                 // tile edge
constexpr uint32_t kWBox = 128 * 128;   // 128 rows x 64 bf16
constexpr int kWMaxNS = 4;
constexpr int kWThreads = 320;
constexpr float kWRescale = 8.0f;       // lazy rescale threshold, log2 units

template <int HD>
struct WinCfg {
    static constexpr int NS = HD == 128 ? 2 : 4;  // K/V stages
    static constexpr uint32_t kTile = (HD / 64) * kWBox;
    static constexpr uint32_t kQOff = 0;  // Q_A, then Q_B
    static constexpr uint32_t kKVOff = 2 * kTile;
    static constexpr uint32_t kStage = 2 * kTile;
    static constexpr uint32_t kBarOff = kKVOff + NS * kStage;
    static constexpr size_t kSmemBytes = 1024 + kBarOff + 256;
    static_assert(kSmemBytes <= 232448, "shared memory over the per-block limit");
    static_assert(NS <= kWMaxNS, "barrier array");
};

// The producer's and the issuer's waits in little code: the tries are not
// unrolled at every place that waits, and a warp's first one ends in a uniform
// branch (S = 65536, window 1024, 4 sinks: 4% off; window 16384: 7%).  At HD =
// 64 the timed tries are a function of their own, at HD = 128 they are inlined
// (each side timed in turn with the other, graphs; HD = 64: S = 65536, H = 32
// 860 us so and 932 inlined, S = 16384, H = 8 67.7 and 73.8, S = 5000 26.7 and
// 28.7; HD = 128: S = 65536, H = 32 + 8 1105 us inlined and 1152 as a
// function, S = 8192, H = 8 45.2 and 47.3, window 16384 1187 and 1232).
__device__ __noinline__ bool win_wait_timed(uint32_t bar, uint32_t parity, const WaitCtl w) {
    return mbar_wait_timed(bar, parity, w);
}
template <int HD>
__device__ __forceinline__ bool win_wait(uint32_t bar, uint32_t parity, const WaitCtl &w) {
#pragma unroll 1
    for (int it = 0; it < 64; ++it)
        if (mbar_try_wait(bar, parity)) return true;
    if constexpr (HD == 64) return win_wait_timed(bar, parity, w);
    return mbar_wait_timed(bar, parity, w);
}
template <int HD>
__device__ __forceinline__ bool win_wait_warp(uint32_t bar, uint32_t parity, const WaitCtl &w) {
    if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
    return __all_sync(0xffffffffu, win_wait<HD>(bar, parity, w));
}

struct WinBars {
    uint64_t q_full, q_empty;
    uint64_t kv_full[kWMaxNS], kv_empty[kWMaxNS];
    uint64_t s_full[2], p_ready[2][2], o_done[2];  // per softmax group (P in two halves)
    uint64_t drain;                             // every MMA of the issuer has completed
    uint32_t tmem_slot;
};

struct WinParams {
    PosGeom g;
    int W, sinks;
    int nst;      // sink tiles
    int npair;    // query tile pairs of a head
    int items;    // pairs of all heads
    int G;        // query heads per key/value head
    float scale;
    __nv_bfloat16 *o;
    float *lse;
    bool wide;    // o is 32-byte aligned
    WaitCtl wc;
};

// One work item: a pair of query tiles and its K/V tiles, [0, ns) and then
// lo, lo + 1, ..
struct WinItem {
    int64_t bh;
    int qa, lo, ns, nt;
    bool has_b;
    __device__ __forceinline__ WinItem(const WinParams &p, int item) {
        bh = item / p.npair;
        qa = 2 * (item - (int)bh * p.npair);
        has_b = qa + 1 < p.g.nt;
        lo = window_lo(p.g, qa, p.W);
        ns = min(p.nst, lo);
        nt = ns + (has_b ? qa + 1 : qa) - lo + 1;
    }
    __device__ __forceinline__ int key_tile(int t) const { return t < ns ? t : lo + t - ns; }
    // The tile that group B leaves out (-1: none), and group x's first and
    // last tile (group B without a query tile: none, first > last).
    __device__ __forceinline__ int skip(const WinParams &p) const {
        return window_lo(p.g, qa + 1, p.W) > lo && lo >= p.nst ? ns : -1;
    }
    __device__ __forceinline__ int first(int x, int skip) const { return !x ? 0 : !has_b ? nt : skip == 0 ? 1 : 0; }
    __device__ __forceinline__ int last(int x) const { return x || !has_b ? nt - 1 : nt - 2; }
};

template <int HD>
__global__ void __launch_bounds__(kWThreads, 1)
    tc_window_fwd_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                         const __grid_constant__ CUtensorMap tmV, const WinParams p) {
    using Cfg = WinCfg<HD>;
    constexpr int NS = Cfg::NS;
    constexpr uint32_t kTile = Cfg::kTile, kQOff = Cfg::kQOff, kKVOff = Cfg::kKVOff, kStage = Cfg::kStage;
    constexpr int kBoxes = HD / 64;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem =
        reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    WinBars *bars = reinterpret_cast<WinBars *>(smem + Cfg::kBarOff);
    const uint32_t sbase = smem_u32(smem);
    const PosGeom &g = p.g;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;

    if (threadIdx.x == 0) {
        mbar_init(smem_u32(&bars->q_full), 1);
        mbar_init(smem_u32(&bars->q_empty), 1);
        for (int s = 0; s < NS; ++s) {
            mbar_init(smem_u32(&bars->kv_full[s]), 1);
            mbar_init(smem_u32(&bars->kv_empty[s]), 1);
        }
        for (int x = 0; x < 2; ++x) {
            mbar_init(smem_u32(&bars->s_full[x]), 1);
            mbar_init(smem_u32(&bars->p_ready[x][0]), 4);
            mbar_init(smem_u32(&bars->p_ready[x][1]), 4);
            mbar_init(smem_u32(&bars->o_done[x]), 1);
        }
        mbar_init(smem_u32(&bars->drain), 1);
        fence_barrier_init();
    }
    if (g.P < WB) {
        // rows past the tile's positions are never loaded: they must hold
        // finite values, because P = 0 times them is added to O
        for (uint32_t i = threadIdx.x * 16; i < kKVOff + NS * kStage; i += kWThreads * 16)
            *reinterpret_cast<uint4 *>(smem + i) = make_uint4(0u, 0u, 0u, 0u);
        fence_proxy_async_smem();
    }
    if (warp == 1) {
        tmem_alloc(smem_u32(&bars->tmem_slot), 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = bars->tmem_slot;

    if (warp == 0 && lane == 0) {
        // ---------------- TMA producer
        tma_prefetch_desc(&tmQ);
        tma_prefetch_desc(&tmK);
        tma_prefetch_desc(&tmV);
        const uint32_t box_bytes = (uint32_t)g.P * 128;
        const uint32_t qbar = smem_u32(&bars->q_full);
        // test hook: the first K/V tile is never loaded, so every wait on it
        // runs out (the kernel must then record the timeout and return)
        const bool skip_first = p.wc.inject == kInjectFwdSkipKV;
        int j = 0;        // K/V tiles so far
        int last_q = -1;  // item (of this CTA) whose Q was loaded last
        bool ok = true;
        for (int item = blockIdx.x; item < p.items && ok; item += gridDim.x) {
            const WinItem w(p, item);
            const int kvh = (int)(w.bh / p.G);
            if (last_q >= 0 && !win_wait<HD>(smem_u32(&bars->q_empty), last_q & 1, p.wc)) break;
            ++last_q;
            mbar_arrive_expect_tx(qbar, (w.has_b ? 2 : 1) * kBoxes * box_bytes);
            for (int x = 0; x < (w.has_b ? 2 : 1); ++x) {
                const TileAt at = tile_at(g, w.qa + x);
#pragma unroll
                for (int c = 0; c < kBoxes; ++c)
                    tma_load_4d(sbase + kQOff + x * kTile + c * kWBox, &tmQ, qbar, 64 * c, at.c1, at.c2,
                                (int)w.bh);
            }
            for (int t = 0; t < w.nt; ++t, ++j) {
                const int s = j % NS;
                if (j >= NS && !win_wait<HD>(smem_u32(&bars->kv_empty[s]), ((j / NS) + 1) & 1, p.wc)) {
                    ok = false;
                    break;
                }
                if (skip_first && j == 0) continue;
                const TileAt at = tile_at(g, w.key_tile(t));
                const uint32_t fb = smem_u32(&bars->kv_full[s]);
                const uint32_t kdst = sbase + kKVOff + s * kStage, vdst = kdst + kTile;
                mbar_arrive_expect_tx(fb, 2 * kBoxes * box_bytes);
#pragma unroll
                for (int c = 0; c < kBoxes; ++c) {
                    tma_load_4d(kdst + c * kWBox, &tmK, fb, 64 * c, at.c1, at.c2, kvh);
                    tma_load_4d(vdst + c * kWBox, &tmV, fb, 64 * c, at.c1, at.c2, kvh);
                }
            }
        }
        // loads [0, j) and the last Q were issued: wait (bounded) for the last
        // of each stage, so that on an error path none lands after the CTA has
        // exited
        if (last_q >= 0) win_wait<HD>(qbar, last_q & 1, p.wc);
        for (int t = j > NS ? j - NS : 0; t < j; ++t)
            if (!(skip_first && t == 0)) win_wait<HD>(smem_u32(&bars->kv_full[t % NS]), (t / NS) & 1, p.wc);
    } else if (warp == 1) {
        // ---------------- MMA issuer: PV_A(t), S_A(next), PV_B(t), S_B(next)
        constexpr uint32_t idesc_qk = idesc_bf16_f32(WB, WB, false, false);
        constexpr uint32_t idesc_pv = idesc_bf16_f32(WB, HD, false, true);
        const bool leader = elect_one();
        const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
        // descriptors of the first Q tile, K tile and V tile; others lie
        // whole 16-byte units above
        const uint64_t dq = sdesc_sw128(sbase + kQOff, 16, 1024), dk = sdesc_sw128(sbase + kKVOff, 16, 1024);
        const uint64_t dv = sdesc_sw128(sbase + kKVOff + kTile, kWBox, 1024);
        int n[2] = {0, 0};      // tiles of each group so far
        int jbase = 0, it = 0;  // K/V tiles and items so far
        int total = 0;          // K/V tiles of this CTA
        for (int item = blockIdx.x; item < p.items; item += gridDim.x) total += WinItem(p, item).nt;
        bool ok = true;
        int seen = -1;  // last tile whose K and V were waited for
        auto issue_s = [&](int x, int j) -> bool {
            const int s = j % NS;
            if (j > seen && !win_wait_warp<HD>(smem_u32(&bars->kv_full[s]), (j / NS) & 1, p.wc)) return false;
            seen = max(seen, j);
            tc_fence_after();
            if (leader) {
                const uint64_t qx = dq + x * (kTile >> 4), ks = dk + s * (kStage >> 4);
#pragma unroll
                for (int kk = 0; kk < HD / 16; ++kk) {
                    const uint32_t off = ((kk >> 2) * kWBox + (kk & 3) * 32) >> 4;
                    mma_ss(tm + 128 * x, qx + off, ks + off, idesc_qk, kk > 0 ? 1u : 0u);
                }
                mma_commit(smem_u32(&bars->s_full[x]));
            }
            return true;
        };
        // O_x += P_x V in two halves of 64 keys, each as soon as its P is there
        auto issue_pv = [&](int x, int j, bool first, bool last) -> bool {
            const uint64_t vs = dv + (j % NS) * (kStage >> 4);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                if (!win_wait_warp<HD>(smem_u32(&bars->p_ready[x][h]), n[x] & 1, p.wc)) return false;
                tc_fence_after();
                if (leader) {
#pragma unroll
                    for (int k4 = 0; k4 < WB / 32; ++k4) {
                        const int kk = h * (WB / 32) + k4;
                        mma_ts(tm + 256 + 128 * x, tm + 128 * x + kk * 8, vs + kk * (2048 >> 4), idesc_pv,
                               (!first || kk > 0) ? 1u : 0u);
                    }
                }
            }
            // the other tiles' products are covered by the next S's commit
            if (leader && last) mma_commit(smem_u32(&bars->o_done[x]));
            ++n[x];
            return true;
        };
        for (int item = blockIdx.x; item < p.items && ok; item += gridDim.x, ++it) {
            const WinItem w(p, item);
            const bool more = item + (int)gridDim.x < p.items;
            const int skip = w.skip(p), last_a = w.last(0);
            const int first_b = w.first(1, skip);
            ok = win_wait_warp<HD>(smem_u32(&bars->q_full), it & 1, p.wc);
            tc_fence_after();
            if (ok) ok = issue_s(0, jbase);
            if (ok && w.has_b) ok = issue_s(1, jbase + first_b);
            for (int t = 0; t < w.nt && ok; ++t) {
                const int j = jbase + t;
                if (t <= last_a) {
                    ok = issue_pv(0, j, t == 0, t == last_a);
                    if (ok && t < last_a) ok = issue_s(0, j + 1);
                    if (!ok) break;
                }
                const bool b = w.has_b && t != skip;
                if (b) ok = issue_pv(1, j, t == first_b, t == w.nt - 1);
                if (!ok) break;
                // every stage is released but the CTA's last ones (no arrival
                // may land after the CTA has exited)
                if (leader && j + NS < total) mma_commit(smem_u32(&bars->kv_empty[j % NS]));
                if (b && t < w.nt - 1) ok = issue_s(1, j + (t + 1 == skip ? 2 : 1));
                // the item's last S has been issued: Q may be replaced once
                // that is complete
                if (leader && ok && more && t == max(w.nt - 2, 0)) mma_commit(smem_u32(&bars->q_empty));
            }
            jbase += w.nt;
        }
        // every MMA issued above completes before TMEM is freed (error paths)
        if (leader) mma_commit(smem_u32(&bars->drain));
        win_wait_warp<HD>(smem_u32(&bars->drain), 0, p.wc);
    } else if (warp >= 2) {
        // ---------------- softmax + epilogue of one query tile
        const int x = (warp - 2) >> 2;       // group: query tile qa or qa + 1
        const int quarter = warp & 3;
        const int ri = quarter * 32 + lane;  // query row of the tile
        const uint32_t lane_off = (uint32_t)(quarter * 32) << 16;
        const uint32_t tS = tmem + 128 * x + lane_off, tO = tmem + 256 + 128 * x + lane_off;
        const float cl2 = p.scale * 1.4426950408889634f;
        int n = 0, m = 0;  // tiles turned into P, items written out
        bool ok = true;
        for (int item = blockIdx.x; item < p.items && ok; item += gridDim.x) {
            const int bh = item / p.npair, qt = 2 * (item - bh * p.npair) + x;
            if (qt >= g.nt) continue;
            const int lo = window_lo(g, qt, p.W), ns = min(p.nst, lo);
            float m_ref = -INFINITY, l = 0.f;
            bool first = true;
            for (int kt = ns > 0 ? 0 : lo; kt <= qt; kt = kt + 1 == ns ? lo : kt + 1) {
                if (!mbar_wait_warp(smem_u32(&bars->s_full[x]), n & 1, p.wc)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                float sv[WB];
                {
                    uint32_t r0[32], r1[32], r2[32], r3[32];
                    tmem_ld32(tS, r0);
                    tmem_ld32(tS + 32, r1);
                    tmem_ld32(tS + 64, r2);
                    tmem_ld32(tS + 96, r3);
                    tmem_ld_wait(r0);
                    tmem_ld_wait(r1);
                    tmem_ld_wait(r2);
                    tmem_ld_wait(r3);
#pragma unroll
                    for (int c = 0; c < 32; ++c) {
                        sv[c] = __uint_as_float(r0[c]);
                        sv[32 + c] = __uint_as_float(r1[c]);
                        sv[64 + c] = __uint_as_float(r2[c]);
                        sv[96 + c] = __uint_as_float(r3[c]);
                    }
                }
                // column c of the tile is kept iff c <= hi and (c >= lo or
                // c < sk); uniform test: every pair of the two tiles is
                const int dist = (qt - kt) * g.P, sk = p.sinks - kt * g.P;
                if (!(g.P == WB && dist > 0 && (dist + WB <= p.W || sk >= WB))) {
                    const int hi = min(ri + dist, g.P - 1), lo = ri + dist - p.W + 1;
#pragma unroll
                    for (int b = 0; b < WB / 32; ++b) {
                        const uint32_t k = kept_bits(32 * b, hi, lo, sk);
                        if (!__all_sync(0xffffffffu, k == ~0u))
#pragma unroll
                            for (int c = 0; c < 32; ++c)
                                if (!(k & (1u << c))) sv[32 * b + c] = -INFINITY;
                    }
                }
                const float m_tile = row_max(sv) * cl2;
                const bool move = first || m_tile > m_ref + kWRescale;
                const float m_new = move ? fmaxf(m_ref, m_tile) : m_ref;
                const float alpha = (first || !move) ? 1.f : ex2(m_ref - m_new);
                const float m_use = (m_new == -INFINITY) ? 0.f : m_new;
                // S(n) was committed after the group's previous product, so O
                // may be corrected now (rare: the max moved by 2^8)
                if (__any_sync(0xffffffffu, alpha != 1.f)) {
#pragma unroll 1
                    for (int c = 0; c < HD / 32; ++c) {
                        uint32_t rr[32];
                        tmem_ld32(tO + c * 32, rr);
                        tmem_ld_wait(rr);
#pragma unroll
                        for (int v = 0; v < 32; ++v) rr[v] = __float_as_uint(__uint_as_float(rr[v]) * alpha);
                        tmem_st32(tO + c * 32, rr);
                    }
                }
                const uint64_t cl2x2 = f2(cl2, cl2), nm2 = f2(-m_use, -m_use);
                uint64_t acc4[4] = {0ull, 0ull, 0ull, 0ull};
                // P in two halves, each handed to the tensor core by itself
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    uint32_t pk[32];
#pragma unroll
                    for (int c = 0; c < 32; ++c) {
                        const float2 e = f2_split(fma2(f2(sv[64 * h + 2 * c], sv[64 * h + 2 * c + 1]), cl2x2, nm2));
                        const float p0 = ex2(e.x), p1 = ex2(e.y);
                        acc4[c & 3] = add2(acc4[c & 3], f2(p0, p1));
                        pk[c] = pack_bf16x2(p0, p1);
                    }
                    tmem_st32(tS + 32 * h, pk);
                    tmem_st_wait();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(smem_u32(&bars->p_ready[x][h]));
                }
                const float2 s01 = f2_split(add2(acc4[0], acc4[1])), s23 = f2_split(add2(acc4[2], acc4[3]));
                l = l * alpha + ((s01.x + s01.y) + (s23.x + s23.y));
                m_ref = m_new;
                ++n;
                first = false;
            }
            // ---------------- epilogue
            if (ok) ok = mbar_wait_warp(smem_u32(&bars->o_done[x]), m++ & 1, p.wc);
            tc_fence_after();
            const bool valid = tile_has(g, qt, ri);
            const bool empty = !(l > 0.f) || !ok;
            const float inv_l = empty ? 0.f : 1.f / l;
            const float lse_row = empty ? -INFINITY : (m_ref + log2f(l)) * 0.6931471805599453f;
            const int64_t row = bh * (int64_t)g.S + (valid ? tile_row(g, qt, ri) : 0);
            if (valid) p.lse[row] = lse_row;
#pragma unroll
            for (int c = 0; c < HD / 32; ++c) {
                uint32_t rr[32];
                tmem_ld32(tO + c * 32, rr);
                tmem_ld_wait(rr);
                if (!valid) continue;
                __nv_bfloat16 *dst = p.o + row * HD + c * 32;
#pragma unroll
                for (int v = 0; v < 2; ++v) {
                    uint32_t o8[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        o8[i] = pack_bf16x2(__uint_as_float(rr[16 * v + 2 * i]) * inv_l,
                                            __uint_as_float(rr[16 * v + 2 * i + 1]) * inv_l);
                    st_global_32(dst + 16 * v, o8, p.wide);
                }
            }
            tc_fence_before();  // O is read out before the next item's first P is announced
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) {
        __syncwarp();
        tmem_dealloc(tmem, 512);
    }
}

template <int HD>
int launch_window_hd(const CUtensorMap &mq, const CUtensorMap &mk, const CUtensorMap &mv, const WinParams &p,
                     int64_t nblocks, cudaStream_t stream) {
    static PerDeviceOnce once;
    const int attr = once.get([] {
        return cuda_status(cudaFuncSetAttribute(tc_window_fwd_kernel<HD>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                (int)WinCfg<HD>::kSmemBytes));
    });
    if (attr != STRIPED_OK) return attr;
    tc_window_fwd_kernel<HD><<<(unsigned)nblocks, kWThreads, WinCfg<HD>::kSmemBytes, stream>>>(mq, mk, mv, p);
    return cuda_status(cudaGetLastError());
}

}  // namespace

int launch_tc_window_fwd(const void *q, const void *k, const void *v, void *o, float *lse, const WindowArgs &a,
                         cudaStream_t stream) {
    WinParams p{};
    if (!pos_geom(&p.g, a.S, a.N, a.layout)) return STRIPED_ERR_UNSUPPORTED;
    p.W = (int)(a.window < a.S ? a.window : a.S);
    p.sinks = (int)(a.sinks < a.S ? a.sinks : a.S);
    p.nst = (p.sinks + p.g.P - 1) / p.g.P;
    p.npair = (p.g.nt + 1) / 2;
    p.G = (int)(a.H / a.Hkv);
    p.scale = a.scale;
    p.o = static_cast<__nv_bfloat16 *>(o);
    p.lse = lse;
    p.wide = (reinterpret_cast<uintptr_t>(o) & 31u) == 0;
    p.wc = device_wait_ctl();
    const int sms = device_sm_count();
    const int64_t items = (int64_t)p.npair * a.B * a.H;
    if (items > 0x7fffffffll - 1024) return STRIPED_ERR_UNSUPPORTED;
    p.items = (int)items;
    const int nblocks = (int)(items < sms ? items : sms);
    CUtensorMap mq, mk, mv;
    int st;
    if ((st = make_pos_map(&mq, q, a.D, p.g, a.B * a.H)) || (st = make_pos_map(&mk, k, a.D, p.g, a.B * a.Hkv)) ||
        (st = make_pos_map(&mv, v, a.D, p.g, a.B * a.Hkv)))
        return st;
    return a.D == 128 ? launch_window_hd<128>(mq, mk, mv, p, nblocks, stream)
                      : launch_window_hd<64>(mq, mk, mv, p, nblocks, stream);
}

}  // namespace striped
