// attn_window_bwd.cu -- backward of the attention over a sliding window and a
// few first tokens (sinks), bf16 on tcgen05.
//
// With P = exp(scale q k^T - LSE) on the pairs that the forward keeps (key
// t <= query p and (p - t < W or t < sinks)) and Delta_p = <dO_p, O_p>:
//   dV = P^T dO,  dP = dO V^T,  dS = P * (dP - Delta),
//   dK = scale * dS^T Q,  dQ = scale * dS K.
// P and dS are rounded to bf16 as tensor-core operands, dS from the unrounded
// P (from the rounded one dQ and dK would be 2.9e-3 off instead of 2.4e-3, of
// which the rounding of the results alone is 1.7e-3); every sum is fp32.
//
// Kernels:
//   window_pre   per query tile of consecutive positions (window.cuh) the
//                block [LSE*log2e 128 | Delta 128], and a zeroed fp32 dQ
//                accumulator in the same tile order
//   window_bwd   one CTA per unit of a key/value head: a key tile against
//                the query tiles whose window reaches it; for a sink tile
//                also far units, each a stretch of the later query tiles
//                (a sink tile is seen by every query: as one CTA it would
//                run alone long after the others).  The units of a sink tile
//                write their dK, dV as fp32 shares
//   window_post  dQ = bf16(scale * accumulator) in the placement's rows, and
//                the sink tiles' dK, dV from their shares in a fixed order
//
// The main kernel has the pipeline of the full attention's backward: warp 0 =
// TMA producer (K, V once; then Q_i with its statistics, 2 stages), warp 2 =
// TMA producer of dO_i, warp 1 = TMEM allocator + MMA issuer (the whole warp
// waits, one elected lane issues), warps 4..11 = two compute warpgroups; thread
// t owns key row t of S^T and dP^T.  Warps 12..15 only carry dQ_i from tensor
// memory to the accumulator, so that the compute warps go on to the next tile;
// the accumulator is laid out so that a warp's 16-byte reductions are whole
// lines.
//   TMEM: S^T [0,128) (P^T bf16 pairs over it), dP^T [128,256) (dQ_i over it
//   once dS_i is formed), dV [256,256+HD), dK [256+HD,256+2HD).
//     S^T  = K Q_i^T      SS, both K-major
//     dP^T = V dO_i^T     SS, both K-major
//     dV  += P^T dO_i     TS, A = P^T in TMEM, B = dO_i MN-major
//     dK  += dS^T Q_i     SS, A = dS smem tile read K-major
//     dQ_i^T = K^T dS^T   SS, A = K read MN-major, B = the dS tile read
//                         MN-major (HD = 128)
//     dQ_i = dS K         SS, A = the dS tile read MN-major (HD = 64)
// The accumulator holds whole tiles, so every reduction is unconditional;
// its order, and with it the last bits of dQ, change from run to run (a few
// fp32 ulps before the rounding to bf16), dK and dV do not.
//
// Bound by the hand-offs and the L2's fp32 reductions (64 KB a tile): tensor
// pipe 45% active; without the reductions the main kernel would take 0.8 of
// its time.  Measured (H = 32 + 8, S = 32768, D = 128, window 2048, 16 sinks,
// zig-zag): 3.03 ms, 885 TFLOP/s of kept pairs, 2.9 us a 128 x 128 tile of one
// multiprocessor (the full attention's backward: 3.04); D = 64, H = 32: 2.01
// ms.  The four kernels follow one another by programmatic launches: 8 us less
// a call.  A unit takes its key tile against all G query heads, so few
// key/value heads on a short sequence leave multiprocessors idle: H = 32, S =
// 2048, window 1024: 116 us on 32 key/value heads, 212 on 4, 782 on 1 (16
// units); S = 8192 480 on 8, 845 on 1.
#include <math.h>

#include "common.cuh"
#include "internal.h"
#include "window.cuh"

namespace striped {

namespace {

constexpr int BT = 128;
constexpr int QS = 2;  // Q/dO stages
constexpr uint32_t kBox = 128 * 128;  // 128 rows x 64 bf16 (one 128-byte-swizzle box)
constexpr uint32_t kStatBytes = 2 * 128 * 4;
constexpr int kThreads = 512;  // warp 0 and 2 TMA, warp 1 MMA, warps 4..11 compute, 12..15 dQ

template <int HD>
struct WinBwdCfg {
    static constexpr uint32_t kTile = (HD / 64) * kBox;
    static constexpr uint32_t kKOff = 0;
    static constexpr uint32_t kVOff = kTile;
    static constexpr uint32_t kQOff = 2 * kTile;                // stage s: Q at kQOff + s*2*kTile, dO after
    static constexpr uint32_t kDSOff = kQOff + QS * 2 * kTile;  // dS (MN-major A operand)
    static constexpr uint32_t kStatOff = kDSOff + 2 * kBox;     // per stage: [LSE*log2e 128 | Delta 128]
    static constexpr uint32_t kBarOff = kStatOff + QS * kStatBytes;
    static constexpr size_t kSmemBytes = kBarOff + 256;           // the dynamic smem base is 1024-aligned
    static_assert(kSmemBytes <= 232448, "shared memory over the per-block limit");
};

struct WinBwdParams {
    PosGeom g;
    int W, sinks;
    int nst;        // sink tiles
    int chunk;      // query tiles of one far unit
    int slots;      // dK/dV shares kept per sink tile (0: no far units)
    int units;      // CTAs of one key/value head
    int G;          // query heads per key/value head
    float scale;
    const float *stats;  // [BH][nt][LSE*log2e 128 | Delta 128], rows of a tile
    float *dq_acc;       // [BH][nt] tiles of fp32: HD = 128 [query / 4][D][4], HD = 64 [D / 4][query][4]
    float *parts;        // [BHkv][nst][slots][dK 128 D | dV 128 D] fp32
    __nv_bfloat16 *dk, *dv;
    bool wide;  // dk and dv are 32-byte aligned
    WaitCtl wc;  // status word, wait bound, test hook
};

// The producers' and the issuer's waits with one place that tries (B = 1, H =
// 8, S = 8192, window 1024: 158 us with the tries unrolled at every place that
// waits, 155 with them in a loop of their own, 152 so).
__device__ __forceinline__ bool bwd_wait(uint32_t bar, uint32_t parity, const WaitCtl &w) {
    uint64_t t0 = 0;
#pragma unroll 1
    for (uint32_t it = 1;; ++it) {
        if (mbar_try_wait(bar, parity)) return true;
        if ((it & 63u) == 0u) {
            const uint64_t now = global_timer_ns();
            if (t0 == 0) t0 = now;
            else if (now - t0 > w.limit_ns) break;
        }
    }
    record_timeout(w);
    return false;
}
__device__ __forceinline__ bool bwd_wait_warp(uint32_t bar, uint32_t parity, const WaitCtl &w) {
    return __all_sync(0xffffffffu, bwd_wait(bar, parity, w));
}

struct Bars {
    uint64_t kv_full;
    uint64_t q_full[QS], q_empty[QS];    // Q_i + statistics of tile i
    uint64_t do_full[QS], do_empty[QS];  // dO_i
    uint64_t s_full, dp_full, p_ready, ds_ready, dq_full, dq_free, acc_done;
    uint64_t drain;  // every MMA of the issuer has completed (before TMEM is freed)
    uint32_t tmem_slot;
};

// Far units of sink tile kt: queries above its window, `chunk` tiles each.
__host__ __device__ __forceinline__ int far_units(const PosGeom &g, int kt, int W, int chunk) {
    const int far = g.nt - 1 - window_hi(g, kt, W);
    return far > 0 ? (far + chunk - 1) / chunk : 0;
}

template <int HD>
__global__ void __launch_bounds__(kThreads, 1)
    tc_window_bwd_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                         const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CUtensorMap tmdO,
                         const WinBwdParams p) {
    using Cfg = WinBwdCfg<HD>;
    constexpr uint32_t kTile = Cfg::kTile, kKOff = Cfg::kKOff, kVOff = Cfg::kVOff, kQOff = Cfg::kQOff,
                       kDSOff = Cfg::kDSOff, kStatOff = Cfg::kStatOff;
    constexpr int kBoxes = HD / 64;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t *smem = smem_raw;
    if ((smem_u32(smem) & 1023u) != 0) {  // operand tiles need 1024-byte alignment
        if (threadIdx.x == 0) record_error(p.wc.st, STRIPED_ERR_ALIGN);
        return;
    }
    Bars *bars = reinterpret_cast<Bars *>(smem + Cfg::kBarOff);
    const uint32_t sbase = smem_u32(smem);
    const PosGeom &g = p.g;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;

    // Head-major order: resident CTAs belong to one key/value head and sweep
    // neighbouring query tiles, sharing Q/dO tiles and dQ accumulator lines
    // in L2.  Units of a head: its key tiles (against their window), then
    // the far units of the sink tiles.
    const int G = p.G;
    const int64_t bh = blockIdx.x / p.units;
    const int unit = blockIdx.x % p.units;
    int kt = unit, a_lo, a_hi, slot = 0;  // query tiles a_lo .. a_hi
    if (unit < g.nt) {
        a_lo = kt;
        a_hi = window_hi(g, kt, p.W);
    } else {
        int i = unit - g.nt;
        kt = 0;
        for (int n; i >= (n = far_units(g, kt, p.W, p.chunk)); ++kt) i -= n;
        slot = 1 + i;
        a_lo = window_hi(g, kt, p.W) + 1 + i * p.chunk;
        a_hi = min(g.nt - 1, a_lo + p.chunk - 1);
    }
    // a sink tile's dK and dV are sums of several units' shares
    const bool shared_tile = kt < p.nst && p.slots > 0;
    const int cnt = a_hi - a_lo + 1;
    const int nt = cnt * G;  // (query head, query tile) pairs, tiles upwards
    const TileAt kat = tile_at(g, kt);
    const int kbase = kt * g.P;

    if (threadIdx.x == 0) {
        mbar_init(smem_u32(&bars->kv_full), 1);
        for (int s = 0; s < QS; ++s) {
            mbar_init(smem_u32(&bars->q_full[s]), 1);
            mbar_init(smem_u32(&bars->q_empty[s]), 1);   // released by dK_i's commit
            mbar_init(smem_u32(&bars->do_full[s]), 1);
            mbar_init(smem_u32(&bars->do_empty[s]), 1);  // released by dV_i's commit
        }
        mbar_init(smem_u32(&bars->s_full), 1);
        mbar_init(smem_u32(&bars->dp_full), 1);
        mbar_init(smem_u32(&bars->p_ready), 8);
        mbar_init(smem_u32(&bars->ds_ready), 8);
        mbar_init(smem_u32(&bars->dq_full), 1);
        mbar_init(smem_u32(&bars->dq_free), 4);
        mbar_init(smem_u32(&bars->acc_done), 1);
        mbar_init(smem_u32(&bars->drain), 1);
        fence_barrier_init();
    }
    if (g.P < BT) {
        // rows past the tile's positions are never loaded: they must hold
        // finite values, because P = 0 times them is added to the gradients
        for (uint32_t i = threadIdx.x * 16; i < kDSOff; i += kThreads * 16)
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
    let_next_begin();
    wait_for_previous();  // statistics and the cleared accumulator
    const uint32_t tmem = bars->tmem_slot;
    const uint32_t tS = tmem, tdP = tmem + 128, tdV = tmem + 256, tdK = tmem + 256 + HD;

    // 512 threads start with 128 registers each; the compute and dQ
    // warpgroups take what the first one gives up: 56 + 2 * 152 + 152 = 4 * 128
    if (warp < 4) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
        if (warp == 0 && lane == 0 && nt > 0) {
            // ---------------- TMA producer: K, V once, then Q_i + statistics
            tma_prefetch_desc(&tmQ);
            tma_prefetch_desc(&tmK);
            tma_prefetch_desc(&tmV);
            tma_prefetch_desc(&tmdO);
            const uint32_t kb = smem_u32(&bars->kv_full);
            const uint32_t tile_bytes = kBoxes * (uint32_t)g.P * 128;
            mbar_arrive_expect_tx(kb, 2 * tile_bytes);
#pragma unroll
            for (int x = 0; x < kBoxes; ++x) tma_load_4d(sbase + kKOff + x * kBox, &tmK, kb, 64 * x, kat.c1, kat.c2, (int)bh);
#pragma unroll
            for (int x = 0; x < kBoxes; ++x) tma_load_4d(sbase + kVOff + x * kBox, &tmV, kb, 64 * x, kat.c1, kat.c2, (int)bh);
            // test hook: the first Q tile is never loaded, so every wait on it
            // runs out (the kernel must then record the timeout and return)
            const bool skip_first = p.wc.inject == kInjectBwdSkipQ;
            int i = 0;
            for (; i < nt; ++i) {
                const int s = i % QS;
                if (i >= QS && !bwd_wait(smem_u32(&bars->q_empty[s]), ((i / QS) + 1) & 1, p.wc)) break;
                if (skip_first && i == 0) continue;
                const uint32_t fb = smem_u32(&bars->q_full[s]);
                const uint32_t qdst = sbase + kQOff + s * 2 * kTile;
                const int64_t bq = bh * G + i / cnt;  // query head
                const int qt = a_lo + i % cnt;
                const TileAt at = tile_at(g, qt);
                mbar_arrive_expect_tx(fb, tile_bytes + kStatBytes);
                bulk_load(sbase + kStatOff + s * kStatBytes, p.stats + ((bq * g.nt + qt) << 8), kStatBytes, fb);
#pragma unroll
                for (int x = 0; x < kBoxes; ++x)
                    tma_load_4d(qdst + x * kBox, &tmQ, fb, 64 * x, at.c1, at.c2, (int)bq);
            }
            // K, V and loads [0, i) were issued: wait (bounded) for the last of
            // each stage, so that on an error path none lands after the CTA exits
            bwd_wait(kb, 0, p.wc);
            for (int t = i > QS ? i - QS : 0; t < i; ++t)
                if (!(skip_first && t == 0)) bwd_wait(smem_u32(&bars->q_full[t % QS]), (t / QS) & 1, p.wc);
        } else if (warp == 2 && lane == 0 && nt > 0) {
            // ---------------- TMA producer: dO_i (its own stream: the buffer is
            // released at dV_i, Q_i's at dK_i)
            tma_prefetch_desc(&tmdO);
            int i = 0;
            for (; i < nt; ++i) {
                const int s = i % QS;
                if (i >= QS && !bwd_wait(smem_u32(&bars->do_empty[s]), ((i / QS) + 1) & 1, p.wc)) break;
                const uint32_t fb = smem_u32(&bars->do_full[s]);
                const uint32_t odst = sbase + kQOff + s * 2 * kTile + kTile;
                const int bq = (int)(bh * G) + i / cnt;
                const TileAt at = tile_at(g, a_lo + i % cnt);
                mbar_arrive_expect_tx(fb, kBoxes * (uint32_t)g.P * 128);
#pragma unroll
                for (int x = 0; x < kBoxes; ++x)
                    tma_load_4d(odst + x * kBox, &tmdO, fb, 64 * x, at.c1, at.c2, bq);
            }
            for (int t = i > QS ? i - QS : 0; t < i; ++t)  // in-flight loads, as above
                bwd_wait(smem_u32(&bars->do_full[t % QS]), (t / QS) & 1, p.wc);
        } else if (warp == 1 && nt > 0) {
            // ---------------- MMA issuer (the whole warp, one lane issues)
            // Per query tile i (TMEM: S = S^T then P^T; DP = dP^T then dQ_i):
            //   dV += P^T dO | S(i+1) | dK += dS^T Q | dQ_i = dS K | dP(i+1)
            // so S(i+1) runs while the compute warps form dS_i and P(i+1), Q_i
            // is released at dK_i, and dP(i+1) follows as soon as dQ_i is out.
            const bool leader = elect_one();
            const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
            const uint32_t uS = tm, udP = tm + 128, udV = tm + 256, udK = tm + 256 + HD;
            constexpr uint32_t id_kk = idesc_bf16_f32(BT, BT, false, false);
            constexpr uint32_t id_kmn = idesc_bf16_f32(BT, HD, false, true);
            constexpr uint32_t id_mnmn = idesc_bf16_f32(BT, HD, true, true);
            constexpr uint32_t id_dqt = idesc_bf16_f32(HD, BT, true, true);  // dQ^T: M = HD, N = 128 queries
            // descriptors of the operand tiles read K-major and MN-major; steps
            // along K and further stages lie whole 16-byte units above
            const uint64_t k_k = sdesc_sw128(sbase + kKOff, 16, 1024), k_mn = sdesc_sw128(sbase + kKOff, kBox, 1024);
            const uint64_t v_k = sdesc_sw128(sbase + kVOff, 16, 1024);
            const uint64_t q_k = sdesc_sw128(sbase + kQOff, 16, 1024), q_mn = sdesc_sw128(sbase + kQOff, kBox, 1024);
            const uint64_t ds_k = sdesc_sw128(sbase + kDSOff, 16, 1024), ds_mn = sdesc_sw128(sbase + kDSOff, kBox, 1024);
            constexpr uint32_t kStep = (2 * kTile) >> 4, kdO = kTile >> 4;  // next stage; dO after Q
            auto along_k = [](int kk) -> uint32_t { return ((kk >> 2) * kBox + (kk & 3) * 32) >> 4; };
            auto issue_s = [&](int t) -> bool {
                const int s = t % QS;
                if (!bwd_wait_warp(smem_u32(&bars->q_full[s]), (t / QS) & 1, p.wc)) return false;
                tc_fence_after();
                if (leader) {
#pragma unroll
                    for (int kk = 0; kk < HD / 16; ++kk)
                        mma_ss(uS, k_k + along_k(kk), q_k + s * kStep + along_k(kk), id_kk, kk > 0 ? 1u : 0u);
                    mma_commit(smem_u32(&bars->s_full));
                }
                return true;
            };
            auto issue_dp = [&](int t) -> bool {
                const int s = t % QS;
                if (!bwd_wait_warp(smem_u32(&bars->do_full[s]), (t / QS) & 1, p.wc)) return false;
                tc_fence_after();
                if (leader) {
#pragma unroll
                    for (int kk = 0; kk < HD / 16; ++kk)
                        mma_ss(udP, v_k + along_k(kk), q_k + s * kStep + kdO + along_k(kk), id_kk, kk > 0 ? 1u : 0u);
                    mma_commit(smem_u32(&bars->dp_full));
                }
                return true;
            };
            bool ok = bwd_wait_warp(smem_u32(&bars->kv_full), 0, p.wc) && issue_s(0);
            if (ok) ok = issue_dp(0);
            for (int i = 0; i < nt && ok; ++i) {
                const int s = i % QS;
                // dV += P^T dO: P^T (bf16 pairs) in TMEM columns [0,32) for
                // queries 0..63 and [64,96) for queries 64..127
                if (!bwd_wait_warp(smem_u32(&bars->p_ready), i & 1, p.wc)) break;
                tc_fence_after();
                if (leader) {
#pragma unroll
                    for (int kk = 0; kk < BT / 16; ++kk)
                        mma_ts(udV, uS + (kk < 4 ? kk * 8 : 64 + (kk - 4) * 8), q_mn + s * kStep + kdO + kk * (2048 >> 4),
                               id_kmn, (i > 0 || kk > 0) ? 1u : 0u);
                    // dO_i (read by dP_i and dV_i only) is free once dV_i completes
                    if (i + QS < nt) mma_commit(smem_u32(&bars->do_empty[s]));
                }
                if (i + 1 < nt && !issue_s(i + 1)) break;
                // dK += dS^T Q (A = dS^T, K-major view of the dS smem tile)
                if (!bwd_wait_warp(smem_u32(&bars->ds_ready), i & 1, p.wc)) break;
                tc_fence_after();
                if (leader) {
#pragma unroll
                    for (int kk = 0; kk < BT / 16; ++kk)
                        mma_ss(udK, ds_k + along_k(kk), q_mn + s * kStep + kk * (2048 >> 4), id_kmn,
                               (i > 0 || kk > 0) ? 1u : 0u);
                    // Q_i (and its statistics) are free once dK_i completes
                    if (i + QS < nt) mma_commit(smem_u32(&bars->q_empty[s]));
                    if constexpr (HD == 128) {
                        // dQ_i^T = K^T dS^T (A = K, MN-major; B = the dS tile,
                        // MN-major) -> DP columns, head dimension in TMEM lanes,
                        // queries in columns
#pragma unroll
                        for (int kk = 0; kk < BT / 16; ++kk)
                            mma_ss(udP, k_mn + kk * (2048 >> 4), ds_mn + kk * (2048 >> 4), id_dqt, kk > 0 ? 1u : 0u);
                    } else {
                        // dQ_i = dS K (A = dS, MN-major view of the same tile) -> DP columns
#pragma unroll
                        for (int kk = 0; kk < BT / 16; ++kk)
                            mma_ss(udP, ds_mn + kk * (2048 >> 4), k_mn + kk * (2048 >> 4), id_mnmn, kk > 0 ? 1u : 0u);
                    }
                    mma_commit(smem_u32(&bars->dq_full));
                }
                if (i + 1 < nt) {
                    if (!bwd_wait_warp(smem_u32(&bars->dq_free), i & 1, p.wc)) break;
                    tc_fence_after();
                    if (!issue_dp(i + 1)) break;
                }
            }
            if (ok && leader) mma_commit(smem_u32(&bars->acc_done));
            // every MMA issued above completes before TMEM is freed (error paths)
            if (leader) mma_commit(smem_u32(&bars->drain));
            bwd_wait_warp(smem_u32(&bars->drain), 0, p.wc);
        }
    } else if (warp < 12) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 152;");
        // ---------------- compute: two warpgroups split the 128 query columns
        // of S^T/dP^T (64 each) and the HD columns of dQ_i, dK, dV (HD/2 each)
        const int wg = (warp - 4) >> 2;       // 0: first half, 1: second half
        const int quarter = warp & 3;
        const int row = quarter * 32 + lane;  // key row of S^T/dP^T; query row of dQ
        const int cbase = wg * 64;            // first query column of this warpgroup
        // first head-dimension column of this warpgroup (at HD = 128 the same
        // value as cbase, and written so for the compiler)
        const int dbase = HD == 128 ? cbase : wg * (HD / 2);
        const uint32_t pbase = wg * 64;       // TMEM columns of this warpgroup's P^T pairs
        const uint32_t lane_off = (uint32_t)(quarter * 32) << 16;
        const float cl2 = p.scale * 1.4426950408889634f;
        const bool key_valid = tile_has(g, kt, row);
        const int kpos = kbase + row;  // position of this key
        uint8_t *sDS = smem + kDSOff + wg * kBox + row * 128;
        bool ok = nt > 0;

        // per-query statistics of tile i (bulk-copied with Q_i/dO_i):
        // LSE*log2e (+inf past the stripe end, so P = 0 there) and Delta
        auto stat_ptr = [&](int i) -> const float * {
            return reinterpret_cast<const float *>(smem + kStatOff + (i % QS) * kStatBytes) + cbase;
        };
        // P^T of the tile: kept in registers, unrounded, for dS; rounded to
        // bf16 into TMEM as the A operand of dV += P^T dO
        uint32_t P[2][32];
        auto compute_p = [&](int i) -> bool {
            if (!mbar_wait_warp(smem_u32(&bars->q_full[i % QS]), (i / QS) & 1, p.wc)) return false;
            if (!mbar_wait_warp(smem_u32(&bars->s_full), i & 1, p.wc)) return false;
            tc_fence_after();
            const float *sL = stat_ptr(i);
            // keep (query, key) iff key <= query <= key + W - 1, or any later
            // query when the key is a sink; uniform test: all pairs are kept
            const int qt = a_lo + i % cnt, qbase = qt * g.P;
            const bool full = kt < qt && (qbase + g.P - 1 - kbase < p.W || kbase + g.P <= p.sinks);
            const int first = kpos - qbase - cbase;
            const int last = kpos < p.sinks ? 0x7fffffff : kpos - qbase + p.W - 1 - cbase;
            tmem_ld32(tS + lane_off + cbase, P[0]);
            tmem_ld32(tS + lane_off + cbase + 32, P[1]);
            tmem_ld_wait(P[0]);
            tmem_ld_wait(P[1]);
#pragma unroll
            for (int u = 0; u < 64; u += 4) {
                // four row statistics per 16-byte shared-memory load
                const float4 l4 = *reinterpret_cast<const float4 *>(sL + u);
                const float lv[4] = {l4.x, l4.y, l4.z, l4.w};
#pragma unroll
                for (int h = 0; h < 4; ++h) {
                    uint32_t &s1 = P[u / 32][u % 32 + h];
                    s1 = __float_as_uint(ex2(fmaf(__uint_as_float(s1), cl2, -lv[h])));
                }
            }
            if (!full || !key_valid) {
                // clear the pairs that are not kept (whatever their exp gave)
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    const uint32_t kept = key_valid ? kept_bits(32 * c, last, first, 0) : 0u;
#pragma unroll
                    for (int u = 0; u < 32; ++u)
                        if (!(kept & (1u << u))) P[c][u] = 0u;
                }
            }
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                uint32_t pk[16];
#pragma unroll
                for (int u = 0; u < 16; ++u)
                    pk[u] = pack_bf16x2(__uint_as_float(P[c][2 * u]), __uint_as_float(P[c][2 * u + 1]));
                tmem_st16(tS + lane_off + pbase + 16 * c, pk);
            }
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&bars->p_ready));
            return true;
        };

        if (ok) ok = compute_p(0);
        for (int i = 0; i < nt && ok; ++i) {
            // ---- dS = P * (dP - Delta) -> smem (A operand of dQ and dK)
            if (!mbar_wait_warp(smem_u32(&bars->dp_full), i & 1, p.wc)) {
                ok = false;
                break;
            }
            tc_fence_after();
            const float *sD = stat_ptr(i) + 128;
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                uint32_t rr[32];
                tmem_ld32(tdP + lane_off + cbase + 32 * c, rr);
                tmem_ld_wait(rr);
#pragma unroll
                for (int v = 0; v < 4; ++v) {
                    uint32_t w[4];
                    // eight Delta values in two 16-byte loads
                    const float4 d0 = *reinterpret_cast<const float4 *>(sD + 32 * c + 8 * v);
                    const float4 d1 = *reinterpret_cast<const float4 *>(sD + 32 * c + 8 * v + 4);
                    const uint64_t dd[4] = {f2(d0.x, d0.y), f2(d0.z, d0.w), f2(d1.x, d1.y), f2(d1.z, d1.w)};
#pragma unroll
                    for (int h = 0; h < 4; ++h) {
                        const int u = 8 * v + 2 * h;  // query columns u, u + 1
                        // dS = P * (dP - Delta), two at a time
                        const float2 ds = f2_split(
                            mul2(f2(__uint_as_float(P[c][u]), __uint_as_float(P[c][u + 1])),
                                 sub2(f2(__uint_as_float(rr[u]), __uint_as_float(rr[u + 1])), dd[h])));
                        w[h] = pack_bf16x2(ds.x, ds.y);
                    }
                    *reinterpret_cast<uint4 *>(sDS + (((4 * c + v) ^ (row & 7)) * 16)) =
                        make_uint4(w[0], w[1], w[2], w[3]);
                }
            }
            fence_proxy_async_smem();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&bars->ds_ready));
            // ---- P of the next tile while the tensor core runs dQ_i / dK_i
            if (i + 1 < nt && !compute_p(i + 1)) ok = false;
        }
        if (ok) {
            ok = mbar_wait_warp(smem_u32(&bars->acc_done), 0, p.wc);
            tc_fence_after();
        }
        // ---------------- epilogue: this warpgroup's columns of dK, dV
        const int64_t krow = (bh * g.S + (key_valid ? tile_row(g, kt, row) : 0)) * HD + dbase;
        float *part = shared_tile
                          ? p.parts + (((bh * p.nst + kt) * p.slots + slot) * 2 * BT + row) * (int64_t)HD + dbase
                          : nullptr;
#pragma unroll
        for (int which = 0; which < 2; ++which) {
            const uint32_t tacc = which ? tdK : tdV;
            __nv_bfloat16 *outp = which ? p.dk : p.dv;
            const float mul = which ? p.scale : 1.f;
#pragma unroll
            for (int c = 0; c < HD / 64; ++c) {
                uint32_t rr[32];
                if (ok) {
                    tmem_ld32(tacc + lane_off + dbase + c * 32, rr);
                    tmem_ld_wait(rr);
                } else {
#pragma unroll
                    for (int u = 0; u < 32; ++u) rr[u] = 0u;
                }
                if (shared_tile) {
                    float *acc = part + (which ? 0 : BT * HD) + c * 32;
#pragma unroll
                    for (int u = 0; u < 32; u += 8) {
                        uint32_t f8[8];
#pragma unroll
                        for (int i = 0; i < 8; ++i) f8[i] = __float_as_uint(__uint_as_float(rr[u + i]) * mul);
                        st_global_32(acc + u, f8, true);  // the workspace is 256-byte aligned
                    }
                } else if (key_valid) {
                    __nv_bfloat16 *dst = outp + krow + c * 32;
#pragma unroll
                    for (int v = 0; v < 2; ++v) {
                        uint32_t o8[8];
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            o8[i] = pack_bf16x2(__uint_as_float(rr[16 * v + 2 * i]) * mul,
                                                __uint_as_float(rr[16 * v + 2 * i + 1]) * mul);
                        st_global_32(dst + 16 * v, o8, p.wide);
                    }
                }
            }
        }
    } else {
        // ---------------- dQ_i out of tensor memory into the fp32 accumulator
        asm volatile("setmaxnreg.inc.sync.aligned.u32 152;");
        const int quarter = warp & 3;
        const int row = quarter * 32 + lane;  // TMEM lane
        const uint32_t lane_off = (uint32_t)(quarter * 32) << 16;
        // Accumulator tile in groups of four columns of dQ_i as it lies in
        // tensor memory: [column / 4][lane][4], so a reduction instruction of
        // the warp covers 512 whole bytes.  HD = 128: lane = dimension,
        // column = query; HD = 64: lane = query, column = dimension.
        constexpr int kCols = HD == 128 ? BT : HD;
        for (int i = 0; i < nt; ++i) {
            if (!mbar_wait_warp(smem_u32(&bars->dq_full), i & 1, p.wc)) break;
            tc_fence_after();
            uint32_t q[kCols / 32][32];
#pragma unroll
            for (int c = 0; c < kCols / 32; ++c) tmem_ld32(tdP + lane_off + 32 * c, q[c]);
#pragma unroll
            for (int c = 0; c < kCols / 32; ++c) tmem_ld_wait(q[c]);
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&bars->dq_free));
            float *dst = p.dq_acc + ((bh * G + i / cnt) * g.nt + a_lo + i % cnt) * BT * HD + row * 4;
#pragma unroll
            for (int c = 0; c < kCols / 32; ++c)
#pragma unroll
                for (int u = 0; u < 32; u += 4)
                    red_add_v4(dst + (8 * c + u / 4) * BT * 4, __uint_as_float(q[c][u]), __uint_as_float(q[c][u + 1]),
                               __uint_as_float(q[c][u + 2]), __uint_as_float(q[c][u + 3]));
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

// Four rows of the padded tiles per warp, eight lanes each: HD/8 elements a
// lane in 16-byte vectors that the eight lanes read side by side.
template <int HD>
__global__ void __launch_bounds__(256)
    window_pre_kernel(const __nv_bfloat16 *__restrict__ o, const __nv_bfloat16 *__restrict__ dO,
                      const float *__restrict__ lse, float *__restrict__ stats, float *__restrict__ dq_acc,
                      const PosGeom g, int64_t padded_rows) {
    constexpr int V = HD / 64;  // 16-byte vectors of a lane
    const int lane = threadIdx.x & 31, sub = lane & 7;
    const int64_t stride = (int64_t)gridDim.x * (blockDim.x >> 3);
    let_next_begin();
    for (int64_t pr = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) >> 3; pr < padded_rows; pr += stride) {
        const int64_t blk = pr >> 7;  // bh * nt + t
        const int r = (int)(pr & 127);
        const int64_t bh = blk / g.nt;
        const int t = (int)(blk - bh * g.nt);
        const bool real = tile_has(g, t, r);
        const int64_t row = bh * g.S + (real ? tile_row(g, t, r) : 0);
        uint4 x[V], y[V];
        float ls = 0.f;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            x[v] = y[v] = make_uint4(0u, 0u, 0u, 0u);
            if (real) {
                x[v] = reinterpret_cast<const uint4 *>(o + row * HD)[8 * v + sub];
                y[v] = reinterpret_cast<const uint4 *>(dO + row * HD)[8 * v + sub];
            }
        }
        if (real && sub == 0) ls = lse[row];
        float4 *z = reinterpret_cast<float4 *>(dq_acc + pr * HD) + sub;
#pragma unroll
        for (int v = 0; v < HD / 32; ++v) z[8 * v] = make_float4(0.f, 0.f, 0.f, 0.f);
        float sum = 0.f;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const __nv_bfloat162 *a = reinterpret_cast<const __nv_bfloat162 *>(&x[v]);
            const __nv_bfloat162 *b = reinterpret_cast<const __nv_bfloat162 *>(&y[v]);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 c = __bfloat1622float2(a[i]), d = __bfloat1622float2(b[i]);
                sum = fmaf(c.x, d.x, sum);
                sum = fmaf(c.y, d.y, sum);
            }
        }
#pragma unroll
        for (int off = 4; off; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
        if (sub == 0) {
            float *st = stats + (blk << 8) + r;
            st[0] = real ? ls * 1.4426950408889634f : INFINITY;
            st[128] = sum;
        }
    }
}

// dQ = bf16(scale * accumulator) from tile order to the placement's rows.
// HD = 128: a warp takes 4 rows, stored [dimension][4]; lane l has dimensions
// 4l .. 4l+3 of each.  HD = 64: a thread takes a row, stored [D / 4][row][4].
template <int HD>
__global__ void __launch_bounds__(256)
    window_post_kernel(const float *dq_acc, __nv_bfloat16 *dq, const PosGeom g,
                       int64_t padded_rows, float scale) {
    constexpr int T = HD == 128 ? 32 : 1, kRows = HD == 128 ? 4 : 1;
    const int64_t stride = (int64_t)gridDim.x * blockDim.x / T * kRows;
    const int part = threadIdx.x % T;
    let_next_begin();
    wait_for_previous();
    for (int64_t pr = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) / T * kRows; pr < padded_rows; pr += stride) {
        const int64_t blk = pr >> 7;
        const int r = (int)(pr & 127);
        const int64_t bh = blk / g.nt;
        const int t = (int)(blk - bh * g.nt);
        if (!tile_has(g, t, r)) continue;  // later rows of the four lie behind it too
        const float4 *src = reinterpret_cast<const float4 *>(dq_acc + blk * BT * HD);
        if constexpr (HD == 128) {
            float v[4][4];
#pragma unroll
            for (int d = 0; d < 4; ++d) {
                const float4 x = src[r / 4 * HD + 4 * part + d];
                v[0][d] = x.x, v[1][d] = x.y, v[2][d] = x.z, v[3][d] = x.w;
            }
#pragma unroll
            for (int q = 0; q < 4; ++q)
                if (tile_has(g, t, r + q))
                    reinterpret_cast<uint2 *>(dq + (bh * g.S + tile_row(g, t, r + q)) * HD)[part] =
                        make_uint2(pack_bf16x2(v[q][0] * scale, v[q][1] * scale),
                                   pack_bf16x2(v[q][2] * scale, v[q][3] * scale));
        } else {
            uint4 *dst = reinterpret_cast<uint4 *>(dq + (bh * g.S + tile_row(g, t, r)) * HD);
#pragma unroll
            for (int d = 0; d < HD / 4; d += 2) {
                const float4 x = src[d * BT + r], y = src[(d + 1) * BT + r];
                dst[d / 2] = make_uint4(pack_bf16x2(x.x * scale, x.y * scale), pack_bf16x2(x.z * scale, x.w * scale),
                                        pack_bf16x2(y.x * scale, y.y * scale), pack_bf16x2(y.z * scale, y.w * scale));
            }
        }
    }
}

// dK and dV of the sink tiles: the units' shares in turn.  One block per
// (key/value head, sink tile, 8 rows): HD/4 threads a row, 4 elements each.
template <int HD>
__global__ void __launch_bounds__(8 * HD / 4)
    window_sink_kernel(const WinBwdParams p) {
    wait_for_previous();  // and with it for the kernel before, which that one waited for
    const PosGeom &g = p.g;
    const int tile = blockIdx.x / (BT / 8);
    const int64_t bh = tile / p.nst;
    const int kt = tile % p.nst;
    const int row = blockIdx.x % (BT / 8) * 8 + threadIdx.x / (HD / 4), col = threadIdx.x % (HD / 4) * 4;
    if (!tile_has(g, kt, row)) return;
    const int n = 1 + far_units(g, kt, p.W, p.chunk);
    const float *src = p.parts + ((bh * p.nst + kt) * p.slots * 2 * BT + row) * (int64_t)HD + col;
    float4 a[2] = {make_float4(0.f, 0.f, 0.f, 0.f), make_float4(0.f, 0.f, 0.f, 0.f)};
#pragma unroll 4
    for (int s = 0; s < n; ++s, src += 2 * BT * HD)
#pragma unroll
        for (int w = 0; w < 2; ++w) {
            const float4 v = *reinterpret_cast<const float4 *>(src + w * BT * HD);
            a[w].x += v.x, a[w].y += v.y, a[w].z += v.z, a[w].w += v.w;
        }
    const int64_t at = (bh * g.S + tile_row(g, kt, row)) * HD + col;
    *reinterpret_cast<uint2 *>(p.dk + at) = make_uint2(pack_bf16x2(a[0].x, a[0].y), pack_bf16x2(a[0].z, a[0].w));
    *reinterpret_cast<uint2 *>(p.dv + at) = make_uint2(pack_bf16x2(a[1].x, a[1].y), pack_bf16x2(a[1].z, a[1].w));
}

// Work units and workspace of a problem; false if it is too large.
struct WinBwdPlan {
    WinBwdParams p;
    int64_t padded_rows;
    size_t dq_bytes, stat_bytes, part_bytes;
};

bool window_bwd_plan(WinBwdPlan *plan, const WindowArgs &a) {
    WinBwdParams &p = plan->p;
    p = WinBwdParams{};
    if (!pos_geom(&p.g, a.S, a.N, a.layout)) return false;
    const PosGeom &g = p.g;
    p.W = (int)(a.window < a.S ? a.window : a.S);
    p.sinks = (int)(a.sinks < a.S ? a.sinks : a.S);
    p.nst = (p.sinks + g.P - 1) / g.P;
    // a far unit is as long as a key tile's window, or longer where that
    // would make more than 64 shares of a sink tile
    const int span = p.W / g.P + 2, most = (g.nt + 63) / 64;
    p.chunk = span > most ? span : most;
    int64_t units = g.nt;
    for (int kt = 0; kt < p.nst; ++kt) units += far_units(g, kt, p.W, p.chunk);
    p.slots = units > g.nt ? 1 + far_units(g, 0, p.W, p.chunk) : 0;
    // one-dimensional grids of the units and of the sink tiles' rows
    const int64_t most_units = 0x7fffffffll / (a.B * a.Hkv);
    if (units > most_units || (p.slots > 0 && p.nst * (BT / 8) > most_units)) return false;
    p.units = (int)units;
    p.G = (int)(a.H / a.Hkv);
    p.scale = a.scale;
    plan->padded_rows = a.B * a.H * g.nt * (int64_t)BT;
    plan->dq_bytes = (size_t)plan->padded_rows * a.D * 4;
    plan->stat_bytes = (size_t)plan->padded_rows * 8;
    plan->part_bytes = (size_t)(a.B * a.Hkv * p.nst) * p.slots * 2 * BT * a.D * 4;
    return true;
}

template <int HD>
int launch_window_bwd_hd(const void *q, const void *k, const void *v, const void *o, const float *lse, const void *dO,
                         void *dq, void *dk, void *dv, void *workspace, const WindowArgs &a, cudaStream_t stream) {
    constexpr size_t kSmemBytes = WinBwdCfg<HD>::kSmemBytes;
    static PerDeviceOnce attr_once;
    const int attr = attr_once.get([] {
        return cuda_status(cudaFuncSetAttribute(tc_window_bwd_kernel<HD>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                (int)kSmemBytes));
    });
    if (attr != STRIPED_OK) return attr;
    WinBwdPlan plan;
    if (!window_bwd_plan(&plan, a)) return STRIPED_ERR_UNSUPPORTED;
    WinBwdParams &p = plan.p;
    char *ws = static_cast<char *>(workspace);
    float *dq_acc = reinterpret_cast<float *>(ws), *stats = reinterpret_cast<float *>(ws + plan.dq_bytes);
    p.dq_acc = dq_acc;
    p.stats = stats;
    p.parts = reinterpret_cast<float *>(ws + plan.dq_bytes + plan.stat_bytes);
    p.dk = static_cast<__nv_bfloat16 *>(dk);
    p.dv = static_cast<__nv_bfloat16 *>(dv);
    p.wide = ((reinterpret_cast<uintptr_t>(dk) | reinterpret_cast<uintptr_t>(dv)) & 31u) == 0;
    p.wc = device_wait_ctl();
    const int64_t bh = a.B * a.H, bh_kv = a.B * a.Hkv;
    CUtensorMap mq, mk, mv, mdo;
    int st;
    if ((st = make_pos_map(&mq, q, a.D, p.g, bh)) || (st = make_pos_map(&mk, k, a.D, p.g, bh_kv)) ||
        (st = make_pos_map(&mv, v, a.D, p.g, bh_kv)) || (st = make_pos_map(&mdo, dO, a.D, p.g, bh)))
        return st;
    const int blocks = device_sm_count() * 8;
    window_pre_kernel<HD><<<blocks, 256, 0, stream>>>((const __nv_bfloat16 *)o, (const __nv_bfloat16 *)dO, lse, stats,
                                                      dq_acc, p.g, plan.padded_rows);
    if ((st = cuda_status(cudaGetLastError()))) return st;
    if ((st = launch_after(tc_window_bwd_kernel<HD>, dim3((unsigned)(p.units * bh_kv)), kThreads, kSmemBytes, stream, mq,
                           mk, mv, mdo, p)))
        return st;
    st = launch_after(window_post_kernel<HD>, dim3((unsigned)blocks), 256, 0, stream, dq_acc, (__nv_bfloat16 *)dq, p.g,
                      plan.padded_rows, a.scale);
    if (st || p.slots == 0) return st;
    return launch_after(window_sink_kernel<HD>, dim3((unsigned)(bh_kv * p.nst * (BT / 8))), 8 * HD / 4, 0, stream, p);
}

}  // namespace

size_t window_bwd_workspace(const WindowArgs &a) {
    WinBwdPlan plan;
    if (!window_bwd_plan(&plan, a)) return 0;
    return plan.dq_bytes + plan.stat_bytes + plan.part_bytes;
}

int launch_tc_window_bwd(const void *q, const void *k, const void *v, const void *o, const float *lse, const void *dO,
                         void *dq, void *dk, void *dv, void *workspace, const WindowArgs &a, cudaStream_t stream) {
    return a.D == 128 ? launch_window_bwd_hd<128>(q, k, v, o, lse, dO, dq, dk, dv, workspace, a, stream)
                      : launch_window_bwd_hd<64>(q, k, v, o, lse, dO, dq, dk, dv, workspace, a, stream);
}

}  // namespace striped
