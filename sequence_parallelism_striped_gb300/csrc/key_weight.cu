// key_weight.cu -- the attention weight that every key of a prompt got, summed
// over its queries and over the query heads that share the key, bf16 on tcgen05:
//     w[t] = sum over heads h of the group, positions p >= max(t, first) of
//            exp(scale q_{h,p} . k_t - lse_{h,p}).
//
// The product is formed transposed, S^T = K Q^T: a lane of tensor memory is a
// key, so a thread sums its key's weights over a tile's 128 queries in its own
// registers, and nothing is exchanged until the key tile is done.  Only the
// log-sum-exp runs along the columns; two warps gather it from the placed
// rows into shared memory.
//
// The bytes are few; per tile of 128 x 128 at D = 128 the products take 512 clocks,
// the exponentials 512 (8 a clock and quarter).  Measured, 32 + 8 heads, all
// queries of S = 16384: 860 us, 1,279 TFLOP/s of kept products (67 % of the
// tensor core's burst), 950 clocks a tile at 2070 MHz (call after call 895 to 907:
// the power cap takes the clock to about 1950): a warp sums 32 columns in about 260
// clocks, half of them its exponentials, and two warps a quarter do not hide the
// hand-offs (a third group: 990 us, four for 32 columns each: 1,080; without
// exponentials 785, without products 870).  The last 64 queries of S = 65536: 65
// us, 2.1 TB/s: 14 items of four half tiles a multiprocessor, for which all
// multiprocessors read the same few query tiles.
//
// One CTA per multiprocessor.  Two neighbouring key tiles are one item, which goes
// over the query tiles together, a group of warps for each; all (item, head,
// query tile) triples of the call are cut into shares of equal length, one per
// CTA.  An item whose triples lie in several shares leaves partial sums, which a
// second kernel adds in order: no atomics, the same result in every run.  A key's
// sum runs over its queries in fp32, and a log-sum-exp is rounded once more in
// units of log2: weights of all queries of S = 16384 are 3.0e-7 off in the root mean
// square (elementary operations in fp32: 0.8e-7).
//
//   warp 0       TMA producer: K tile of an item, Q tiles
//   warp 1       TMEM allocator + tcgen05.mma issuer (one elected lane)
//   warps 2, 3   log-sum-exp of the query tiles
//   warps 4..11  two groups, one for each key tile; thread t of a group owns key t
//   warps 12..15 K tiles from shared to tensor memory: as the left operand they are
//                read there, and a product takes half the bytes from shared
//                memory (both operands from there: 512 clocks a tile of its
//                bandwidth, beside TMA's and the log-sum-exp's)
// Tensor memory: three S^T of 128 columns, taken in turn, two K tiles.
#include <math.h>

#include <type_traits>

#include "common.cuh"
#include "internal.h"
#include "window.cuh"

namespace striped {

namespace {

constexpr int KT = 128;
constexpr uint32_t kWBox = 128 * 128;  // 128 rows x 64 bf16
constexpr int kWtThreads = 512;
constexpr int kSBufs = 3;
// Log-sum-exp buffers: an even number, so that each is filled by one of the two
// warps alone.  (A wait tells a phase from the next one only; whoever could be
// two phases ahead or behind must not wait there.)
constexpr int kLBufs = 4;

template <int HD>
struct WeightCfg {
    static constexpr int NS = HD == 128 ? 3 : 6;  // Q stages
    static constexpr int NK = HD == 128 ? 3 : 6;  // K tiles
    static constexpr uint32_t kTile = (HD / 64) * kWBox;
    static constexpr uint32_t kKOff = NS * kTile;
    static constexpr uint32_t kLseOff = kKOff + NK * kTile;
    static constexpr uint32_t kBarOff = kLseOff + kLBufs * KT * 4;
    static constexpr size_t kSmemBytes = 1024 + kBarOff + 512;
    static_assert(kSmemBytes <= 232448, "shared memory over the per-block limit");
};

template <int NS, int NK>
struct WeightBars {
    uint64_t k_full[NK], k_empty[NK];  // in shared memory
    uint64_t kt_full, kt_empty;        // in tensor memory
    uint64_t q_full[NS], q_empty[NS];
    uint64_t s_full[kSBufs], s_empty[kSBufs];
    uint64_t lse_full[kLBufs], lse_empty[kLBufs];
    uint64_t drain;
    uint32_t tmem_slot;
};

struct WeightParams {
    PosGeom g;
    int64_t total;        // triples of the call
    int parts;            // CTAs
    int H, Hkv, G;
    int first, f0;        // first query that counts, its tile
    float scale;
    int accumulate;
    const float *lse;
    float *weight;
    float *part;          // [parts][2][2 KT]: of a CTA's first and last item
    WaitCtl wc;
};

// Triples of a key/value head before its item kp (key tiles 2 kp and 2 kp + 1), over
// the group's heads; the queries of an item begin at the tile of its first key,
// or at f0.
__host__ __device__ __forceinline__ int64_t weight_before(const PosGeom &g, int f0, int G, int64_t kp) {
    const int64_t nt = g.nt, f = f0, kf = f / 2 + 1;  // items that begin at f0
    if (kp <= kf) return G * kp * (nt - f);
    return G * (kf * (nt - f) + (kp - kf) * nt - (kp * (kp - 1) - kf * (kf - 1)));
}
__host__ __device__ __forceinline__ int weight_items(const PosGeom &g) { return (g.nt + 1) / 2; }

__host__ __device__ __forceinline__ int64_t weight_share(const WeightParams &p, int c) {
    return p.total / p.parts * c + p.total % p.parts * c / p.parts;
}

// The stretch [n0, n1) of the triples of one item that begins at x; next() goes
// on to the one behind it.
struct WeightItem {
    int64_t x;
    int line, kp;       // key/value head of the batch, item
    int qlo, cnt, all;  // first query tile, query tiles, triples
    int n0, n1;
    __device__ __forceinline__ WeightItem(const WeightParams &p, int64_t from, int64_t x1) {
        x = from;
        const int64_t per = weight_before(p.g, p.f0, p.G, weight_items(p.g));
        line = (int)(x / per);
        const int64_t in = x - line * per;
        int a = 0, b = weight_items(p.g) - 1;
        while (a < b) {
            const int m = (int)(((int64_t)a + b + 1) >> 1);
            if (weight_before(p.g, p.f0, p.G, m) <= in) a = m;
            else b = m - 1;
        }
        kp = a;
        n0 = (int)(in - weight_before(p.g, p.f0, p.G, kp));
        sizes(p, x1);
    }
    __device__ __forceinline__ void next(const WeightParams &p, int64_t x1) {
        x += n1 - n0;
        n0 = 0;
        if (++kp == weight_items(p.g)) kp = 0, ++line;
        sizes(p, x1);
    }
    __device__ __forceinline__ bool has(const WeightParams &p, int h) const { return 2 * kp + h < p.g.nt; }

  private:
    __device__ __forceinline__ void sizes(const WeightParams &p, int64_t x1) {
        qlo = max(2 * kp, p.f0);
        cnt = p.g.nt - qlo;
        all = p.G * cnt;
        n1 = (int)min((int64_t)all, n0 + (x1 - x));
    }
};

__device__ __forceinline__ void write_weight(const WeightParams &p, int line, int kt, int r, float sum) {
    if (kt >= p.g.nt || !tile_has(p.g, kt, r)) return;
    float *dst = p.weight + (int64_t)line * p.g.S + tile_row(p.g, kt, r);
    *dst = p.accumulate ? *dst + sum : sum;
}

template <int HD>
__global__ void __launch_bounds__(kWtThreads, 1)
    tc_key_weight_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                         const WeightParams p) {
    using Cfg = WeightCfg<HD>;
    constexpr int NS = Cfg::NS, NK = Cfg::NK, kBoxes = HD / 64;
    constexpr uint32_t kTile = Cfg::kTile, kKCol = kSBufs * KT;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem =
        reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    WeightBars<NS, NK> *bars = reinterpret_cast<WeightBars<NS, NK> *>(smem + Cfg::kBarOff);
    float *lse_s = reinterpret_cast<float *>(smem + Cfg::kLseOff);
    const uint32_t sbase = smem_u32(smem);
    const PosGeom &g = p.g;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;

    if (threadIdx.x == 0) {
        for (int i = 0; i < NK; ++i) {
            mbar_init(smem_u32(&bars->k_full[i]), 1);
            mbar_init(smem_u32(&bars->k_empty[i]), 4);
        }
        mbar_init(smem_u32(&bars->kt_full), 4);
        mbar_init(smem_u32(&bars->kt_empty), 1);
        for (int s = 0; s < NS; ++s) {
            mbar_init(smem_u32(&bars->q_full[s]), 1);
            mbar_init(smem_u32(&bars->q_empty[s]), 1);
        }
        for (int i = 0; i < kSBufs; ++i) {
            mbar_init(smem_u32(&bars->s_full[i]), 1);
            mbar_init(smem_u32(&bars->s_empty[i]), 4);
        }
        for (int i = 0; i < kLBufs; ++i) {
            mbar_init(smem_u32(&bars->lse_full[i]), 1);
            mbar_init(smem_u32(&bars->lse_empty[i]), 8);
        }
        mbar_init(smem_u32(&bars->drain), 1);
        fence_barrier_init();
    }
    if (g.P < KT) {
        // rows past a tile's positions are never loaded: a query there counts
        // nothing only if its scores are finite
        for (uint32_t i = threadIdx.x * 16; i < Cfg::kLseOff; i += kWtThreads * 16)
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
    const uint32_t tmem = bars->tmem_slot;
    const int64_t x0 = weight_share(p, blockIdx.x), x1 = weight_share(p, blockIdx.x + 1);
    const int nx = (int)(x1 - x0);

    if (warp == 0 && lane == 0) {
        // ---------------- TMA producer
        const bool skip_first = p.wc.inject == kInjectFwdSkipKV;  // test hook: the first K tile is never loaded
        const uint32_t bytes = (uint32_t)g.P * 128 * kBoxes;
        int j = 0, kn = 0, kdone = 0;  // query tiles; K tiles asked for, and those of the items begun
        bool ok = true;
        WeightItem kit(p, x0, x1);
        int kh = 0;
        for (WeightItem it(p, x0, x1); it.x < x1 && ok; it.next(p, x1)) {
            // this item's K tiles, and of the next ones as many as there is room for
            kdone += it.has(p, 1) ? 2 : 1;
            while (kit.x < x1) {
                const int ks = kn % NK;
                if (kn >= NK) {
                    const uint32_t bar = smem_u32(&bars->k_empty[ks]), phase = ((kn / NK) + 1) & 1;
                    if (kn < kdone ? !mbar_wait(bar, phase, p.wc) : !mbar_try_wait(bar, phase)) {
                        ok = kn >= kdone;
                        break;
                    }
                }
                if (!(skip_first && kn == 0)) {
                    const TileAt at = tile_at(g, 2 * kit.kp + kh);
                    const uint32_t fb = smem_u32(&bars->k_full[ks]), dst = sbase + Cfg::kKOff + ks * kTile;
                    mbar_arrive_expect_tx(fb, bytes);
#pragma unroll
                    for (int c = 0; c < kBoxes; ++c)
                        tma_load_4d(dst + c * kWBox, &tmK, fb, 64 * c, at.c1, at.c2, kit.line);
                }
                ++kn;
                if (kh == 0 && kit.has(p, 1)) kh = 1;
                else kh = 0, kit.next(p, x1);
            }
            if (!ok) break;
            const int b = it.line / p.Hkv, hkv = it.line - b * p.Hkv;
            int head = b * p.H + hkv * p.G + it.n0 / it.cnt, qt = it.qlo + it.n0 % it.cnt;
            for (int n = it.n0; n < it.n1; ++n, ++j) {
                const int s = j % NS;
                if (j >= NS && !mbar_wait(smem_u32(&bars->q_empty[s]), ((j / NS) + 1) & 1, p.wc)) {
                    ok = false;
                    break;
                }
                const TileAt at = tile_at(g, qt);
                const uint32_t fb = smem_u32(&bars->q_full[s]), dst = sbase + s * kTile;
                mbar_arrive_expect_tx(fb, bytes);
#pragma unroll
                for (int c = 0; c < kBoxes; ++c) tma_load_4d(dst + c * kWBox, &tmQ, fb, 64 * c, at.c1, at.c2, head);
                if (++qt == g.nt) qt = it.qlo, ++head;
            }
        }
        // the last load of each stage has landed before the CTA exits
        for (int t = j > NS ? j - NS : 0; t < j; ++t) mbar_wait(smem_u32(&bars->q_full[t % NS]), (t / NS) & 1, p.wc);
        for (int t = kn > NK ? kn - NK : 0; t < kn; ++t)
            if (!(skip_first && t == 0)) mbar_wait(smem_u32(&bars->k_full[t % NK]), (t / NK) & 1, p.wc);
    } else if (warp == 1) {
        // ---------------- MMA issuer (the whole warp, one lane issues)
        const bool leader = elect_one();
        const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
        const uint64_t dq = sdesc_sw128(sbase, 16, 1024);
        int j = 0, seg = 0;
        bool ok = true;
        for (WeightItem it(p, x0, x1); it.x < x1 && ok; it.next(p, x1), ++seg) {
            ok = mbar_wait_warp(smem_u32(&bars->kt_full), seg & 1, p.wc);
            int qt = it.qlo + it.n0 % it.cnt;
            for (int n = it.n0; n < it.n1 && ok; ++n, ++j) {
                const int s = j % NS, at = qt;
                ok = mbar_wait_warp(smem_u32(&bars->q_full[s]), (j / NS) & 1, p.wc);
                // queries before `first` in its tile are left out, 32 at a time
                const int skip = at == p.f0 ? (p.first - at * g.P) / 32 : 0;
                if (++qt == g.nt) qt = it.qlo;
                const uint32_t idesc = idesc_bf16_f32(KT, KT, false, false) - ((uint32_t)(skip * 32 / 8) << 17);
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int i = 2 * j + h, u = i % kSBufs;
                    if (ok && i >= kSBufs) ok = mbar_wait_warp(smem_u32(&bars->s_empty[u]), ((i / kSBufs) + 1) & 1, p.wc);
                    if (!ok) break;
                    tc_fence_after();
                    if (leader) {
                        const uint64_t db = dq + s * (kTile >> 4) + (skip * 32 * 128 >> 4);
                        if (it.has(p, h) && at >= 2 * it.kp + h)  // else no key of the tile is kept
#pragma unroll
                            for (int kk = 0; kk < HD / 16; ++kk)
                                mma_ts(tm + 128 * u + 32 * skip, tm + kKCol + h * (HD / 2) + kk * 8,
                                       db + (((kk >> 2) * kWBox + (kk & 3) * 32) >> 4), idesc, kk > 0 ? 1u : 0u);
                        // only what will be refilled is released
                        if (h && j + NS < nx) mma_commit(smem_u32(&bars->q_empty[s]));
                        mma_commit(smem_u32(&bars->s_full[u]));
                        if (h && n + 1 == it.n1 && it.x + (it.n1 - it.n0) < x1) mma_commit(smem_u32(&bars->kt_empty));
                    }
                }
            }
        }
        // every MMA issued above completes before TMEM is freed
        if (leader) mma_commit(smem_u32(&bars->drain));
        mbar_wait_warp(smem_u32(&bars->drain), 0, p.wc);
    } else if (warp == 2 || warp == 3) {
        // ---------------- log-sum-exp of the query tiles: negative, in units of
        // log2, -infinity for queries that do not count.  Warps 2 and 3 take every
        // other tile and read two of theirs ahead (read when its buffer is free,
        // a tile waits for memory: 2.4 instead of 1.1 ms at S = 16384)
        WeightItem it(p, x0, x1);
        int n = it.n0, at = 0;  // the walk stands at tile `at` of the CTA, triple n of its item
        int b = it.line / p.Hkv, head = b * p.H + (it.line - b * p.Hkv) * p.G + it.n0 / it.cnt, qt = it.qlo + it.n0 % it.cnt;
        int off[4];             // rows of this lane's queries, from the tile's first row
#pragma unroll
        for (int i = 0; i < 4; ++i) off[i] = (int)tile_row(g, 0, lane + 32 * i);
        auto step = [&]() {
            ++at;
            if (++n == it.n1) {
                it.next(p, x1);
                if (it.x >= x1) return;
                n = it.n0;
                b = it.line / p.Hkv;
                head = b * p.H + (it.line - b * p.Hkv) * p.G + it.n0 / it.cnt;
                qt = it.qlo + it.n0 % it.cnt;
            } else if (++qt == g.nt) {
                qt = it.qlo;
                ++head;
            }
        };
        auto read = [&](float (&v)[4]) {  // the tile that the walk stands at, then two on
            if (at >= nx) return;
            const float *src = p.lse + (int64_t)head * g.S + tile_row(g, qt, 0);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int r = lane + 32 * i;
                const bool on = tile_has(g, qt, r) && qt * g.P + r >= p.first;
                v[i] = on ? __ldg(src + off[i]) : INFINITY;
            }
            step();
            if (at < nx) step();
        };
        auto put = [&](int j, const float (&v)[4]) -> bool {
            const int u = j % kLBufs;
            if (j >= kLBufs && !mbar_wait_warp(smem_u32(&bars->lse_empty[u]), ((j / kLBufs) + 1) & 1, p.wc)) return false;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                lse_s[u * KT + lane + 32 * i] = v[i] == -INFINITY ? v[i] : -1.4426950408889634f * v[i];
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&bars->lse_full[u]));
            return true;
        };
        float v0[4], v1[4];
        if (warp == 3) step();
        read(v0);
        read(v1);
        for (int j = warp - 2; j < nx; j += 4) {
            if (!put(j, v0)) break;
            read(v0);
            if (j + 2 >= nx || !put(j + 2, v1)) break;
            read(v1);
        }
    } else if (warp >= 12) {
        // ---------------- K tiles: shared -> tensor memory
        const int r = (warp & 3) * 32 + lane;
        const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
        int seg = 0, kn = 0;
        bool ok = true;
        for (WeightItem it(p, x0, x1); it.x < x1 && ok; it.next(p, x1), ++seg) {
#pragma unroll 1
            for (int h = 0; h < (it.has(p, 1) ? 2 : 1); ++h, ++kn) {
                const int kb = kn % NK;
                ok = mbar_wait_warp(smem_u32(&bars->k_full[kb]), (kn / NK) & 1, p.wc);
                if (!ok) break;
                const uint8_t *src = smem + Cfg::kKOff + kb * kTile + r * 128;
                uint32_t k[HD / 64][32];
#pragma unroll
                for (int c = 0; c < kBoxes; ++c)
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const uint4 w = *reinterpret_cast<const uint4 *>(src + c * kWBox + ((i ^ (r & 7)) * 16));
                        k[c][4 * i] = w.x, k[c][4 * i + 1] = w.y, k[c][4 * i + 2] = w.z, k[c][4 * i + 3] = w.w;
                    }
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&bars->k_empty[kb]));
                if (h == 0 && seg > 0) {  // the last item's products have read theirs
                    ok = mbar_wait_warp(smem_u32(&bars->kt_empty), (seg + 1) & 1, p.wc);
                    if (!ok) break;
                }
                tc_fence_after();
#pragma unroll
                for (int c = 0; c < kBoxes; ++c) tmem_st32(tmem + kKCol + h * (HD / 2) + 32 * c + lane_off, k[c]);
            }
            if (!ok) break;
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&bars->kt_full));
        }
    } else if (warp >= 4) {
        // ---------------- weights of the keys
        const int group = (warp - 4) >> 2, quarter = warp & 3;
        const int r = quarter * 32 + lane;
        const uint32_t lane_off = (uint32_t)(quarter * 32) << 16;
        const float cl2 = p.scale * 1.4426950408889634f;
        const uint64_t cl2x2 = f2(cl2, cl2);
        bool ok = true;
        // the group's products are every second one: their buffer and its phase
        int j = 0, u = group, phase = 0;
        for (WeightItem it(p, x0, x1); it.x < x1 && ok; it.next(p, x1)) {
            float sum = 0.f;
            const int kt = 2 * it.kp + group;
            const bool has = kt < g.nt;
            int qt = it.qlo + it.n0 % it.cnt;
            for (int n = it.n0; n < it.n1; ++n, ++j) {
                const int at = qt;
                if (++qt == g.nt) qt = it.qlo;
                const int lb = j % kLBufs;
                const uint32_t lse_bar = smem_u32(&bars->lse_full[lb]), s_bar = smem_u32(&bars->s_full[u]);
                const bool l_ok = mbar_try_wait(lse_bar, (j / kLBufs) & 1), s_ok = mbar_try_wait(s_bar, phase);
                if (!__all_sync(0xffffffffu, l_ok && s_ok) &&
                    (!mbar_wait_warp(lse_bar, (j / kLBufs) & 1, p.wc) || !mbar_wait_warp(s_bar, phase, p.wc))) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const float4 *lse4 = reinterpret_cast<const float4 *>(lse_s + lb * KT);
                const uint32_t src = tmem + 128 * u + lane_off;
                uint64_t acc[4] = {0ull, 0ull, 0ull, 0ull};
                // 32 columns; in the keys' own tile the first ones that a warp
                // looks at are cut along the diagonal
                auto add = [&](int c, auto cut, bool last) {
                    uint32_t s[32];
                    tmem_ld32(src + 32 * c, s);
                    float4 l4[8];  // all on their way before the first is used
#pragma unroll
                    for (int i = 0; i < 8; ++i) l4[i] = lse4[8 * c + i];
                    tmem_ld_wait(s);
                    if (last) {
                        // the buffers are read: products and log-sum-exps may go on
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) {
                            mbar_arrive(smem_u32(&bars->s_empty[u]));
                            mbar_arrive(smem_u32(&bars->lse_empty[lb]));
                        }
                    }
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float4 l = l4[i];
                        const float2 a = f2_split(
                            fma2(f2(__uint_as_float(s[4 * i]), __uint_as_float(s[4 * i + 1])), cl2x2, f2(l.x, l.y)));
                        const float2 b = f2_split(fma2(
                            f2(__uint_as_float(s[4 * i + 2]), __uint_as_float(s[4 * i + 3])), cl2x2, f2(l.z, l.w)));
                        float e[4] = {ex2(a.x), ex2(a.y), ex2(b.x), ex2(b.y)};
                        if constexpr (decltype(cut)::value)
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                if (4 * i + k < lane) e[k] = 0.f;
                        acc[(2 * i) & 3] = add2(acc[(2 * i) & 3], f2(e[0], e[1]));
                        acc[(2 * i + 1) & 3] = add2(acc[(2 * i + 1) & 3], f2(e[2], e[3]));
                    }
                };
                if (has && at > kt && at != p.f0 && at + 1 != g.nt) {
#pragma unroll
                    for (int c = 0; c < KT / 32; ++c) add(c, std::false_type{}, c == KT / 32 - 1);
                } else {
                    // columns that count for some key of this warp: queries from
                    // `first` and, in the keys' own tile, from the warp's first key
                    const bool diag = at == kt;
                    int c = max(max(0, p.first - at * g.P) / 32, diag ? quarter : 0);
                    const int c1 = has && at >= kt ? (min(g.P, g.S - at * g.P) + 31) / 32 : 0;
                    if (diag && c == quarter && c < c1) add(c++, std::true_type{}, false);
#pragma unroll 1
                    for (; c < c1; ++c) add(c, std::false_type{}, false);
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) {
                        mbar_arrive(smem_u32(&bars->s_empty[u]));
                        mbar_arrive(smem_u32(&bars->lse_empty[lb]));
                    }
                }
                u += 2;
                if (u >= kSBufs) u -= kSBufs, phase ^= 1;
                const float2 t = f2_split(add2(add2(acc[0], acc[1]), add2(acc[2], acc[3])));
                sum += t.x + t.y;
            }
            if (!ok) break;
            if (it.n0 == 0 && it.n1 == it.all) write_weight(p, it.line, kt, r, sum);
            else p.part[(((int64_t)blockIdx.x * 2 + (it.n0 == 0)) * 2 + group) * KT + r] = sum;
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

// An item that lies in several shares: block c - 1 adds its sums, if the boundary
// between the shares of CTAs c - 1 and c is the first one inside it.
__global__ void __launch_bounds__(2 * KT) key_weight_join_kernel(const WeightParams p) {
    wait_for_previous();
    const int c = blockIdx.x + 1;
    const int64_t x = weight_share(p, c);
    const WeightItem it(p, x, x + 1);
    const int64_t begin = x - it.n0, end = begin + it.all;
    if (it.n0 == 0 || weight_share(p, c - 1) > begin) return;
    const int r = threadIdx.x;
    float sum = p.part[((int64_t)(c - 1) * 2 + 1) * 2 * KT + r];
    for (int d = c; d < p.parts && weight_share(p, d) < end; ++d) sum += p.part[(int64_t)d * 4 * KT + r];
    write_weight(p, it.line, 2 * it.kp + r / KT, r % KT, sum);
}

bool weight_plan(WeightParams *p, const KeyWeightArgs &a) {
    *p = WeightParams{};
    if (!pos_geom(&p->g, a.S, a.N, a.layout)) return false;
    p->H = (int)a.H;
    p->Hkv = (int)a.Hkv;
    p->G = (int)(a.H / a.Hkv);
    p->first = (int)a.first;
    p->f0 = (int)(a.first / p->g.P);
    p->scale = a.scale;
    p->accumulate = a.accumulate;
    const int64_t lines = a.B * a.Hkv;
    const int n = device_sm_count(), sms = n > 0 ? n : 152;  // no device: sizes are still told
    // a head's triples and a CTA's share are counted in 32 bits
    const double all = (double)lines * p->G * p->g.nt * (p->g.nt - p->f0);
    if (all > (double)(1ll << 30) * sms || (double)p->G * p->g.nt > (double)(1ll << 30)) return false;
    p->total = lines * weight_before(p->g, p->f0, p->G, weight_items(p->g));
    p->parts = (int)(p->total < sms ? p->total : sms);
    return true;
}

template <int HD>
int launch_hd(const void *q, const void *k, const float *lse, float *weight, void *workspace, const KeyWeightArgs &a,
              cudaStream_t stream) {
    static PerDeviceOnce once;
    const int attr = once.get([] {
        return cuda_status(cudaFuncSetAttribute(tc_key_weight_kernel<HD>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                (int)WeightCfg<HD>::kSmemBytes));
    });
    if (attr != STRIPED_OK) return attr;
    WeightParams p;
    if (!weight_plan(&p, a)) return STRIPED_ERR_UNSUPPORTED;
    p.lse = lse;
    p.weight = weight;
    p.part = static_cast<float *>(workspace);
    p.wc = device_wait_ctl();
    CUtensorMap mq, mk;
    int st;
    if ((st = make_pos_map(&mq, q, a.D, p.g, a.B * a.H)) || (st = make_pos_map(&mk, k, a.D, p.g, a.B * a.Hkv))) return st;
    tc_key_weight_kernel<HD><<<p.parts, kWtThreads, WeightCfg<HD>::kSmemBytes, stream>>>(mq, mk, p);
    if ((st = cuda_status(cudaGetLastError()))) return st;
    if (p.parts < 2) return STRIPED_OK;
    return launch_after(key_weight_join_kernel, dim3((unsigned)(p.parts - 1)), 2 * KT, 0, stream, p);
}

}  // namespace

size_t key_weight_workspace(const KeyWeightArgs &a) {
    WeightParams p;
    return weight_plan(&p, a) ? (size_t)p.parts * 4 * KT * 4 : 0;
}

int launch_tc_key_weight(const void *q, const void *k, const float *lse, float *weight, void *workspace,
                         const KeyWeightArgs &a, cudaStream_t stream) {
    return a.D == 128 ? launch_hd<128>(q, k, lse, weight, workspace, a, stream)
                      : launch_hd<64>(q, k, lse, weight, workspace, a, stream);
}

}  // namespace striped
