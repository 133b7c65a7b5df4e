// attn_decode_kv4_tc.cu -- decoding against a prompt in 4 bits when more than 32
// query rows share a prompt's key/value head (many requests on one prompt), on
// tcgen05.
//
// Rows, items, shares, segments and their join are those of attn_decode.cu; what
// differs is that a prompt's tile comes in 4 bits and is made into the bf16
// operand here, and that it is a quarter of the bytes: no longer memory bounds
// the call (18 KB of 128 keys at D = 128 take 780 clocks of a
// multiprocessor's share) but the products (1024 clocks for 128 rows) and what
// feeds them.  So every stage is wide enough to keep up with the products:
//
//   warp 0        TMA producer of the tails' K/V tiles
//   warp 1        TMEM allocator + tcgen05.mma issuer (one elected lane)
//   warps 4..11   two softmax groups: one for the first 64 keys of every tile,
//                 one for the last 64, each with maxima, sums and an O of its
//                 own; they meet at the end of a segment.  One group for all
//                 128 keys is bounded by a warp's latency: 131 instead of
//                 110 us for 32 requests on 131072, tails of 1000
//   warps 12..19  4 bits -> bf16, four for K and four for V: thread t takes the
//                 codes and scales of row t from memory, a tile ahead, and writes
//                 the values (bf16 numbers, times 2^-6: kv4.cuh) where TMA would
//                 put a bf16 row
// P is rounded to bf16 as a tensor-core operand, the sum of a row adds the unrounded
// weights.  32 requests on one prompt of 131072, tails of 1000, take 110 us in a
// graph, as on a bf16 prompt, where memory is the bound (5.8 TB/s); here it is a
// tile's hand-offs: tensor pipe and DRAM are each busy a quarter of the time.
// Tensor memory: O of both groups [0, 2 HD), Q [2 HD, + HD / 2), three S of 64
// columns behind it, taken in turn.
#include <math.h>

#include <type_traits>

#include "common.cuh"
#include "decode.cuh"
#include "internal.h"
#include "kv4.cuh"
#include "window.cuh"

namespace striped {

namespace {

constexpr uint32_t kDBox = 128 * 128;  // 128 rows x 64 bf16
constexpr int kThreads = 640;
constexpr float kRescale = 8.0f;       // lazy rescale threshold, log2 units
constexpr int kHalf = DT / 2;
constexpr int kSBufs = 3;

template <int HD>
struct Kv4Cfg {
    static constexpr int NS = HD == 128 ? 3 : 6;  // K/V stages
    static constexpr uint32_t kTile = (HD / 64) * kDBox;
    static constexpr uint32_t kStage = 2 * kTile;
    static constexpr uint32_t kCombOff = NS * kStage;            // [row] maximum, sum of the second group
    static constexpr uint32_t kCumOff = kCombOff + DT * 8;
    static constexpr uint32_t kBarOff = kCumOff + (kMaxEntries + 4) * 4;
    static constexpr size_t kSmemBytes = 1024 + kBarOff + 512;
    static_assert(kSmemBytes <= 232448, "shared memory over the per-block limit");
};

template <int NS>
struct Kv4Bars {
    uint64_t q_full;
    uint64_t kv_full[NS], kv_empty[NS];
    uint64_t s_full[kSBufs], p_ready[2], o_done[2];
    uint64_t comb_full, comb_empty, drain;
    uint32_t tmem_slot;
    int scan[kThreads / 32];
};

template <int HD>
__global__ void __launch_bounds__(kThreads, 1)
    tc_decode_kv4_kernel(const __grid_constant__ CUtensorMap tmKt, const __grid_constant__ CUtensorMap tmVt,
                         const DecParams p) {
    using Cfg = Kv4Cfg<HD>;
    constexpr int NS = Cfg::NS;
    constexpr uint32_t kTile = Cfg::kTile, kStage = Cfg::kStage;
    constexpr int kBoxes = HD / 64;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem =
        reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    Kv4Bars<NS> *bars = reinterpret_cast<Kv4Bars<NS> *>(smem + Cfg::kBarOff);
    int *cum = reinterpret_cast<int *>(smem + Cfg::kCumOff);  // [entries + 1]
    float2 *comb = reinterpret_cast<float2 *>(smem + Cfg::kCombOff);
    const uint32_t sbase = smem_u32(smem);
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;

    if (threadIdx.x == 0) {
        mbar_init(smem_u32(&bars->q_full), 4);
        for (int s = 0; s < NS; ++s) {
            mbar_init(smem_u32(&bars->kv_full[s]), 9);  // TMA producer, eight dequantising warps
            mbar_init(smem_u32(&bars->kv_empty[s]), 1);
        }
        for (int i = 0; i < kSBufs; ++i) mbar_init(smem_u32(&bars->s_full[i]), 1);
        for (int h = 0; h < 2; ++h) {
            mbar_init(smem_u32(&bars->p_ready[h]), 4);
            mbar_init(smem_u32(&bars->o_done[h]), 1);
        }
        mbar_init(smem_u32(&bars->comb_full), 4);
        mbar_init(smem_u32(&bars->comb_empty), 4);
        mbar_init(smem_u32(&bars->drain), 1);
        fence_barrier_init();
    }
    if (warp == 1) {
        tmem_alloc(smem_u32(&bars->tmem_slot), 512);
        tmem_relinquish();
    }
    entry_costs<DT, kThreads>(p, cum, bars->scan);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    // the joining kernel may be set up now (it waits for this grid's results)
    let_next_begin();
    const uint32_t tmem = bars->tmem_slot;
    constexpr uint32_t kQCol = 2 * HD, kSCol = kQCol + HD / 2;
    const int64_t total = (int64_t)cum[p.entries] * p.Hkv;
    const int parts = (int)min((int64_t)gridDim.x, total), cta = blockIdx.x;
    const int x0 = cta < parts ? share(total, cta, parts) : 0;
    const int x1 = cta < parts ? share(total, cta + 1, parts) : 0;
    auto segment = [&](int x) { return segment_of(cum, p.entries, p.Hkv, p.over, x, x1); };
    int nx = 0;  // key tiles of this CTA
    for (int x = x0; x < x1;) {
        const Segment sg = segment(x);
        nx += max(0, sg.t1 - sg.t0);
        x = sg.next;
    }

    if (warp == 0 && lane == 0 && nx > 0) {
        // ---------------- TMA producer of the tails
        // test hook: the first tail tile is never loaded, so every wait on it
        // runs out (the kernel must then record the timeout and return)
        bool skip = p.wc.inject == kInjectFwdSkipKV;
        int j = 0, loaded[NS];
        bool ok = true;
#pragma unroll
        for (int s = 0; s < NS; ++s) loaded[s] = -1;
        for (int x = x0; x < x1 && ok;) {
            const Segment sg = segment(x);
            x = sg.next;
            const bool tail = sg.e >= p.ep;
            const int head = tail ? (sg.e - p.ep) / p.nrt_t * p.Hkv + sg.hkv : 0;
            for (int t = sg.t0; t < sg.t1; ++t, ++j) {
                const int s = j % NS;
                if (j >= NS && !mbar_wait(smem_u32(&bars->kv_empty[s]), ((j / NS) + 1) & 1, p.wc)) {
                    ok = false;
                    break;
                }
                const uint32_t fb = smem_u32(&bars->kv_full[s]);
                if (!tail) {
                    mbar_arrive(fb);  // the dequantising warps write this tile
                    continue;
                }
                if (skip) {
                    skip = false;
                    continue;
                }
                const uint32_t kdst = sbase + s * kStage, vdst = kdst + kTile;
                mbar_arrive_expect_tx(fb, 2 * kTile);
#pragma unroll
                for (int c = 0; c < kBoxes; ++c) {
                    tma_load_4d(kdst + c * kDBox, &tmKt, fb, 64 * c, t * DT, 0, head);
                    tma_load_4d(vdst + c * kDBox, &tmVt, fb, 64 * c, t * DT, 0, head);
                }
#pragma unroll
                for (int i = 0; i < NS; ++i)
                    if (i == s) loaded[i] = j;
            }
        }
        // the last load of each stage lands (bounded) before the CTA exits
#pragma unroll
        for (int s = 0; s < NS; ++s)
            if (loaded[s] >= 0 && loaded[s] + NS >= j) mbar_wait(smem_u32(&bars->kv_full[s]), (loaded[s] / NS) & 1, p.wc);
    } else if (warp == 1 && nx > 0) {
        // ---------------- MMA issuer (the whole warp, one lane issues)
        constexpr uint32_t idesc_qk = idesc_bf16_f32(DT, kHalf, false, false);
        constexpr uint32_t idesc_pv = idesc_bf16_f32(DT, HD, false, true);
        const bool leader = elect_one();
        const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
        const uint64_t dk = sdesc_sw128(sbase, 16, 1024), dv = sdesc_sw128(sbase + kTile, kDBox, 1024);
        // unit i is half i % 2 of tile i / 2
        auto issue_s = [&](int i) -> bool {
            const int j = i >> 1, h = i & 1, s = j % NS, u = i % kSBufs;
            if (!mbar_wait_warp(smem_u32(&bars->kv_full[s]), (j / NS) & 1, p.wc)) return false;
            tc_fence_after();
            if (leader) {
#pragma unroll
                for (int kk = 0; kk < HD / 16; ++kk)
                    mma_ts(tm + kSCol + kHalf * u, tm + kQCol + kk * 8,
                           dk + s * (kStage >> 4) + (((kk >> 2) * kDBox + (kk & 3) * 32 + h * kHalf * 128) >> 4), idesc_qk,
                           kk > 0 ? 1u : 0u);
                mma_commit(smem_u32(&bars->s_full[u]));
            }
            return true;
        };
        bool ok = true;
        int i = 0;
        for (int x = x0, seg = 0; x < x1 && ok;) {
            const Segment sg = segment(x);
            x = sg.next;
            if (sg.t1 <= sg.t0) continue;
            const int first = i, i1 = i + 2 * (sg.t1 - sg.t0);
            ok = mbar_wait_warp(smem_u32(&bars->q_full), seg++ & 1, p.wc);
            tc_fence_after();
            for (int k = 0; k < kSBufs && ok; ++k)
                if (i + k < i1) ok = issue_s(i + k);
            for (; i < i1 && ok; ++i) {
                const int j = i >> 1, h = i & 1, s = j % NS;
                ok = mbar_wait_warp(smem_u32(&bars->p_ready[h]), j & 1, p.wc);
                if (!ok) break;
                tc_fence_after();
                if (leader) {
#pragma unroll
                    for (int kk = 0; kk < kHalf / 16; ++kk)
                        mma_ts(tm + HD * h, tm + kSCol + kHalf * (i % kSBufs) + kk * 8,
                               dv + s * (kStage >> 4) + ((h * (kHalf / 16) + kk) * 2048 >> 4), idesc_pv,
                               (i - h > first || kk > 0) ? 1u : 0u);
                    // only stages that will be filled again get a release (no
                    // arrival may land after the CTA has exited)
                    if (h && j + NS < nx) mma_commit(smem_u32(&bars->kv_empty[s]));
                    mma_commit(smem_u32(&bars->o_done[h]));
                }
                if (i + kSBufs < i1) ok = issue_s(i + kSBufs);
            }
        }
        // every MMA issued above completes before TMEM is freed (error paths)
        if (leader) mma_commit(smem_u32(&bars->drain));
        mbar_wait_warp(smem_u32(&bars->drain), 0, p.wc);
    } else if (warp >= 12 && nx > 0) {
        // ---------------- 4 bits -> bf16
        const bool is_v = warp >= 16;
        const int r = threadIdx.x & 127;  // row of the tile
        constexpr int V = HD / 32;        // groups of a row: 16 bytes of codes, one scale
        using Scales = typename std::conditional<HD == 128, uint2, uint32_t>::type;
        const uint4 *codes = reinterpret_cast<const uint4 *>(is_v ? p.v_codes : p.k_codes);
        const Scales *scales = reinterpret_cast<const Scales *>(is_v ? p.v_scales : p.k_scales);
        // this thread's row of the tile that is written next
        uint4 code[V];
        Scales scale{};
        // walks over the prompt tiles of this CTA, one ahead of the writing
        int fx = x0, ft = 0;
        Segment fs{};
        fs.t1 = 0;
        auto fetch = [&]() {
            ++ft;
            while (ft >= fs.t1) {
                if (fx >= x1) return;
                fs = segment(fx);
                fx = fs.next;
                ft = fs.e < p.ep ? fs.t0 : fs.t1;  // tails are not ours
            }
            const int row = ft * DT + r;
#pragma unroll
            for (int i = 0; i < V; ++i) code[i] = make_uint4(0u, 0u, 0u, 0u);
            scale = Scales{};
            if (row < p.P) {
                const int64_t at = ((int64_t)(fs.e / p.nrt_p) * p.Hkv + fs.hkv) * p.P + row;
#pragma unroll
                for (int i = 0; i < V; ++i) code[i] = __ldg(codes + at * V + i);
                scale = __ldg(scales + at);
            }
        };
        fetch();
        int j = 0;
        bool ok = true;
        for (int x = x0; x < x1 && ok;) {
            const Segment sg = segment(x);
            x = sg.next;
            const bool tail = sg.e >= p.ep;
            for (int t = sg.t0; t < sg.t1; ++t, ++j) {
                const int s = j % NS;
                if (j >= NS && !mbar_wait_warp(smem_u32(&bars->kv_empty[s]), ((j / NS) + 1) & 1, p.wc)) {
                    ok = false;
                    break;
                }
                if (!tail) {
                    uint8_t *tile = smem + s * kStage + (is_v ? kTile : 0) + r * 128;
                    const uint32_t *sw = reinterpret_cast<const uint32_t *>(&scale);
#pragma unroll
                    for (int i = 0; i < V; ++i) {
                        const uint32_t s2 = __byte_perm(sw[i / 2], 0, i % 2 ? 0x3232 : 0x1010);
                        const uint32_t w[4] = {code[i].x, code[i].y, code[i].z, code[i].w};
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const int chunk = 4 * i + k;  // 8 channels
                            uint32_t c[4];
                            kv4_pairs(w[k], c);
                            *reinterpret_cast<uint4 *>(tile + chunk / 8 * kDBox + (((chunk & 7) ^ (r & 7)) * 16)) =
                                make_uint4(bf16x2_mul(c[0], s2), bf16x2_mul(c[1], s2), bf16x2_mul(c[2], s2),
                                           bf16x2_mul(c[3], s2));
                        }
                    }
                    fetch();
                    fence_proxy_async_smem();
                    __syncwarp();
                }
                if (lane == 0) mbar_arrive(smem_u32(&bars->kv_full[s]));
            }
        }
    } else if (warp >= 4 && nx > 0) {
        // ---------------- softmax + partial results
        const int h = (warp - 4) >> 2, quarter = warp & 3;
        const int ri = quarter * 32 + lane;  // row of the tile
        const uint32_t lane_off = (uint32_t)(quarter * 32) << 16;
        const uint32_t tO = tmem + HD * h + lane_off;
        const int per = p.G * p.T;
        int j = 0, seg = 0;
        int u = h, phase = 0;  // S buffer of the group's next unit 2 j + h, and its phase
        bool ok = true;
        for (int x = x0; x < x1 && ok;) {
            const Segment sg = segment(x);
            x = sg.next;
            if (sg.t1 <= sg.t0) continue;
            const bool tail = sg.e >= p.ep;
            const float unit = tail ? 1.f : kKv4Unit;  // of the values in the tiles
            const bool by_scale = p.scale <= kKv4MostScale;  // what undoes the keys' 2^-6
            const float cl2 = p.scale * 1.4426950408889634f * (by_scale ? unit : 1.f);
            // this thread's query row: request b, head hq, token t
            int grp, rt, rows;
            if (tail) {
                grp = (sg.e - p.ep) / p.nrt_t;
                rt = (sg.e - p.ep) - grp * p.nrt_t;
                rows = p.rows_t;
            } else {
                grp = sg.e / p.nrt_p;
                rt = sg.e - grp * p.nrt_p;
                rows = p.rows_p;
            }
            const int r = rt * DT + ri;
            const bool row_on = r < rows;
            const bool warp_on = rt * DT + quarter * 32 < rows;  // uniform in the warp
            const int jr = row_on ? r / per : 0, in = row_on ? r - jr * per : 0;
            const int b = tail ? grp : grp * p.R + jr;
            const int hq = sg.hkv * p.G + in / p.T, t = in % p.T;
            const int len = len_of(p, b);
            const int qpos = p.P + len - p.T + t - (tail ? p.P : 0);  // relative to key 0, like hi
            const int hi = min(qpos, (tail ? len : p.P) - 1);
            const bool inside = !tail && __any_sync(0xffffffffu, qpos < p.P - 1);  // a query inside the prompt
            if (h == 0) {
                if (warp_on) {
                    // Q row -> TMEM as bf16 pairs: the A operand of S = Q K^T.  The
                    // last segment's products that read it are complete (both
                    // groups have had their S)
                    const uint4 *src =
                        reinterpret_cast<const uint4 *>(p.q + (((int64_t)b * p.H + hq) * p.T + t) * HD);
#pragma unroll
                    for (int c = 0; c < HD / 64; ++c) {
                        uint32_t qa[32];
#pragma unroll
                        for (int v = 0; v < 8; ++v) {
                            const uint4 w = row_on ? __ldg(src + 8 * c + v) : make_uint4(0u, 0u, 0u, 0u);
                            qa[4 * v] = w.x, qa[4 * v + 1] = w.y, qa[4 * v + 2] = w.z, qa[4 * v + 3] = w.w;
                        }
                        if (!tail && !by_scale)
#pragma unroll
                            for (int v = 0; v < 32; ++v) qa[v] = bf16x2_mul(qa[v], kKv4Query);
                        tmem_st32(tmem + kQCol + lane_off + 32 * c, qa);
                    }
                    tmem_st_wait();
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&bars->q_full));
            } else if (seg > 0 && !mbar_wait_warp(smem_u32(&bars->comb_empty), (seg + 1) & 1, p.wc)) {
                break;  // the first group has taken this one's O of the last segment
            }
            float m_ref = -INFINITY, l = 0.f;
            const int nseg = sg.t1 - sg.t0;
            for (int n = 0; n < nseg; ++n, ++j) {
                const int kbase = (sg.t0 + n) * DT + kHalf * h;  // the group's first key
                // a tail tile with rows that were never written: clear V there
                const int written = tail ? len - (sg.t0 + n) * DT : DT;
                if (written < DT) {
                    const int s = j % NS;
                    if (!mbar_wait_warp(smem_u32(&bars->kv_full[s]), (j / NS) & 1, p.wc)) {
                        ok = false;
                        break;
                    }
                    if (ri >= written && ri / kHalf == h) {
                        uint8_t *v = smem + s * kStage + kTile + ri * 128;
#pragma unroll
                        for (int c = 0; c < kBoxes; ++c)
#pragma unroll
                            for (int i = 0; i < 8; ++i)
                                *reinterpret_cast<uint4 *>(v + c * kDBox + 16 * i) = make_uint4(0u, 0u, 0u, 0u);
                    }
                    fence_proxy_async_smem();
                }
                float alpha = 1.f;
                if (warp_on) {
                    const uint32_t tS = tmem + kSCol + kHalf * u + lane_off;
                    if (!mbar_wait_warp(smem_u32(&bars->s_full[u]), phase, p.wc)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const bool full = !inside && __all_sync(0xffffffffu, kbase + kHalf - 1 <= hi);
                    uint32_t keep[2];
                    if (!full) {
#pragma unroll
                        for (int w = 0; w < 2; ++w) {
                            keep[w] = kept_bits(32 * w, hi - kbase, 0, 0);
                            if (inside) {  // rows by their position
                                keep[w] = 0;
#pragma unroll 1
                                for (int c = 0; c < 32; ++c) {
                                    const int row = kbase + 32 * w + c;
                                    if (row < p.P && row_position(p, row) <= qpos) keep[w] |= 1u << c;
                                }
                            }
                        }
                    }
                    auto scores = [&](int w, uint32_t (&y)[32]) {
                        tmem_ld32(tS + 32 * w, y);
                        tmem_ld_wait(y);
                        if (!full)
#pragma unroll
                            for (int c = 0; c < 32; ++c)
                                if (!(keep[w] & (1u << c))) y[c] = 0xff800000u;  // -infinity
                    };
                    // the maximum, then the scores again (96 registers a thread)
                    float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                    for (int w = 0; w < 2; ++w) {
                        uint32_t y[32];
                        scores(w, y);
#pragma unroll
                        for (int c = 0; c < 32; c += 2)
                            top[(c >> 1) & 3] = fmax3(top[(c >> 1) & 3], __uint_as_float(y[c]), __uint_as_float(y[c + 1]));
                    }
                    const float m_tile = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])) * cl2;
                    const bool move = n == 0 || m_tile > m_ref + kRescale;
                    const float m_new = move ? fmaxf(m_ref, m_tile) : m_ref;
                    // a first tile may keep nothing: the maximum is still to come
                    alpha = (n == 0 || !move) ? 1.f : ex2(m_ref - m_new);
                    const float m_use = (m_new == -INFINITY) ? 0.f : m_new;
                    const uint64_t cl2x2 = f2(cl2, cl2), nm2 = f2(-m_use, -m_use);
                    uint64_t acc[2] = {0ull, 0ull};
#pragma unroll
                    for (int w = 0; w < 2; ++w) {
                        uint32_t y[32], pk[16];
                        scores(w, y);
#pragma unroll
                        for (int c = 0; c < 16; ++c) {
                            const float2 e = f2_split(
                                fma2(f2(__uint_as_float(y[2 * c]), __uint_as_float(y[2 * c + 1])), cl2x2, nm2));
                            const float p0 = ex2(e.x), p1 = ex2(e.y);
                            acc[c & 1] = add2(acc[c & 1], f2(p0, p1));
                            pk[c] = pack_bf16x2(p0, p1);
                        }
                        tmem_st16(tS + 16 * w, pk);  // over scores that were read
                    }
                    tmem_st_wait();
                    const float2 sum = f2_split(add2(acc[0], acc[1]));
                    l = l * alpha + (sum.x + sum.y);
                    m_ref = m_new;
                }
                u += 2;
                if (u >= kSBufs) u -= kSBufs, phase ^= 1;
                if (n > 0) {
                    // the previous product must be complete before O is
                    // touched (and before this warp's next arrival)
                    if (!mbar_wait_warp(smem_u32(&bars->o_done[h]), (j - 1) & 1, p.wc)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    if (warp_on && __any_sync(0xffffffffu, alpha != 1.f)) {
#pragma unroll
                        for (int c = 0; c < HD / 32; ++c) {
                            uint32_t rr[32];
                            tmem_ld32(tO + c * 32, rr);
                            tmem_ld_wait(rr);
#pragma unroll
                            for (int v = 0; v < 32; ++v) rr[v] = __float_as_uint(__uint_as_float(rr[v]) * alpha);
                            tmem_st32(tO + c * 32, rr);
                        }
                        tmem_st_wait();
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&bars->p_ready[h]));
            }
            if (!ok) break;
            if (!mbar_wait_warp(smem_u32(&bars->o_done[h]), (j - 1) & 1, p.wc)) {
                ok = false;
                break;
            }
            tc_fence_after();
            if (h == 1) {
                comb[ri] = make_float2(m_ref, l);
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&bars->comb_full));
            } else {
                if (!mbar_wait_warp(smem_u32(&bars->comb_full), seg & 1, p.wc)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                if (warp_on) {
                    const float2 other = comb[ri];
                    const float m = fmaxf(m_ref, other.x);
                    const float w0 = m_ref == -INFINITY ? 0.f : ex2(m_ref - m);
                    const float w1 = other.x == -INFINITY ? 0.f : ex2(other.x - m);
                    // segments in order: one more per item begun or CTA begun
                    const int item = (tail ? sg.e - p.ep : sg.e) * p.Hkv + sg.hkv;
                    const int64_t at = (int64_t)(item + (int)blockIdx.x) * p.slot_rows[tail] + ri;
                    if (row_on)
                        *reinterpret_cast<float2 *>(p.part_ml[tail] + 2 * at) = make_float2(m, l * w0 + other.y * w1);
                    const float f0 = w0 * unit, f1 = w1 * unit;
                    float4 *dst = reinterpret_cast<float4 *>(p.part_o[tail] + at * HD);
#pragma unroll
                    for (int c = 0; c < HD / 16; ++c) {
                        uint32_t a[16], d[16];
                        tmem_ld16(tO + c * 16, a);
                        tmem_ld16(tO + HD + c * 16, d);
                        tmem_ld_wait16(a, d);
                        if (row_on)
#pragma unroll
                            for (int v = 0; v < 4; ++v)
                                dst[4 * c + v] =
                                    make_float4(__uint_as_float(a[4 * v]) * f0 + __uint_as_float(d[4 * v]) * f1,
                                                __uint_as_float(a[4 * v + 1]) * f0 + __uint_as_float(d[4 * v + 1]) * f1,
                                                __uint_as_float(a[4 * v + 2]) * f0 + __uint_as_float(d[4 * v + 2]) * f1,
                                                __uint_as_float(a[4 * v + 3]) * f0 + __uint_as_float(d[4 * v + 3]) * f1);
                    }
                    tc_fence_before();
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&bars->comb_empty));
            }
            ++seg;
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
int launch_hd(DecPlan &plan, const void *kt, const void *vt, const DecodeArgs &a, cudaStream_t stream) {
    static PerDeviceOnce once;
    const int attr = once.get([] {
        return cuda_status(cudaFuncSetAttribute(tc_decode_kv4_kernel<HD>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                (int)Kv4Cfg<HD>::kSmemBytes));
    });
    if (attr != STRIPED_OK) return attr;
    CUtensorMap mkt, mvt;
    int st;
    if ((st = make_bf16_map(&mkt, kt, a.D, a.C, 1, a.B * a.Hkv, a.C * a.D, a.C * a.D, DT)) ||
        (st = make_bf16_map(&mvt, vt, a.D, a.C, 1, a.B * a.Hkv, a.C * a.D, a.C * a.D, DT)))
        return st;
    tc_decode_kv4_kernel<HD><<<plan.parts, kThreads, Kv4Cfg<HD>::kSmemBytes, stream>>>(mkt, mvt, plan.p);
    if ((st = cuda_status(cudaGetLastError()))) return st;
    return launch_after(decode_join_kernel<HD>, dim3((unsigned)(a.B * a.H * a.T)), 128, 0, stream, plan.p, plan.parts);
}

}  // namespace

int launch_tc_decode_kv4(const void *q, const Kv4Prompt &prompt, const void *kt, const void *vt, const int32_t *lens,
                         void *o, float *lse, void *workspace, const DecodeArgs &a, cudaStream_t stream) {
    DecPlan plan;
    if (!decode_plan(&plan, a)) return STRIPED_ERR_UNSUPPORTED;
    decode_buffers(&plan, q, prompt, lens, o, lse, workspace);
    return a.D == 128 ? launch_hd<128>(plan, kt, vt, a, stream) : launch_hd<64>(plan, kt, vt, a, stream);
}

}  // namespace striped
