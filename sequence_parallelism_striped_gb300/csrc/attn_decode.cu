// attn_decode.cu -- a few new tokens of every request against a placed prompt
// (one prompt may serve several requests) and the request's own tail, bf16 on
// tcgen05.
//
// Request b's positions 0 .. P-1 are the prompt of entry b / (B/Bp), held in
// the rows of its placement as the prefill left them; positions P, P+1, ...
// are rows 0, 1, ... of its tail.  Query token t of T stands at position
// P + len_b - T + t and keeps the keys that full (or window) attention keeps:
// key <= query and (no window, or query - key < W, or key < sinks).
//
// Bound by HBM: every K and V row is read once (4 D bytes) for the 4 D R
// operations that the R query rows above it need, R = (requests on the
// prompt) * (query heads per key/value head) * T.  So
//  * the rows of all requests that share a prompt and of all query heads of
//    a key/value head are stacked into the 128 rows of one MMA tile, and the
//    prompt is read once for them (more than 128 rows: once per 128, from L2
//    while it is there);
//  * one CTA per multiprocessor, and all (item, key tile) pairs of the call
//    are cut into contiguous shares of equal cost, one per CTA, whatever the
//    lengths (an item is a row tile of one key/value head: of a prompt or of
//    a tail; beginning one costs as much as a few tiles, so that a CTA with
//    many short tails gets fewer tiles).  A CTA's loads run ahead of the
//    arithmetic across item boundaries, so they never pause for a prologue or
//    an epilogue;
//  * each stretch of an item in a CTA (a segment) leaves unnormalised fp32
//    partial results, and a second kernel joins the segments of every row
//    in a fixed order.
//
//   warp 0      TMA producer: K/V tiles of 128 keys (a prompt tile is
//               consecutive positions over all stripes, window.cuh)
//   warp 1      TMEM allocator + tcgen05.mma issuer (one elected lane)
//   warps 2..5  softmax; thread t owns row t (warps without rows only keep
//               the barriers going)
// Tensor memory: S0 [0,128), S1 [128,256), O [256,256+HD), Q [256+HD, +HD/2).
// Tail rows from len on may hold anything (NaN included): their scores are
// masked by selection and their V rows are cleared in shared memory before
// the product, where a weight of 0 would not hide them.
//
// P is rounded to bf16 as a tensor-core operand, the row sum adds the
// unrounded values (attn_window_fwd.cu); partial results are joined in fp32.
//
// Measured in a graph at D = 128, 32 query heads on 8: 32 requests on one
// prompt of 131072 positions, tails of 1000: 110 us, 5.8 TB/s; 16 requests with
// prompts of their own of 32768: 310 us, 6.9 TB/s (a copy reaches 6.69); one
// request on 4096: 11 us, two launches and one tile's chain of load, product,
// softmax, product and join.
#include <math.h>

#include "common.cuh"
#include "internal.h"
#include "window.cuh"

namespace striped {

namespace {

constexpr int DT = 128;                 // rows and keys of a tile
constexpr uint32_t kDBox = 128 * 128;   // 128 rows x 64 bf16
constexpr int kDThreads = 192;
constexpr float kDRescale = 8.0f;       // lazy rescale threshold, log2 units
constexpr int kMaxEntries = 2048;       // row tiles of prompts and tails, over one key/value head

template <int HD>
struct DecCfg {
    static constexpr int NS = HD == 128 ? 3 : 6;  // K/V stages
    static constexpr uint32_t kTile = (HD / 64) * kDBox;
    static constexpr uint32_t kStage = 2 * kTile;
    static constexpr uint32_t kSpanOff = NS * kStage;
    static constexpr uint32_t kBarOff = kSpanOff + (3 * kMaxEntries + 4) * 4;
    static constexpr size_t kSmemBytes = 1024 + kBarOff + 256;
    static_assert(kSmemBytes <= 232448, "shared memory over the per-block limit");
};

template <int NS>
struct DecBars {
    uint64_t q_full;
    uint64_t kv_full[NS], kv_empty[NS];
    uint64_t s_full[2], p_ready, o_done, drain;
    uint32_t tmem_slot;
    int scan[kDThreads / 32];
};

struct DecParams {
    PosGeom g;            // the prompt (S = 0 positions if there is none)
    int P;                // prompt positions
    int B, R, H, Hkv, G, T, C;
    int W, sinks;         // W = 0: no window
    int rows_p, rows_t;   // query rows over a prompt / a tail
    int nrt_p, nrt_t;     // their row tiles
    int ep, entries;      // prompt entries, all entries
    float scale;
    const __nv_bfloat16 *q;
    const int32_t *lens;
    __nv_bfloat16 *o;
    float *lse;
    int over;             // what beginning an item costs, in key tiles
    int32_t *cum;         // [entries + 1] cost of the entries before each one (over one key/value head)
    float *part_o[2], *part_ml[2];  // prompt and tail slots: [slot][rows][D], [slot][rows][m, l]
    int slot_rows[2];
    WaitCtl wc;
};

// The key tiles that an entry's rows need: ns sink tiles, then lo, lo + 1, ..
struct Span {
    int ns, lo, n;
};

__device__ __forceinline__ int len_of(const DecParams &p, int b) {
    return min(max(p.lens[b], 0), p.C);
}

__device__ __forceinline__ Span span_of(int first, int last, int tile, int sinks, int rows) {
    // first .. last: the keys between the lowest window edge and the highest
    // query; sinks of `rows` keys stay visible below it
    first = max(first, 0);
    last = min(last, rows - 1);
    const int nst = (min(max(sinks, 0), rows) + tile - 1) / tile;
    if (last < first) return Span{nst, 0, nst};
    const int lo = first / tile, ns = min(nst, lo);
    return Span{ns, lo, ns + last / tile - lo + 1};
}

__device__ Span entry_span(const DecParams &p, int e) {
    if (e < p.ep) {
        if (p.W == 0) return Span{0, 0, p.g.nt};
        const int bp = e / p.nrt_p, rt = e - bp * p.nrt_p;
        const int per = p.G * p.T;
        const int j0 = rt * DT / per, j1 = min((rt * DT + DT - 1) / per, p.R - 1);
        int shortest = 0x7fffffff, longest = 0;
        for (int j = j0; j <= j1; ++j) {
            const int n = len_of(p, bp * p.R + j);
            shortest = min(shortest, n);
            longest = max(longest, n);
        }
        return span_of(p.P + shortest - p.T - p.W + 1, p.P + longest - 1, p.g.P, p.sinks, p.P);
    }
    const int n = len_of(p, (e - p.ep) / p.nrt_t);
    const int first = p.W == 0 ? 0 : n - p.T - p.W + 1;
    return span_of(first, n - 1, DT, p.sinks - p.P, n);
}

// Share of CTA c of `parts`: tiles [share(c), share(c + 1)).
__device__ __forceinline__ int share(int64_t total, int c, int parts) { return (int)(total * c / parts); }

// One stretch of an item inside a CTA's share [x, x1) of the costs; every item
// costs `over` and then one per key tile.
struct Segment {
    int e, hkv, t0, t1, nt;  // entry, key/value head, tiles t0 .. t1-1 of the entry's nt (none if t1 <= t0)
    int next;                // where the next segment begins
    Span s;
};

__device__ __forceinline__ Segment segment_at(const int *cum, const int *lo, const int *ns, int entries, int hkv_n,
                                              int over, int x, int x1) {
    int a = 0, b = entries - 1;  // last entry that begins at or below x (entries without tiles are passed over)
    while (a < b) {
        const int m = (a + b + 1) >> 1;
        if (cum[m] * hkv_n <= x) a = m;
        else b = m - 1;
    }
    Segment s;
    s.e = a;
    const int cost = cum[a + 1] - cum[a];
    const int in = x - cum[a] * hkv_n;
    s.hkv = in / cost;
    s.nt = cost - over;
    const int off = in - s.hkv * cost;
    s.t0 = max(0, off - over);
    s.t1 = min(s.nt, off + (x1 - x) - over);
    s.next = min(x1, x + cost - off);
    s.s = Span{ns[a], lo[a], s.nt};
    return s;
}

template <int HD>
__global__ void __launch_bounds__(kDThreads, 1)
    tc_decode_kernel(const __grid_constant__ CUtensorMap tmKp, const __grid_constant__ CUtensorMap tmVp,
                     const __grid_constant__ CUtensorMap tmKt, const __grid_constant__ CUtensorMap tmVt,
                     const DecParams p) {
    using Cfg = DecCfg<HD>;
    constexpr int NS = Cfg::NS;
    constexpr uint32_t kTile = Cfg::kTile, kStage = Cfg::kStage;
    constexpr int kBoxes = HD / 64;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem =
        reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    DecBars<NS> *bars = reinterpret_cast<DecBars<NS> *>(smem + Cfg::kBarOff);
    int *cum = reinterpret_cast<int *>(smem + Cfg::kSpanOff);  // [entries + 1]
    int *lo_of = cum + kMaxEntries + 4, *ns_of = lo_of + kMaxEntries;
    const uint32_t sbase = smem_u32(smem);
    const PosGeom &g = p.g;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;

    if (threadIdx.x == 0) {
        mbar_init(smem_u32(&bars->q_full), 4);
        for (int s = 0; s < NS; ++s) {
            mbar_init(smem_u32(&bars->kv_full[s]), 1);
            mbar_init(smem_u32(&bars->kv_empty[s]), 1);
        }
        mbar_init(smem_u32(&bars->s_full[0]), 1);
        mbar_init(smem_u32(&bars->s_full[1]), 1);
        mbar_init(smem_u32(&bars->p_ready), 4);
        mbar_init(smem_u32(&bars->o_done), 1);
        mbar_init(smem_u32(&bars->drain), 1);
        fence_barrier_init();
    }
    if (warp == 1) {
        tmem_alloc(smem_u32(&bars->tmem_slot), 512);
        tmem_relinquish();
    }
    if (p.ep > 0 && g.P < DT) {
        // rows past a prompt tile's positions are never loaded: V has to be
        // finite there, because P = 0 times it is added to O
        for (uint32_t i = threadIdx.x * 16; i < NS * kStage; i += kDThreads * 16)
            *reinterpret_cast<uint4 *>(smem + i) = make_uint4(0u, 0u, 0u, 0u);
        fence_proxy_async_smem();
    }
    // every entry's span, and the running count of key tiles before it
    {
        const int per = (p.entries + kDThreads - 1) / kDThreads;
        const int e0 = min((int)threadIdx.x * per, p.entries), e1 = min(e0 + per, p.entries);
        int sum = 0;
        for (int e = e0; e < e1; ++e) {
            const Span s = entry_span(p, e);
            lo_of[e] = s.lo;
            ns_of[e] = s.ns;
            cum[e + 1] = sum += s.n > 0 ? s.n + p.over : 0;
        }
        int run = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, run, o);
            if (lane >= o) run += v;
        }
        if (lane == 31) bars->scan[warp] = run;
        __syncthreads();
        int before = run - sum;
        for (int w = 0; w < warp; ++w) before += bars->scan[w];
        for (int e = e0; e < e1; ++e) {
            cum[e + 1] += before;
            if (blockIdx.x == 0) p.cum[e + 1] = cum[e + 1];
        }
        if (threadIdx.x == 0) {
            cum[0] = 0;
            if (blockIdx.x == 0) p.cum[0] = 0;
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    // the joining kernel may be set up now (it waits for this grid's results)
    let_next_begin();
    const uint32_t tmem = bars->tmem_slot;
    const uint32_t tS0 = tmem, tS1 = tmem + 128, tO = tmem + 256, tQ = tmem + 256 + HD;
    const int64_t total = (int64_t)cum[p.entries] * p.Hkv;
    // no more shares than costs: the segments of an item are those of
    // consecutive CTAs
    const int parts = (int)min((int64_t)gridDim.x, total), cta = blockIdx.x;
    const int x0 = cta < parts ? share(total, cta, parts) : 0;
    const int x1 = cta < parts ? share(total, cta + 1, parts) : 0;
    auto segment = [&](int x) { return segment_at(cum, lo_of, ns_of, p.entries, p.Hkv, p.over, x, x1); };
    int nx = 0;  // key tiles of this CTA
    for (int x = x0; x < x1;) {
        const Segment sg = segment(x);
        nx += max(0, sg.t1 - sg.t0);
        x = sg.next;
    }

    if (warp == 0 && lane == 0 && nx > 0) {
        // ---------------- TMA producer
        // test hook: the first K/V tile is never loaded, so every wait on it
        // runs out (the kernel must then record the timeout and return)
        const bool skip_first = p.wc.inject == kInjectFwdSkipKV;
        int j = 0;
        bool ok = true;
        for (int x = x0; x < x1 && ok;) {
            const Segment sg = segment(x);
            x = sg.next;
            const bool tail = sg.e >= p.ep;
            const int head = (tail ? (sg.e - p.ep) / p.nrt_t : sg.e / p.nrt_p) * p.Hkv + sg.hkv;
            const CUtensorMap *mk = tail ? &tmKt : &tmKp, *mv = tail ? &tmVt : &tmVp;
            const uint32_t bytes = (uint32_t)(tail ? DT : g.P) * 128 * 2 * kBoxes;
            for (int t = sg.t0; t < sg.t1; ++t, ++j) {
                const int s = j % NS;
                if (j >= NS && !mbar_wait(smem_u32(&bars->kv_empty[s]), ((j / NS) + 1) & 1, p.wc)) {
                    ok = false;
                    break;
                }
                if (skip_first && j == 0) continue;
                const int kt = t < sg.s.ns ? t : sg.s.lo + t - sg.s.ns;
                const TileAt at = tail ? TileAt{kt * DT, 0} : tile_at(g, kt);
                const uint32_t fb = smem_u32(&bars->kv_full[s]);
                const uint32_t kdst = sbase + s * kStage, vdst = kdst + kTile;
                mbar_arrive_expect_tx(fb, bytes);
#pragma unroll
                for (int c = 0; c < kBoxes; ++c) {
                    tma_load_4d(kdst + c * kDBox, mk, fb, 64 * c, at.c1, at.c2, head);
                    tma_load_4d(vdst + c * kDBox, mv, fb, 64 * c, at.c1, at.c2, head);
                }
            }
        }
        // loads [0, j) were issued: wait (bounded) for the last of each stage,
        // so that on an error path none lands after the CTA has exited
        for (int t = j > NS ? j - NS : 0; t < j; ++t)
            if (!(skip_first && t == 0)) mbar_wait(smem_u32(&bars->kv_full[t % NS]), (t / NS) & 1, p.wc);
    } else if (warp == 1 && nx > 0) {
        // ---------------- MMA issuer (the whole warp, one lane issues)
        constexpr uint32_t idesc_qk = idesc_bf16_f32(DT, DT, false, false);
        constexpr uint32_t idesc_pv = idesc_bf16_f32(DT, HD, false, true);
        const bool leader = elect_one();
        const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
        const uint32_t uO = tm + 256, uQ = tm + 256 + HD;
        const uint64_t dk = sdesc_sw128(sbase, 16, 1024), dv = sdesc_sw128(sbase + kTile, kDBox, 1024);
        auto issue_s = [&](int t) -> bool {
            const int s = t % NS;
            if (!mbar_wait_warp(smem_u32(&bars->kv_full[s]), (t / NS) & 1, p.wc)) return false;
            tc_fence_after();
            if (leader) {
#pragma unroll
                for (int kk = 0; kk < HD / 16; ++kk)
                    mma_ts(tm + 128 * (t & 1), uQ + kk * 8,
                           dk + s * (kStage >> 4) + (((kk >> 2) * kDBox + (kk & 3) * 32) >> 4), idesc_qk,
                           kk > 0 ? 1u : 0u);
                mma_commit(smem_u32(&bars->s_full[t & 1]));
            }
            return true;
        };
        bool ok = true;
        int j = 0;
        for (int x = x0, seg = 0; x < x1 && ok;) {
            const Segment sg = segment(x);
            x = sg.next;
            if (sg.t1 <= sg.t0) continue;
            const int j1 = j + sg.t1 - sg.t0;
            const int first = j;
            ok = mbar_wait_warp(smem_u32(&bars->q_full), seg++ & 1, p.wc);
            tc_fence_after();
            if (ok) ok = issue_s(j);
            if (ok && j + 1 < j1) ok = issue_s(j + 1);
            for (; j < j1 && ok; ++j) {
                ok = mbar_wait_warp(smem_u32(&bars->p_ready), j & 1, p.wc);
                if (!ok) break;
                tc_fence_after();
                const int s = j % NS;
                if (leader) {
#pragma unroll
                    for (int kk = 0; kk < DT / 16; ++kk)
                        mma_ts(uO, tm + 128 * (j & 1) + kk * 8, dv + s * (kStage >> 4) + kk * (2048 >> 4), idesc_pv,
                               (j > first || kk > 0) ? 1u : 0u);
                    // only stages the producer will refill get a release (no
                    // arrival may land after the CTA has exited)
                    if (j + NS < nx) mma_commit(smem_u32(&bars->kv_empty[s]));
                    mma_commit(smem_u32(&bars->o_done));
                }
                if (j + 2 < j1) ok = issue_s(j + 2);
            }
        }
        // every MMA issued above completes before TMEM is freed (error paths)
        if (leader) mma_commit(smem_u32(&bars->drain));
        mbar_wait_warp(smem_u32(&bars->drain), 0, p.wc);
    } else if (warp >= 2 && nx > 0) {
        // ---------------- softmax + partial results
        const int quarter = warp & 3;
        const int ri = quarter * 32 + lane;  // row of the tile
        const uint32_t lane_off = (uint32_t)(quarter * 32) << 16;
        const float cl2 = p.scale * 1.4426950408889634f;
        const int per = p.G * p.T;
        int j = 0;
        bool ok = true;
        for (int x = x0; x < x1 && ok;) {
            const Segment sg = segment(x);
            x = sg.next;
            if (sg.t1 <= sg.t0) continue;
            const bool tail = sg.e >= p.ep;
            // this thread's query row: request b, head h, token t
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
            const int h = sg.hkv * p.G + in / p.T, t = in % p.T;
            const int len = len_of(p, b);
            const int base_pos = tail ? p.P : 0;                  // position of key 0
            const int qpos = p.P + len - p.T + t - base_pos;      // relative to it, like hi, lo and sk
            const int hi = min(qpos, (tail ? len : p.P) - 1);
            const int lo = p.W == 0 ? 0 : qpos - p.W + 1;
            const int sk = p.sinks - base_pos;
            if (warp_on) {
                // Q row -> TMEM as bf16 pairs: the A operand of S = Q K^T.
                // The previous segment's products that read it are complete
                // (their S was waited for).
                const uint4 *src =
                    reinterpret_cast<const uint4 *>(p.q + (((int64_t)b * p.H + h) * p.T + t) * HD);
#pragma unroll
                for (int c = 0; c < HD / 64; ++c) {
                    uint32_t qa[32];
#pragma unroll
                    for (int v = 0; v < 8; ++v) {
                        const uint4 w = row_on ? __ldg(src + 8 * c + v) : make_uint4(0u, 0u, 0u, 0u);
                        qa[4 * v] = w.x, qa[4 * v + 1] = w.y, qa[4 * v + 2] = w.z, qa[4 * v + 3] = w.w;
                    }
                    tmem_st32(tQ + lane_off + 32 * c, qa);
                }
                tmem_st_wait();
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&bars->q_full));
            float m_ref = -INFINITY, l = 0.f;
            const int tile_w = tail ? DT : g.P;
            const int nseg = sg.t1 - sg.t0;
            for (int n = 0; n < nseg; ++n, ++j) {
                const int tt = sg.t0 + n;
                const int kt = tt < sg.s.ns ? tt : sg.s.lo + tt - sg.s.ns;
                const int kbase = kt * tile_w;
                // a tail tile with rows that were never written: clear V there
                const int written = tail ? len - kbase : DT;
                if (written < DT) {
                    const int s = j % NS;
                    if (!mbar_wait_warp(smem_u32(&bars->kv_full[s]), (j / NS) & 1, p.wc)) {
                        ok = false;
                        break;
                    }
                    if (ri >= written) {
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
                    const uint32_t tS = ((j & 1) ? tS1 : tS0) + lane_off;
                    if (!mbar_wait_warp(smem_u32(&bars->s_full[j & 1]), (j >> 1) & 1, p.wc)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    float sv[DT];
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
                    const bool full = tile_w == DT && kbase + DT - 1 <= hi && (kbase >= lo || kbase + DT <= sk);
                    if (!__all_sync(0xffffffffu, full)) {
                        // columns past the tile's positions are never kept
                        const int h2 = min(hi - kbase, tile_w - 1), l2 = lo - kbase, s2 = sk - kbase;
#pragma unroll
                        for (int w = 0; w < DT / 32; ++w) {
                            const uint32_t k = kept_bits(32 * w, h2, l2, s2);
                            if (!__all_sync(0xffffffffu, k == ~0u))
#pragma unroll
                                for (int c = 0; c < 32; ++c)
                                    if (!(k & (1u << c))) sv[32 * w + c] = -INFINITY;
                        }
                    }
                    const float m_tile = row_max(sv) * cl2;
                    const bool move = n == 0 || m_tile > m_ref + kDRescale;
                    const float m_new = move ? fmaxf(m_ref, m_tile) : m_ref;
                    alpha = (n == 0 || !move) ? 1.f : ex2(m_ref - m_new);
                    const float m_use = (m_new == -INFINITY) ? 0.f : m_new;
                    const uint64_t cl2x2 = f2(cl2, cl2), nm2 = f2(-m_use, -m_use);
                    uint64_t acc4[4] = {0ull, 0ull, 0ull, 0ull};
                    uint32_t pk[DT / 2];
#pragma unroll
                    for (int c = 0; c < DT / 2; ++c) {
                        const float2 x = f2_split(fma2(f2(sv[2 * c], sv[2 * c + 1]), cl2x2, nm2));
                        const float p0 = ex2(x.x), p1 = ex2(x.y);
                        acc4[c & 3] = add2(acc4[c & 3], f2(p0, p1));
                        pk[c] = pack_bf16x2(p0, p1);
                    }
                    const float2 s01 = f2_split(add2(acc4[0], acc4[1])), s23 = f2_split(add2(acc4[2], acc4[3]));
                    {
                        uint32_t (&a)[32] = *reinterpret_cast<uint32_t(*)[32]>(&pk[0]);
                        uint32_t (&c)[32] = *reinterpret_cast<uint32_t(*)[32]>(&pk[32]);
                        tmem_st32(tS, a);
                        tmem_st32(tS + 32, c);
                    }
                    tmem_st_wait();
                    l = l * alpha + ((s01.x + s01.y) + (s23.x + s23.y));
                    m_ref = m_new;
                }
                if (n > 0) {
                    // the previous product must be complete before O is
                    // touched (and before this warp's next arrival)
                    if (!mbar_wait_warp(smem_u32(&bars->o_done), (j - 1) & 1, p.wc)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    if (warp_on && __any_sync(0xffffffffu, alpha != 1.f)) {
#pragma unroll
                        for (int c = 0; c < HD / 32; ++c) {
                            uint32_t rr[32];
                            tmem_ld32(tO + lane_off + c * 32, rr);
                            tmem_ld_wait(rr);
#pragma unroll
                            for (int v = 0; v < 32; ++v) rr[v] = __float_as_uint(__uint_as_float(rr[v]) * alpha);
                            tmem_st32(tO + lane_off + c * 32, rr);
                        }
                        tmem_st_wait();
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&bars->p_ready));
            }
            if (!ok) break;
            if (!mbar_wait_warp(smem_u32(&bars->o_done), (j - 1) & 1, p.wc)) {
                ok = false;
                break;
            }
            tc_fence_after();
            if (warp_on) {
                // segments in order: one more per item begun or CTA begun
                const int item = (tail ? sg.e - p.ep : sg.e) * p.Hkv + sg.hkv;
                const int64_t at = (int64_t)(item + (int)blockIdx.x) * p.slot_rows[tail] + ri;
                if (row_on) *reinterpret_cast<float2 *>(p.part_ml[tail] + 2 * at) = make_float2(m_ref, l);
                float4 *dst = reinterpret_cast<float4 *>(p.part_o[tail] + at * HD);
#pragma unroll
                for (int c = 0; c < HD / 32; ++c) {
                    uint32_t rr[32];
                    tmem_ld32(tO + lane_off + c * 32, rr);
                    tmem_ld_wait(rr);
                    if (row_on)
#pragma unroll
                        for (int v = 0; v < 8; ++v)
                            dst[8 * c + v] = make_float4(__uint_as_float(rr[4 * v]), __uint_as_float(rr[4 * v + 1]),
                                                         __uint_as_float(rr[4 * v + 2]), __uint_as_float(rr[4 * v + 3]));
                }
                tc_fence_before();
            }
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

// o and lse of every row from its segments: those of its prompt's row tile,
// then those of its tail's.  One block per row; warp w takes every fourth
// segment from the w-th on, eight loads in flight, and the four are added in
// order.
template <int HD>
__global__ void __launch_bounds__(128) decode_join_kernel(const DecParams p, int grid) {
    wait_for_previous();
    constexpr int E = HD / 32;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t row = blockIdx.x;  // (b, h, t)
    const int t = (int)(row % p.T);
    const int64_t bh = row / p.T;
    const int b = (int)(bh / p.H), h = (int)(bh % p.H), hkv = h / p.G;
    const int64_t total = (int64_t)p.cum[p.entries] * p.Hkv, parts = min((int64_t)grid, total);
    // first slot and count of the row's segments: prompt, tail
    int64_t at[2];
    int n[2];
#pragma unroll
    for (int tail = 0; tail < 2; ++tail) {
        const int in = (h % p.G) * p.T + t;
        const int r = tail ? in : (b % p.R) * p.G * p.T + in;
        const int e = (tail ? p.ep + b * p.nrt_t : b / p.R * p.nrt_p) + r / DT;
        n[tail] = 0;
        at[tail] = 0;
        if (!tail && p.ep == 0) continue;
        const int cost = p.cum[e + 1] - p.cum[e];
        if (cost == 0) continue;
        const int64_t first = (int64_t)p.cum[e] * p.Hkv + (int64_t)hkv * cost + p.over;  // its tile 0
        const int64_t last = first + cost - p.over - 1;
        const int c0 = (int)(((first + 1) * parts - 1) / total), c1 = (int)(((last + 1) * parts - 1) / total);
        n[tail] = c1 - c0 + 1;
        at[tail] = (int64_t)((tail ? e - p.ep : e) * p.Hkv + hkv + c0) * p.slot_rows[tail] + r % DT;
    }
    float m = -INFINITY, l = 0.f, acc[E];
#pragma unroll
    for (int i = 0; i < E; ++i) acc[i] = 0.f;
    const int all = n[0] + n[1];
    constexpr int U = 8;
    for (int s0 = warp; s0 < all; s0 += 4 * U) {
        float2 ml[U];
        float v[U][E];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int s = s0 + 4 * u, tail = s >= n[0];
            ml[u] = make_float2(-INFINITY, 0.f);
            if (s < all) {
                const int64_t slot = at[tail] + (int64_t)(s - (tail ? n[0] : 0)) * p.slot_rows[tail];
                ml[u] = *reinterpret_cast<const float2 *>(p.part_ml[tail] + 2 * slot);
                const float *src = p.part_o[tail] + slot * HD + lane * E;
                if constexpr (E == 4) {
                    const float4 x = *reinterpret_cast<const float4 *>(src);
                    v[u][0] = x.x, v[u][1] = x.y, v[u][2] = x.z, v[u][3] = x.w;
                } else {
                    const float2 x = *reinterpret_cast<const float2 *>(src);
                    v[u][0] = x.x, v[u][1] = x.y;
                }
            }
        }
        float m_new = m;
#pragma unroll
        for (int u = 0; u < U; ++u) m_new = fmaxf(m_new, ml[u].x);
        if (m_new == -INFINITY) continue;
        const float old = ex2(m - m_new);
        l *= old;
#pragma unroll
        for (int i = 0; i < E; ++i) acc[i] *= old;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (ml[u].x == -INFINITY) continue;  // no key kept, or no segment
            const float w = ex2(ml[u].x - m_new);
            l = fmaf(ml[u].y, w, l);
#pragma unroll
            for (int i = 0; i < E; ++i) acc[i] = fmaf(v[u][i], w, acc[i]);
        }
        m = m_new;
    }
    __shared__ float sm[4], sl[4], sa[4][HD];
    if (lane == 0) sm[warp] = m, sl[warp] = l;
#pragma unroll
    for (int i = 0; i < E; ++i) sa[warp][lane * E + i] = acc[i];
    __syncthreads();
    m = fmaxf(fmaxf(sm[0], sm[1]), fmaxf(sm[2], sm[3]));
    float w[4];
    l = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        w[i] = sm[i] == -INFINITY ? 0.f : ex2(sm[i] - m);
        l = fmaf(sl[i], w[i], l);
    }
    const float inv = l > 0.f ? 1.f / l : 0.f;
    if (threadIdx.x == 0) p.lse[row] = l > 0.f ? (m + log2f(l)) * 0.6931471805599453f : -INFINITY;
    if (threadIdx.x < HD / 2) {
        float o2[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const int d = 2 * threadIdx.x + k;
            o2[k] = ((sa[0][d] * w[0] + sa[1][d] * w[1]) + (sa[2][d] * w[2] + sa[3][d] * w[3])) * inv;
        }
        reinterpret_cast<uint32_t *>(p.o + row * HD)[threadIdx.x] = pack_bf16x2(o2[0], o2[1]);
    }
}

struct DecPlan {
    DecParams p;
    int parts;
    size_t cum_bytes, ml_bytes[2], o_bytes[2];
};

bool decode_plan(DecPlan *plan, const DecodeArgs &a) {
    DecParams &p = plan->p;
    p = DecParams{};
    if (a.P > 0 && !pos_geom(&p.g, a.P, a.N, a.layout)) return false;
    p.P = (int)a.P;
    p.B = (int)a.B;
    p.R = (int)(a.B / a.Bp);
    p.H = (int)a.H;
    p.Hkv = (int)a.Hkv;
    p.G = (int)(a.H / a.Hkv);
    p.T = (int)a.T;
    p.C = (int)a.C;
    // a window that no query can leave is none
    p.W = a.window >= a.P + a.C ? 0 : (int)a.window;
    p.sinks = p.W == 0 ? 0 : (int)(a.sinks < a.P + a.C ? a.sinks : a.P + a.C);
    const int64_t per = (int64_t)p.G * p.T, rows_p = per * p.R;
    const int64_t nrt_p = (rows_p + DT - 1) / DT, nrt_t = (per + DT - 1) / DT;
    const int64_t ep = a.P > 0 ? a.Bp * nrt_p : 0, entries = ep + a.B * nrt_t;
    if (entries > kMaxEntries) return false;
    // a segment of one tile takes about 2.8 us more than a further tile of a
    // long one, which takes 1.35 us at D = 128 and half of that at D = 64:
    // counted as so many tiles.  16 requests on prompts of their own of 32768,
    // D = 128: 386 us at a cost of 1, 308 at 2, 307 at 3, 309 at 4; 24
    // requests, window 4096, D = 64: 40.3 us at 1, 37.5 at 2, 34.8 at 4, 36.2
    // at 6, 37.5 at 8
    p.over = a.D == 128 ? 2 : 4;
    const int64_t tiles =
        (ep * (a.P > 0 ? p.g.nt + p.over : 0) + a.B * nrt_t * ((a.C + DT - 1) / DT + p.over)) * a.Hkv;
    if (tiles > (1ll << 30)) return false;
    p.rows_p = (int)rows_p;
    p.rows_t = (int)per;
    p.nrt_p = (int)nrt_p;
    p.nrt_t = (int)nrt_t;
    p.ep = (int)ep;
    p.entries = (int)entries;
    p.scale = a.scale;
    const int sms = device_sm_count();
    plan->parts = (int)(tiles < sms ? tiles : sms);
    p.slot_rows[0] = (int)(rows_p < DT ? rows_p : DT);
    p.slot_rows[1] = (int)(per < DT ? per : DT);
    plan->cum_bytes = ((size_t)(entries + 1) * 4 + 255) & ~size_t(255);
    for (int t = 0; t < 2; ++t) {
        const size_t slots = (size_t)((t ? a.B * nrt_t : ep) * a.Hkv + plan->parts);
        plan->ml_bytes[t] = (slots * p.slot_rows[t] * 8 + 255) & ~size_t(255);
        plan->o_bytes[t] = (slots * p.slot_rows[t] * a.D * 4 + 255) & ~size_t(255);
    }
    return true;
}

template <int HD>
int launch_decode_hd(const void *q, const void *kp, const void *vp, const void *kt, const void *vt,
                     const int32_t *lens, void *o, float *lse, void *workspace, const DecodeArgs &a,
                     cudaStream_t stream) {
    static PerDeviceOnce once;
    const int attr = once.get([] {
        return cuda_status(cudaFuncSetAttribute(tc_decode_kernel<HD>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                (int)DecCfg<HD>::kSmemBytes));
    });
    if (attr != STRIPED_OK) return attr;
    DecPlan plan;
    if (!decode_plan(&plan, a)) return STRIPED_ERR_UNSUPPORTED;
    DecParams &p = plan.p;
    p.q = static_cast<const __nv_bfloat16 *>(q);
    p.lens = lens;
    p.o = static_cast<__nv_bfloat16 *>(o);
    p.lse = lse;
    char *ws = static_cast<char *>(workspace);
    p.cum = reinterpret_cast<int32_t *>(ws);
    ws += plan.cum_bytes;
    for (int t = 0; t < 2; ++t) {
        p.part_ml[t] = reinterpret_cast<float *>(ws);
        p.part_o[t] = reinterpret_cast<float *>(ws + plan.ml_bytes[t]);
        ws += plan.ml_bytes[t] + plan.o_bytes[t];
    }
    p.wc = device_wait_ctl();
    CUtensorMap mkp, mvp, mkt, mvt;
    int st;
    if ((st = make_bf16_map(&mkt, kt, a.D, a.C, 1, a.B * a.Hkv, a.C * a.D, a.C * a.D, DT)) ||
        (st = make_bf16_map(&mvt, vt, a.D, a.C, 1, a.B * a.Hkv, a.C * a.D, a.C * a.D, DT)))
        return st;
    if (p.ep > 0) {
        if ((st = make_pos_map(&mkp, kp, a.D, p.g, a.Bp * a.Hkv)) ||
            (st = make_pos_map(&mvp, vp, a.D, p.g, a.Bp * a.Hkv)))
            return st;
    } else {
        mkp = mkt;  // never read
        mvp = mvt;
    }
    tc_decode_kernel<HD><<<plan.parts, kDThreads, DecCfg<HD>::kSmemBytes, stream>>>(mkp, mvp, mkt, mvt, p);
    if ((st = cuda_status(cudaGetLastError()))) return st;
    return launch_after(decode_join_kernel<HD>, dim3((unsigned)(a.B * a.H * a.T)), 128, 0, stream, p, plan.parts);
}

}  // namespace

size_t decode_workspace(const DecodeArgs &a) {
    DecPlan plan;
    if (!decode_plan(&plan, a)) return 0;
    return plan.cum_bytes + plan.ml_bytes[0] + plan.ml_bytes[1] + plan.o_bytes[0] + plan.o_bytes[1];
}

int launch_tc_decode(const void *q, const void *kp, const void *vp, const void *kt, const void *vt,
                     const int32_t *lens, void *o, float *lse, void *workspace, const DecodeArgs &a,
                     cudaStream_t stream) {
    return a.D == 128 ? launch_decode_hd<128>(q, kp, vp, kt, vt, lens, o, lse, workspace, a, stream)
                      : launch_decode_hd<64>(q, kp, vp, kt, vt, lens, o, lse, workspace, a, stream);
}

}  // namespace striped
