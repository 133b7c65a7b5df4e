// decode.cuh -- what the decoding kernels share: the (row tile, key tile) pairs
// of a call cut into one contiguous share per CTA, and the join of the
// segments that the shares leave (attn_decode.cu has the picture).
#pragma once

#include <math.h>

#include "common.cuh"
#include "internal.h"
#include "window.cuh"

namespace striped {

namespace {

constexpr int DT = 128;              // rows and keys of a tile
constexpr int kMaxEntries = 2048;    // row tiles of prompts and tails, over one key/value head
constexpr int kTailTile = 32;        // keys of a tail's tile beside a 4-bit prompt and few rows: about
                                     // the bytes of 128 stored keys

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
    // a prompt in 4 bits (kv4.cuh): its tiles are rows as they lie, g counts
    // them as a contiguous sequence, and these place them
    const uint32_t *k_codes, *v_codes;
    const __nv_bfloat16 *k_scales, *v_scales;
    int layout, N, L;
    WaitCtl wc;
};

// The position that row r of a 4-bit prompt holds.
__device__ __forceinline__ int row_position(const DecParams &p, int r) {
    if (p.N == 1) return r;
    const int d = r / p.L, i = r - d * p.L;
    if (p.layout == STRIPED_LAYOUT_STRIPED) return i * p.N + d;
    const int C = p.L / 2;
    return i < C ? d * C + i : (2 * p.N - 1 - d) * C + i - C;
}

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

// Key tiles of an entry without a window, tails in tiles of TT keys.
template <int TT>
__device__ __forceinline__ int entry_tiles(const DecParams &p, int e) {
    if (e < p.ep) return p.g.nt;
    return (len_of(p, (e - p.ep) / p.nrt_t) + TT - 1) / TT;
}

// The running cost of the entries, cum[0 .. entries] in shared memory and, by
// block 0, in p.cum, without windows: by all NT threads of a block, with a
// barrier at the end.
template <int TT, int NT>
__device__ __forceinline__ void entry_costs(const DecParams &p, int *cum, int *scan) {
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    const int per = (p.entries + NT - 1) / NT;
    const int e0 = min((int)threadIdx.x * per, p.entries), e1 = min(e0 + per, p.entries);
    int sum = 0;
    for (int e = e0; e < e1; ++e) {
        const int n = entry_tiles<TT>(p, e);
        cum[e + 1] = sum += n > 0 ? n + p.over : 0;
    }
    int run = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, run, o);
        if (lane >= o) run += v;
    }
    if (lane == 31) scan[warp] = run;
    __syncthreads();
    int before = run - sum;
    for (int w = 0; w < warp; ++w) before += scan[w];
    for (int e = e0; e < e1; ++e) {
        cum[e + 1] += before;
        if (blockIdx.x == 0) p.cum[e + 1] = cum[e + 1];
    }
    if (threadIdx.x == 0) {
        cum[0] = 0;
        if (blockIdx.x == 0) p.cum[0] = 0;
    }
    __syncthreads();
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

__device__ __forceinline__ Segment segment_of(const int *cum, int entries, int hkv_n, int over, int x, int x1) {
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
    s.s = Span{0, 0, s.nt};
    return s;
}
__device__ __forceinline__ Segment segment_at(const int *cum, const int *lo, const int *ns, int entries, int hkv_n,
                                              int over, int x, int x1) {
    Segment s = segment_of(cum, entries, hkv_n, over, x, x1);
    s.s.ns = ns[s.e];
    s.s.lo = lo[s.e];
    return s;
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
        // a segment without a maximum has the sum 0, or NaN if its scores are no
        // numbers: that one is kept
        if (m_new == -INFINITY) {
#pragma unroll
            for (int u = 0; u < U; ++u) l += ml[u].y;
            continue;
        }
        const float old = ex2(m - m_new);
        l *= old;
#pragma unroll
        for (int i = 0; i < E; ++i) acc[i] *= old;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const float w = ex2(ml[u].x - m_new);
            l = fmaf(ml[u].y, w, l);
            if (ml[u].x == -INFINITY) continue;  // no key kept, or no segment
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
    // l is 0 if no key was kept, NaN if scores are no numbers: so is the result then
    const float inv = l > 0.f ? 1.f / l : l;
    if (threadIdx.x == 0) p.lse[row] = l > 0.f ? (m + log2f(l)) * 0.6931471805599453f : l == 0.f ? -INFINITY : l;
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
    bool small;  // a 4-bit prompt under few rows (attn_decode_kv4.cu)
    size_t cum_bytes, ml_bytes[2], o_bytes[2];
};

bool decode_plan(DecPlan *plan, const DecodeArgs &a) {
    DecParams &p = plan->p;
    p = DecParams{};
    if (a.kv4) {
        p.layout = a.layout;
        p.N = a.layout == STRIPED_LAYOUT_CONTIGUOUS ? 1 : a.N;
        p.L = (int)(a.P / p.N);
    }
    if (a.P > 0 && !pos_geom(&p.g, a.P, a.kv4 ? 1 : a.N, a.kv4 ? STRIPED_LAYOUT_CONTIGUOUS : a.layout)) return false;
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
    // With a 4-bit prompt a tile takes less: 4 at both D (1 request: 11.5 us at 2,
    // 10.8 at 4, 11.0 at 6; 32 on one of 131072, tails of 8: 137, 98, 100; tails of
    // 1000: 110, 111, 114)
    p.over = a.D == 128 && !a.kv4 ? 2 : 4;
    // Few rows on a 4-bit prompt go to attn_decode_kv4.cu, more to
    // attn_decode_kv4_tc.cu.  16 prompts of 32768, 8 heads, D = 128 (64), us: 8 rows
    // 123 against 278 (80, 230), 16 rows 162 against 285 (125, 233), 24 rows 215
    // against 302 (155, 235), 32 rows 265 against 312 (179, 237)
    plan->small = a.kv4 && rows_p <= 32;
    const int tail_tile = plan->small ? kTailTile : DT;
    const int64_t tiles =
        (ep * (a.P > 0 ? p.g.nt + p.over : 0) + a.B * nrt_t * ((a.C + tail_tile - 1) / tail_tile + p.over)) * a.Hkv;
    if (tiles > (1ll << 30)) return false;
    p.rows_p = (int)rows_p;
    p.rows_t = (int)per;
    p.nrt_p = (int)nrt_p;
    p.nrt_t = (int)nrt_t;
    p.ep = (int)ep;
    p.entries = (int)entries;
    p.scale = a.scale;
    const int sms = device_sm_count();  // no device: sizes are still told
    const int ctas = (sms > 0 ? sms : 152) * (plan->small && rows_p <= 8 ? 2 : 1);
    plan->parts = (int)(tiles < ctas ? tiles : ctas);
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

// The call's pointers, and the workspace cut up.
void decode_buffers(DecPlan *plan, const void *q, const Kv4Prompt &prompt, const int32_t *lens, void *o, float *lse,
                    void *workspace) {
    DecParams &p = plan->p;
    p.q = static_cast<const __nv_bfloat16 *>(q);
    p.lens = lens;
    p.o = static_cast<__nv_bfloat16 *>(o);
    p.lse = lse;
    p.k_codes = static_cast<const uint32_t *>(prompt.k_codes);
    p.v_codes = static_cast<const uint32_t *>(prompt.v_codes);
    p.k_scales = static_cast<const __nv_bfloat16 *>(prompt.k_scales);
    p.v_scales = static_cast<const __nv_bfloat16 *>(prompt.v_scales);
    char *ws = static_cast<char *>(workspace);
    p.cum = reinterpret_cast<int32_t *>(ws);
    ws += plan->cum_bytes;
    for (int t = 0; t < 2; ++t) {
        p.part_ml[t] = reinterpret_cast<float *>(ws);
        p.part_o[t] = reinterpret_cast<float *>(ws + plan->ml_bytes[t]);
        ws += plan->ml_bytes[t] + plan->o_bytes[t];
    }
    p.wc = device_wait_ctl();
}

}  // namespace

}  // namespace striped
