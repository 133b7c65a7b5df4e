// attn_decode_kv4.cu -- decoding against a prompt in 4 bits when few query rows
// share a prompt's key/value head (up to 32: its query heads and new tokens).
// More rows go to attn_decode_kv4_tc.cu.
//
// A stored key and value take 9/32 of their bf16 bytes, so for few rows what
// bounds the call is no longer only memory (18 KB for 128 keys at D = 128: 780
// clocks of a multiprocessor's share), but also the instructions that turn
// codes into numbers.  They are made here as the operands of warp-level
// products, in registers: nothing is written to shared memory and read again,
// and there is no row tile of 128 to fill (two tcgen05 products of 128 x 128
// x 128 alone are 1024 clocks).  Both products are transposed, so that keys and
// channels are the 16 rows of an m16n8k16 and the query rows its 8 columns (one to four
// products beside one another, so that codes are turned into numbers once):
//     S^T = K Q^T,  O^T = V^T P^T.
//  * K: the word with 8 channels of a key gives four pairs of channels, which
//    are a lane's part of two products; which channel stands where in the
//    contraction is free, so Q is read in the same order.  Codes go in as whole
//    numbers, and the 32 channels of a group are one sum that the group's scale
//    multiplies in fp32: no value is scaled by itself.
//  * V: words of two keys are interleaved by two byte permutations; then a word's
//    four pairs are pairs of keys, as the product wants them, and are
//    multiplied by the pair of scales (exactly: kv4.cuh).
//  * P^T is S^T's accumulator, transposed 8 x 8 by movmatrix.
// Each warp takes every eighth stretch of 32 keys of the CTA's segment, its
// codes copied to shared memory one stretch ahead (rows 16 bytes further apart
// than they are long: no bank conflicts), and has a running maximum of its own;
// nothing waits for another warp before the segment is done.  Shares, segments
// and their join are those of attn_decode.cu; tails are read straight to
// registers.
//
// The weights P are rounded to bf16 (2^-8 of a weight at most), as everywhere in
// this library: an m16n8k16 of 16-bit operands takes them as they are, and fp32
// ones would be two products of halves each.  The sum of a row adds the
// unrounded ones.
//
// Measured in a graph at D = 128, 32 query heads on 8, one new token: 16 requests
// with prompts of their own of 32768 122 us, 5.1 TB/s (bf16 prompts 309); one
// request on 4096 10.7 us (10.5).  What bounds it is latency: the integer pipe,
// the issue slots and DRAM are each busy about half of the time (47, 50 and 50 %;
// a stretch is read one stretch ahead), so that fewer operations a word helped
// (kv4_pairs: 152 us before).  On the tcgen05 kernel the 16 requests took 452.
#include <math.h>

#include "common.cuh"
#include "decode.cuh"
#include "internal.h"
#include "kv4.cuh"

namespace striped {

namespace {

constexpr int kQThreads = 256;
constexpr int kQWarps = kQThreads / 32;
constexpr int kStep = 32;  // keys of a stretch
constexpr float kQRescale = 8.0f;  // lazy rescale threshold, log2 units

template <int HD, int NT>
struct SmallCfg {
    static constexpr int kGroups = HD / 32;
    static constexpr int kRow = HD / 2 + 16;                     // bytes between rows of codes
    static constexpr int kVOff = kStep * kRow;
    static constexpr int kScaleOff = 2 * kVOff;                  // [key][K groups], [key][V groups]
    static constexpr int kStage = kScaleOff + kStep * kGroups * 4;
    static constexpr int kQRow = HD * 2 + 16;
    static constexpr int kORow = HD + 4;                         // floats between rows of a warp's partial O
    static constexpr int kStages = kQWarps * 2 * kStage, kPartial = kQWarps * 8 * NT * kORow * 4;
    static constexpr int kQOff = kStages > kPartial ? kStages : kPartial;  // partial results lie over the stages
    static constexpr int kStatOff = kQOff + 8 * NT * kQRow;      // [warp][row] maxima, sums
    static constexpr int kCumOff = kStatOff + kQWarps * 8 * NT * 8;
};

__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transposed8x8(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
// `bytes` (0 or N) of N are read, the rest is cleared.
template <int N>
__device__ __forceinline__ void copy_async(uint32_t dst, const void *src, int bytes) {
    if constexpr (N == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(dst), "l"(src), "n"(N), "r"(bytes) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// The state of a warp's query rows: of n-tile n, this thread has rows 8 n + 2 t
// and 8 n + 2 t + 1 (t = lane % 4), as scores of keys lane / 4 (+ 8), as maxima
// and sums, and in O^T as channels of lane / 4.
template <int HD, int NT>
struct SmallRows {
    float o[HD / 16][NT][4];
    float m[NT][2], l[NT][2];
    int hi[NT][2];  // last key that the row keeps

    // Scores s (unscaled) of M * 16 keys -> P^T operands; O and the sums follow
    // the maximum.
    template <int M>
    __device__ __forceinline__ void softmax(float (&s)[M][NT][4], uint32_t (&p)[M][NT][2], float cl2) {
        bool up = false;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                float top = fmaxf(s[0][n][r], s[0][n][r + 2]);
#pragma unroll
                for (int i = 1; i < M; ++i) top = fmax3(top, s[i][n][r], s[i][n][r + 2]);
                up |= top * cl2 > m[n][r] + kQRescale;
            }
        if (__any_sync(0xffffffffu, up)) {
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    float top = fmaxf(s[0][n][r], s[0][n][r + 2]);
#pragma unroll
                    for (int i = 1; i < M; ++i) top = fmax3(top, s[i][n][r], s[i][n][r + 2]);
#pragma unroll
                    for (int x = 4; x < 32; x <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
                    const float now = fmaxf(m[n][r], top * cl2);
                    const float a = now == m[n][r] ? 1.f : ex2(m[n][r] - now);
                    m[n][r] = now;
                    l[n][r] *= a;
#pragma unroll
                    for (int c = 0; c < HD / 16; ++c) o[c][n][r] *= a, o[c][n][r + 2] *= a;
                }
        }
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const float m0 = m[n][0] == -INFINITY ? 0.f : m[n][0], m1 = m[n][1] == -INFINITY ? 0.f : m[n][1];
#pragma unroll
            for (int i = 0; i < M; ++i) {
                const float e0 = ex2(fmaf(s[i][n][0], cl2, -m0)), e1 = ex2(fmaf(s[i][n][1], cl2, -m1));
                const float e2 = ex2(fmaf(s[i][n][2], cl2, -m0)), e3 = ex2(fmaf(s[i][n][3], cl2, -m1));
                l[n][0] += e0 + e2;
                l[n][1] += e1 + e3;
                p[i][n][0] = transposed8x8(pack_bf16x2(e0, e1));
                p[i][n][1] = transposed8x8(pack_bf16x2(e2, e3));
            }
        }
    }
};

template <int HD, int NT>
__global__ void __launch_bounds__(kQThreads, NT == 1 ? 2 : 1)
    decode_kv4_small_kernel(const DecParams p, const __nv_bfloat16 *k_tail, const __nv_bfloat16 *v_tail) {
    using Cfg = SmallCfg<HD, NT>;
    constexpr int V = Cfg::kGroups;
    constexpr int kCopies = HD / 64 * 2;  // 16-byte pieces of a stretch's K (or V) codes, over the lanes
    extern __shared__ __align__(16) uint8_t smem[];
    int *cum = reinterpret_cast<int *>(smem + Cfg::kCumOff);
    float *stat = reinterpret_cast<float *>(smem + Cfg::kStatOff);
    __shared__ int scan[kQWarps];
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, g = lane / 4, t = lane % 4;

    entry_costs<kTailTile, kQThreads>(p, cum, scan);
    let_next_begin();
    const int64_t total = (int64_t)cum[p.entries] * p.Hkv;
    const int parts = (int)min((int64_t)gridDim.x, total), cta = blockIdx.x;
    if (cta >= parts) return;
    const int x0 = share(total, cta, parts), x1 = share(total, cta + 1, parts);

    uint8_t *stages = smem + warp * 2 * Cfg::kStage;
    for (int x = x0; x < x1;) {
        const Segment sg = segment_of(cum, p.entries, p.Hkv, p.over, x, x1);
        x = sg.next;
        if (sg.t1 <= sg.t0) continue;  // the same for all threads
        const bool tail = sg.e >= p.ep;
        const int grp = tail ? sg.e - p.ep : sg.e;
        const int rows = tail ? p.rows_t : p.rows_p, per = p.G * p.T;
        const int end = tail ? len_of(p, grp) : p.P;  // keys of the item
        const bool by_scale = p.scale <= kKv4MostScale;  // what undoes the keys' 2^-6
        const float cl2 = p.scale * 1.4426950408889634f * (!tail && by_scale ? kKv4Unit : 1.f);

        // ---------------- query rows
        __syncthreads();  // shared memory of the segment before is free
        for (int i = threadIdx.x; i < 8 * NT * (HD / 8); i += kQThreads) {
            const int r = i / (HD / 8), c = i % (HD / 8);
            uint4 w = make_uint4(0u, 0u, 0u, 0u);
            if (r < rows) {
                const int j = r / per, in = r - j * per;
                const int b = tail ? grp : grp * p.R + j, h = sg.hkv * p.G + in / p.T;
                w = __ldg(reinterpret_cast<const uint4 *>(p.q + (((int64_t)b * p.H + h) * p.T + in % p.T) * HD) + c);
                if (!tail && !by_scale)
                    w = make_uint4(bf16x2_mul(w.x, kKv4Query), bf16x2_mul(w.y, kKv4Query), bf16x2_mul(w.z, kKv4Query),
                                   bf16x2_mul(w.w, kKv4Query));
            }
            *reinterpret_cast<uint4 *>(smem + Cfg::kQOff + r * Cfg::kQRow + c * 16) = w;
        }
        SmallRows<HD, NT> st;
        int hi_min = 0x7fffffff, qpos_min = 0x7fffffff;
        int qpos[NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const int r = 8 * n + 2 * t + k;
                st.m[n][k] = -INFINITY;
                st.l[n][k] = 0.f;
                st.hi[n][k] = qpos[n][k] = 0x7fffffff;  // no row: keeps everything, is not written
                if (r < rows) {
                    const int j = r / per, in = r - j * per;
                    const int len = tail ? end : len_of(p, grp * p.R + j);
                    qpos[n][k] = p.P + len - p.T + in % p.T;
                    st.hi[n][k] = tail ? min(qpos[n][k] - p.P, end - 1) : end - 1;
                    qpos_min = min(qpos_min, qpos[n][k]);
                }
                hi_min = min(hi_min, st.hi[n][k]);
            }
#pragma unroll
        for (int c = 0; c < HD / 16; ++c)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int k = 0; k < 4; ++k) st.o[c][n][k] = 0.f;
        hi_min = __reduce_min_sync(0xffffffffu, hi_min);
        // a query that stands inside the prompt keeps rows by their position
        const bool inside = !tail && __reduce_min_sync(0xffffffffu, qpos_min) < p.P - 1;
        __syncthreads();
        auto q_at = [&](int n, int i) -> uint4 {  // channels 32 i + 8 t .. + 7 of query row 8 n + g
            return *reinterpret_cast<const uint4 *>(smem + Cfg::kQOff + (8 * n + g) * Cfg::kQRow + i * 64 + t * 16);
        };
        // scores of keys that are not kept, key0 + 16 i + g (+ 8)
        auto masked = [&](auto &s, int key0) {
            constexpr int M = sizeof(s) / sizeof(s[0]);
#pragma unroll
            for (int i = 0; i < M; ++i)
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int key = key0 + 16 * i + g + (k & 2) * 4;
                    const int pos = inside && key < p.P ? row_position(p, key) : -1;
#pragma unroll
                    for (int n = 0; n < NT; ++n)
                        if (key > st.hi[n][k & 1] || pos > qpos[n][k & 1]) s[i][n][k] = -INFINITY;
                }
        };

        if (!tail) {
            // ---------------- 4-bit keys
            const int64_t first = ((int64_t)grp * p.Hkv + sg.hkv) * p.P;
            const int k0 = sg.t0 * DT, k1 = min(sg.t1 * DT, end);
            auto fetch = [&](int key0, int buf) {
                const uint32_t dst = smem_u32(stages + buf * Cfg::kStage);
#pragma unroll
                for (int i = 0; i < kCopies; ++i) {
                    const int c = i * 32 + lane, r = c / (HD / 32), in = c % (HD / 32);
                    const int n = key0 + r < end ? 16 : 0;
                    const int64_t at = (first + min(key0 + r, end - 1)) * (HD / 8) + in * 4;
                    copy_async<16>(dst + r * Cfg::kRow + in * 16, p.k_codes + at, n);
                    copy_async<16>(dst + Cfg::kVOff + r * Cfg::kRow + in * 16, p.v_codes + at, n);
                }
                const int64_t at = (first + min(key0 + lane, end - 1)) * V;
                const int n = key0 + lane < end ? V * 2 : 0;
                copy_async<V * 2>(dst + Cfg::kScaleOff + lane * V * 2, p.k_scales + at, n);
                copy_async<V * 2>(dst + Cfg::kScaleOff + (kStep + lane) * V * 2, p.v_scales + at, n);
            };
            int key0 = k0 + warp * kStep, buf = 0;
            if (key0 < k1) fetch(key0, 0);
            copy_commit();
            for (; key0 < k1; key0 += kQWarps * kStep, buf ^= 1) {
                if (key0 + kQWarps * kStep < k1) fetch(key0 + kQWarps * kStep, buf ^ 1);
                copy_commit();
                copy_wait<1>();
                __syncwarp();
                const uint8_t *at = stages + buf * Cfg::kStage;
                float s[2][NT][4];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    float ks[2][V];
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const uint32_t *sc = reinterpret_cast<const uint32_t *>(
                            at + Cfg::kScaleOff + (16 * i + 8 * h + g) * V * 2);
                        uint32_t w[V / 2];
                        if constexpr (V == 4) {
                            const uint2 x2 = *reinterpret_cast<const uint2 *>(sc);
                            w[0] = x2.x, w[1] = x2.y;
                        } else {
                            w[0] = *sc;
                        }
#pragma unroll
                        for (int v = 0; v < V; ++v)
                            ks[h][v] = __uint_as_float(v & 1 ? w[v / 2] & 0xffff0000u : w[v / 2] << 16);
                    }
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int k = 0; k < 4; ++k) s[i][n][k] = 0.f;
#pragma unroll
                    for (int v = 0; v < V; ++v) {
                        const uint32_t *row = reinterpret_cast<const uint32_t *>(at + (16 * i + g) * Cfg::kRow) + v * 4 + t;
                        const uint32_t a = row[0], b = row[8 * Cfg::kRow / 4];
                        uint32_t ca[4], cb[4];
                        kv4_pairs(a, ca);
                        kv4_pairs(b, cb);
#pragma unroll
                        for (int n = 0; n < NT; ++n) {
                            const uint4 q = q_at(n, v);
                            float d[4] = {0.f, 0.f, 0.f, 0.f};
                            mma16816(d, ca[0], cb[0], ca[1], cb[1], q.x, q.y);
                            mma16816(d, ca[2], cb[2], ca[3], cb[3], q.z, q.w);
                            s[i][n][0] = fmaf(d[0], ks[0][v], s[i][n][0]);
                            s[i][n][1] = fmaf(d[1], ks[0][v], s[i][n][1]);
                            s[i][n][2] = fmaf(d[2], ks[1][v], s[i][n][2]);
                            s[i][n][3] = fmaf(d[3], ks[1][v], s[i][n][3]);
                        }
                    }
                }
                if (inside || key0 + kStep - 1 > hi_min) masked(s, key0);
                uint32_t pt[2][NT][2];
                st.template softmax<2>(s, pt, cl2);
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    // this thread's keys 2 t, 2 t + 1, 2 t + 8, 2 t + 9 of the 16
                    const uint8_t *row = at + Cfg::kVOff + (16 * i + 2 * t) * Cfg::kRow + g * (HD / 16);
                    const uint16_t *sc = reinterpret_cast<const uint16_t *>(
                                             at + Cfg::kScaleOff + (kStep + 16 * i + 2 * t) * V * 2) + g * (HD / 8) / 32;
                    const uint32_t s0 = sc[0] | (uint32_t)sc[V] << 16, s1 = sc[8 * V] | (uint32_t)sc[9 * V] << 16;
                    uint32_t w[4][HD / 64];
#pragma unroll
                    for (int h = 0; h < 4; ++h) {
                        const uint8_t *r = row + ((h & 1) + (h & 2) * 4) * Cfg::kRow;
                        if constexpr (HD == 128) {
                            const uint2 x2 = *reinterpret_cast<const uint2 *>(r);
                            w[h][0] = x2.x, w[h][1] = x2.y;
                        } else {
                            w[h][0] = *reinterpret_cast<const uint32_t *>(r);
                        }
                    }
#pragma unroll
                    for (int u = 0; u < HD / 64; ++u) {
                        const uint32_t e0 = __byte_perm(w[0][u], w[1][u], 0x5410), o0 = __byte_perm(w[0][u], w[1][u], 0x7632);
                        const uint32_t e1 = __byte_perm(w[2][u], w[3][u], 0x5410), o1 = __byte_perm(w[2][u], w[3][u], 0x7632);
                        uint32_t ce0[4], co0[4], ce1[4], co1[4];
                        kv4_pairs(e0, ce0);
                        kv4_pairs(o0, co0);
                        kv4_pairs(e1, ce1);
                        kv4_pairs(o1, co1);
#pragma unroll
                        for (int j = 0; j < 4; ++j)
#pragma unroll
                            for (int n = 0; n < NT; ++n)
                                mma16816(st.o[4 * u + j][n], bf16x2_mul(ce0[j], s0), bf16x2_mul(co0[j], s0),
                                         bf16x2_mul(ce1[j], s1), bf16x2_mul(co1[j], s1), pt[i][n][0], pt[i][n][1]);
                    }
                }
                __syncwarp();  // the stage is free
            }
            copy_wait<0>();
        } else {
            // ---------------- bf16 keys of a tail, 16 at a time
            const int64_t first = ((int64_t)grp * p.Hkv + sg.hkv) * p.C;
            const int k0 = sg.t0 * kTailTile, k1 = min(sg.t1 * kTailTile, end);
            const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
            for (int key0 = k0 + warp * 16; key0 < k1; key0 += kQWarps * 16) {
                float s[1][NT][4];
                const bool on0 = key0 + g < end, on1 = key0 + g + 8 < end;
                const uint4 *ka = reinterpret_cast<const uint4 *>(k_tail + (first + key0 + g) * HD) + t;
                const uint4 *kb = ka + 8 * (HD / 8);
                uint4 a[V], b[V];
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    a[v] = on0 ? __ldg(ka + 4 * v) : zero;
                    b[v] = on1 ? __ldg(kb + 4 * v) : zero;
                }
                // values of this thread's four keys: rows that were never
                // written are 0, where a weight of 0 would not hide them
                const uint4 *va = reinterpret_cast<const uint4 *>(v_tail + (first + key0 + 2 * t) * HD + g * (HD / 8));
                uint4 w[4][HD / 64];
#pragma unroll
                for (int h = 0; h < 4; ++h)
#pragma unroll
                    for (int u = 0; u < HD / 64; ++u) {
                        const int r = (h & 1) + (h & 2) * 4;
                        w[h][u] = key0 + 2 * t + r < end ? __ldg(va + r * (HD / 8) + u) : zero;
                    }
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    float d[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int v = 0; v < V; ++v) {
                        const uint4 q = q_at(n, v);
                        mma16816(d, a[v].x, b[v].x, a[v].y, b[v].y, q.x, q.y);
                        mma16816(d, a[v].z, b[v].z, a[v].w, b[v].w, q.z, q.w);
                    }
#pragma unroll
                    for (int k = 0; k < 4; ++k) s[0][n][k] = d[k];
                }
                if (key0 + 15 > hi_min) masked(s, key0);
                uint32_t pt[1][NT][2];
                st.template softmax<1>(s, pt, cl2);
#pragma unroll
                for (int u = 0; u < HD / 64; ++u) {
                    const uint32_t x[4][4] = {{w[0][u].x, w[0][u].y, w[0][u].z, w[0][u].w},
                                              {w[1][u].x, w[1][u].y, w[1][u].z, w[1][u].w},
                                              {w[2][u].x, w[2][u].y, w[2][u].z, w[2][u].w},
                                              {w[3][u].x, w[3][u].y, w[3][u].z, w[3][u].w}};
#pragma unroll
                    for (int j = 0; j < 4; ++j)
#pragma unroll
                        for (int n = 0; n < NT; ++n)
                            mma16816(st.o[4 * u + j][n], __byte_perm(x[0][j], x[1][j], 0x5410),
                                     __byte_perm(x[0][j], x[1][j], 0x7632), __byte_perm(x[2][j], x[3][j], 0x5410),
                                     __byte_perm(x[2][j], x[3][j], 0x7632), pt[0][n][0], pt[0][n][1]);
                }
            }
        }

        // ---------------- the warps' results -> one partial result
        float *sm = stat, *sl = stat + kQWarps * 8 * NT;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
#pragma unroll
                for (int y = 4; y < 32; y <<= 1) st.l[n][k] += __shfl_xor_sync(0xffffffffu, st.l[n][k], y);
                if (g == 0) {
                    sm[warp * 8 * NT + 8 * n + 2 * t + k] = st.m[n][k];
                    sl[warp * 8 * NT + 8 * n + 2 * t + k] = st.l[n][k];
                }
            }
        __syncthreads();  // every warp is done with the stages, too
        float *po = reinterpret_cast<float *>(smem);  // [warp][row][channel]
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const int r = 8 * n + 2 * t + k;
                float top = -INFINITY;
#pragma unroll
                for (int w = 0; w < kQWarps; ++w) top = fmaxf(top, sm[w * 8 * NT + r]);
                const float a = st.m[n][k] == -INFINITY ? 0.f : ex2(st.m[n][k] - top) * (tail ? 1.f : kKv4Unit);
                float *dst = po + (warp * 8 * NT + r) * Cfg::kORow + g * (HD / 8);
#pragma unroll
                for (int c = 0; c < HD / 16; c += 2)
                    *reinterpret_cast<float4 *>(dst + 2 * c) =
                        make_float4(st.o[c][n][k] * a, st.o[c][n][k + 2] * a, st.o[c + 1][n][k] * a, st.o[c + 1][n][k + 2] * a);
            }
        __syncthreads();
        const int64_t slot = (int64_t)(grp * p.Hkv + sg.hkv + cta) * p.slot_rows[tail];
        for (int i = threadIdx.x; i < rows * (HD / 4); i += kQThreads) {
            const int r = i / (HD / 4), c = i % (HD / 4);
            float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int w = 0; w < kQWarps; ++w) {
                const float4 y = *reinterpret_cast<const float4 *>(po + (w * 8 * NT + r) * Cfg::kORow + 4 * c);
                sum.x += y.x, sum.y += y.y, sum.z += y.z, sum.w += y.w;
            }
            *reinterpret_cast<float4 *>(p.part_o[tail] + (slot + r) * HD + 4 * c) = sum;
            if (c == 0) {
                float top = -INFINITY, l = 0.f;
#pragma unroll
                for (int w = 0; w < kQWarps; ++w) top = fmaxf(top, sm[w * 8 * NT + r]);
#pragma unroll
                for (int w = 0; w < kQWarps; ++w) {
                    const float m = sm[w * 8 * NT + r];
                    // without a maximum the sum is 0, or NaN, which stays
                    l += m == -INFINITY ? sl[w * 8 * NT + r] : sl[w * 8 * NT + r] * ex2(m - top);
                }
                *reinterpret_cast<float2 *>(p.part_ml[tail] + 2 * (slot + r)) = make_float2(top, l);
            }
        }
    }
}

template <int HD, int NT>
int launch_small(DecPlan &plan, const void *kt, const void *vt, const DecodeArgs &a, cudaStream_t stream) {
    static PerDeviceOnce once;
    const size_t most = SmallCfg<HD, NT>::kCumOff + (kMaxEntries + 4) * 4;
    const int attr = once.get([most] {
        return cuda_status(cudaFuncSetAttribute(decode_kv4_small_kernel<HD, NT>,
                                                cudaFuncAttributeMaxDynamicSharedMemorySize, (int)most));
    });
    if (attr != STRIPED_OK) return attr;
    const size_t smem = SmallCfg<HD, NT>::kCumOff + (size_t)(plan.p.entries + 1) * 4;
    decode_kv4_small_kernel<HD, NT><<<plan.parts, kQThreads, smem, stream>>>(
        plan.p, static_cast<const __nv_bfloat16 *>(kt), static_cast<const __nv_bfloat16 *>(vt));
    const int st = cuda_status(cudaGetLastError());
    if (st) return st;
    return launch_after(decode_join_kernel<HD>, dim3((unsigned)(a.B * a.H * a.T)), 128, 0, stream, plan.p, plan.parts);
}

}  // namespace

int launch_decode_kv4(const void *q, const Kv4Prompt &prompt, const void *kt, const void *vt, const int32_t *lens,
                      void *o, float *lse, void *workspace, const DecodeArgs &a, cudaStream_t stream) {
    DecPlan plan;
    if (!decode_plan(&plan, a)) return STRIPED_ERR_UNSUPPORTED;
    if (!plan.small) return launch_tc_decode_kv4(q, prompt, kt, vt, lens, o, lse, workspace, a, stream);
    decode_buffers(&plan, q, prompt, lens, o, lse, workspace);
    const int tiles = (plan.p.rows_p + 7) / 8;
    if (a.D == 128)
        return tiles == 1   ? launch_small<128, 1>(plan, kt, vt, a, stream)
               : tiles == 2 ? launch_small<128, 2>(plan, kt, vt, a, stream)
               : tiles == 3 ? launch_small<128, 3>(plan, kt, vt, a, stream)
                            : launch_small<128, 4>(plan, kt, vt, a, stream);
    return tiles == 1   ? launch_small<64, 1>(plan, kt, vt, a, stream)
           : tiles == 2 ? launch_small<64, 2>(plan, kt, vt, a, stream)
           : tiles == 3 ? launch_small<64, 3>(plan, kt, vt, a, stream)
                        : launch_small<64, 4>(plan, kt, vt, a, stream);
}

}  // namespace striped
