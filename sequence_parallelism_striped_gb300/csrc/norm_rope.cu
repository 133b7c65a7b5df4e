// norm_rope.cu -- RMS norm of every query and key head and the rotary
// position rotation in one pass over the data, and their gradient.
//
// For a row x of D elements at position p (one head of one token):
//   r = 1 / sqrt(mean(x^2) + eps),  n = x r,  y = n w,
//   (y_a, y_b) -> (y_a cos t - y_b sin t, y_b cos t + y_a sin t),
//   t = p * inv_freq[j] for the pair j = (a, b): (j, j + rot/2), or
//   (2j, 2j + 1) when interleaved; elements from rot on are not rotated.
// Gradient: with g the cotangent turned back by the same angle, h = g w,
//   dw = sum over rows of g n,   dx = r (h - n mean(h n)),
// with mean(h n) formed as r mean(h x): r and n stay in the range of fp32
// wherever the squares do, r^3 only for rows between 1e-13 and 4e12.
//
// The position of a row is the one the placement puts there (striped:
// i*N + d; research.elamur.ai summary page, §Summary "every N-th token"), or
// given.  Angles: inv_freq is turned once per block into a 64-bit fraction
// of a turn, F = 2^64 * frac(inv_freq / 2 pi); p * F modulo 2^64 is then the
// phase of position p, reduced to one turn without loss by the integer
// multiplication.  What is left is the rounding of F, in fp64: the angle is
// off by about 2^-53 of itself, as p * inv_freq in fp64 is (1e-6 at p = 2^33).
// The top 32 bits of the phase go to sincospi (fp32, an error of one ulp) or
// to the fast sine (bf16, rope_angles).
//
// Bound by HBM (read and write each element once: 2 or 3 element sizes an
// element).  A group of TP threads owns a row; each thread holds two 16-byte
// vectors of it that contain both members of every pair, so the only
// exchange is the sum for the mean.  The angles of a row are computed once
// and serve every head of the block's chunk.  Rows are brought in by bulk
// copies well ahead of the arithmetic (see the streamed form below).
// Measured at B = 1, H = 32 + 8, S = 65536, D = 128, bf16: 203 us forward
// (6.61 TB/s), 299 us backward (6.73 TB/s); a copy reaches 6.69 TB/s.  fp32 at
// D = 64, the same bytes: 200 and 305 us.
#include <math.h>

#include "common.cuh"
#include "internal.h"

namespace striped {

namespace {

constexpr int kRopeThreads = 128;

struct RopeTensor {
    const void *x;       // [B][heads][S][D]
    const void *g;       // backward: cotangent of the output, same shape
    void *y;             // forward: output; backward: dx
    const float *w;      // [D]
    int heads;
    int chunks;          // head chunks of hc heads each
};

struct RopeParams {
    RopeTensor t[2];     // queries, keys
    const double *inv_freq;
    const int64_t *positions;  // [B][S] or NULL: by placement
    int64_t rows, S, L;  // rows = B * S; L = rows of one stripe
    int D, rot, interleaved;
    int N, layout, stripe;  // stripe >= 0: the rows are that stripe's
    int hc;
    float eps;
    float *parts;        // backward: [gridDim.x * (chunks of both)][D] shares of dw
    WaitCtl wc;
};

__device__ __forceinline__ int64_t position_of(const RopeParams &p, int64_t row, int64_t s) {
    if (p.positions) return p.positions[row];
    int64_t d = p.stripe, i = s;
    if (d < 0) {
        d = s / p.L;
        i = s - d * p.L;
    }
    if (p.layout == STRIPED_LAYOUT_STRIPED) return i * p.N + d;
    if (p.layout == STRIPED_LAYOUT_CONTIGUOUS) return d * p.L + i;
    const int64_t c = p.L / 2;
    return i < c ? d * c + i : (2 * (int64_t)p.N - 1 - d) * c + (i - c);
}

// 16-byte vectors of bf16 (8 values) or fp32 (4 values)
template <typename T>
struct Vec;
template <>
struct Vec<__nv_bfloat16> {
    static constexpr int n = 8;
    static __device__ __forceinline__ void unpack(const uint4 &v, float *f) {
        const __nv_bfloat162 *b = reinterpret_cast<const __nv_bfloat162 *>(&v);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 x = __bfloat1622float2(b[i]);
            f[2 * i] = x.x, f[2 * i + 1] = x.y;
        }
    }
    static __device__ __forceinline__ uint4 pack(const float *f) {
        return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                          pack_bf16x2(f[6], f[7]));
    }
};
template <>
struct Vec<float> {
    static constexpr int n = 4;
    static __device__ __forceinline__ void unpack(const uint4 &v, float *f) {
        f[0] = __uint_as_float(v.x), f[1] = __uint_as_float(v.y), f[2] = __uint_as_float(v.z),
        f[3] = __uint_as_float(v.w);
    }
    static __device__ __forceinline__ uint4 pack(const float *f) {
        return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
    }
};

// Rotate the VN pairs that a thread holds: v[0..VN) and v[VN..2VN) are its
// two vectors; sign +1 turns forward, -1 back.
template <int VN>
__device__ __forceinline__ void turn(float *v, const float *c, const float *s, float sign, int interleaved) {
#pragma unroll
    for (int j = 0; j < VN; ++j) {
        // pair j: (v[j], v[VN + j]), or interleaved (v[2j], v[2j + 1])
        float &a = interleaved ? v[2 * j] : v[j];
        float &b = interleaved ? v[2 * j + 1] : v[VN + j];
        const float sj = sign * s[j], a0 = a;
        a = a * c[j] - b * sj;
        b = b * c[j] + a0 * sj;
    }
}

// What a thread keeps of its place in a row: where its two vectors lie, its
// part of the weight, and (backward) its share of dw.
template <int VN, bool kBwd>
struct RopeLane {
    int off0, off1;
    bool live;  // a row of D elements may need fewer threads than TP
    float w[2 * VN];
    float dw[kBwd ? 2 * VN : 1];
};

template <int VN, bool kBwd, bool kInterleaved>
__device__ __forceinline__ void rope_lane(RopeLane<VN, kBwd> &t, const RopeParams &p, const float *weight, int c) {
    const int nrot = p.rot / (2 * VN);
    t.live = c < p.D / (2 * VN);
    if (c < nrot) {
        t.off0 = kInterleaved ? 2 * VN * c : VN * c;
        t.off1 = kInterleaved ? t.off0 + VN : p.rot / 2 + VN * c;
    } else {
        t.off0 = p.rot + 2 * VN * (c - nrot);
        t.off1 = t.off0 + VN;
    }
#pragma unroll
    for (int j = 0; j < VN; ++j) {
        t.w[j] = t.live ? weight[t.off0 + j] : 0.f;
        t.w[VN + j] = t.live ? weight[t.off1 + j] : 0.f;
    }
    if (kBwd)
#pragma unroll
        for (int j = 0; j < 2 * VN; ++j) t.dw[j] = 0.f;
}

// The pairs' frequencies as fractions of a turn, needed once per row.
__device__ __forceinline__ void rope_freq(uint64_t *freq, const RopeParams &p, int n, int threads) {
    for (int i = threadIdx.x; i < n; i += threads) {
        const double turns = i < p.rot / 2 ? p.inv_freq[i] * 0.15915494309189533577 : 0.0;
        freq[i] = (uint64_t)((turns - floor(turns)) * 18446744073709551616.0);
    }
}

template <typename T, int VN>
__device__ __forceinline__ void rope_angles(const uint64_t *freq, uint64_t pos, float *cs, float *sn) {
#pragma unroll
    for (int j = 0; j < VN; ++j) {
        const int32_t top = (int32_t)((pos * freq[j]) >> 32);
        const float half_turns = (float)top * 4.656612873077393e-10f;  // top / 2^31
        // bf16 results are rounded by up to 2^-8 of their size: the fast
        // instructions' 2^-21 of the pair's size on [-pi, pi] is far below
        if (sizeof(T) == 2) __sincosf(half_turns * 3.14159265f, &sn[j], &cs[j]);
        else sincospif(half_turns, &sn[j], &cs[j]);
    }
}

// One head of a row: rx (and rg, the cotangent) in, result in rx.  `on`: this
// thread has a part of a real row; all lanes of the warp take part.
template <typename T, int TP, bool kBwd, bool kInterleaved>
__device__ __forceinline__ void rope_row(RopeLane<Vec<T>::n, kBwd> &t, uint4 *rx, const uint4 *rg, const float *cs,
                                         const float *sn, float inv_d, float eps, bool on) {
    constexpr int VN = Vec<T>::n;
    float x[2 * VN], g[2 * VN];
    Vec<T>::unpack(rx[0], x);
    Vec<T>::unpack(rx[1], x + VN);
    float sum = 0.f, dot = 0.f;
#pragma unroll
    for (int j = 0; j < 2 * VN; ++j) sum = fmaf(x[j], x[j], sum);
    if (kBwd) {
        Vec<T>::unpack(rg[0], g);
        Vec<T>::unpack(rg[1], g + VN);
        turn<VN>(g, cs, sn, -1.f, kInterleaved);
#pragma unroll
        for (int j = 0; j < 2 * VN; ++j) dot = fmaf(g[j] * t.w[j], x[j], dot);
        if (!on) dot = 0.f;  // angles of rows that do not exist were never set
    }
#pragma unroll
    for (int o = TP / 2; o; o >>= 1) {
        sum += __shfl_xor_sync(0xffffffffu, sum, o);
        if (kBwd) dot += __shfl_xor_sync(0xffffffffu, dot, o);
    }
    if (!on) return;
    const float r = rsqrtf(sum * inv_d + eps);
    float y[2 * VN];
    if (kBwd) {
        const float m = dot * r * inv_d;  // mean(h n)
#pragma unroll
        for (int j = 0; j < 2 * VN; ++j) {
            const float n = x[j] * r;
            t.dw[j] = fmaf(g[j], n, t.dw[j]);
            y[j] = r * (g[j] * t.w[j] - n * m);
        }
    } else {
#pragma unroll
        for (int j = 0; j < 2 * VN; ++j) y[j] = x[j] * r * t.w[j];
        turn<VN>(y, cs, sn, 1.f, kInterleaved);
    }
    rx[0] = Vec<T>::pack(y);
    rx[1] = Vec<T>::pack(y + VN);
}

// The block's share of dw: its rows are summed in a fixed order (within a
// warp by exchange, over the warps in turn), so the result does not change
// from run to run.
template <int VN, int TP>
__device__ __forceinline__ void rope_dw(RopeLane<VN, true> &t, const RopeParams &p) {
    __shared__ float sum[kRopeThreads / 32][2 * VN * TP];
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, c = threadIdx.x % TP;
#pragma unroll
    for (int j = 0; j < 2 * VN; ++j) {
#pragma unroll
        for (int o = 16; o >= TP; o >>= 1) t.dw[j] += __shfl_xor_sync(0xffffffffu, t.dw[j], o);
        if (lane < TP) sum[warp][c * 2 * VN + j] = t.dw[j];
    }
    asm volatile("bar.sync 1, %0;" ::"n"(kRopeThreads) : "memory");
    if (threadIdx.x < TP && t.live) {
        float *out = p.parts + ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * p.D;
#pragma unroll
        for (int j = 0; j < 2 * VN; ++j) {
            float v = 0.f;
#pragma unroll
            for (int k = 0; k < kRopeThreads / 32; ++k) v += sum[k][c * 2 * VN + j];
            out[(j < VN ? t.off0 : t.off1 - VN) + j] = v;
        }
    }
}

// Rows one by one, wherever they lie: for sequences too short for the
// streamed form below.  kInterleaved is a template parameter so that every
// register array is indexed by constants.
template <typename T, int TP, bool kBwd, bool kInterleaved>
__global__ void __launch_bounds__(kRopeThreads, kBwd ? 4 : 7) norm_rope_kernel(const RopeParams p) {
    constexpr int VN = Vec<T>::n;
    constexpr int kRows = kRopeThreads / TP;  // rows a block works on at a time
    const int c = threadIdx.x % TP, slot = threadIdx.x / TP;
    const int which = (int)blockIdx.y >= p.t[0].chunks;
    const RopeTensor &t = p.t[which];
    const int chunk = (int)blockIdx.y - (which ? p.t[0].chunks : 0);
    const int h0 = chunk * p.hc, h1 = min(t.heads, h0 + p.hc);
    __shared__ uint64_t freq[VN * TP];
    rope_freq(freq, p, VN * TP, kRopeThreads);
    RopeLane<VN, kBwd> ln;
    rope_lane<VN, kBwd, kInterleaved>(ln, p, t.w, c);
    __syncthreads();
    const float inv_d = 1.f / (float)p.D;
    for (int64_t row0 = (int64_t)blockIdx.x * kRows; row0 < p.rows; row0 += (int64_t)gridDim.x * kRows) {
        const int64_t row = row0 + slot;
        const bool on = ln.live && row < p.rows;
        int64_t base = 0;
        float cs[VN], sn[VN];
        if (row < p.rows) {
            const int64_t b = row / p.S, s = row - b * p.S;
            base = (b * t.heads * p.S + s) * p.D;
            rope_angles<T, VN>(freq + VN * c, (uint64_t)position_of(p, row, s), cs, sn);
        }
        for (int h = h0; h < h1; ++h) {
            const int64_t at = base + (int64_t)h * p.S * p.D;
            uint4 rx[2] = {make_uint4(0u, 0u, 0u, 0u), make_uint4(0u, 0u, 0u, 0u)}, rg[2] = {rx[0], rx[0]};
            if (on) {
                const T *x = static_cast<const T *>(t.x) + at;
                rx[0] = *reinterpret_cast<const uint4 *>(x + ln.off0);
                rx[1] = *reinterpret_cast<const uint4 *>(x + ln.off1);
                if (kBwd) {
                    const T *g = static_cast<const T *>(t.g) + at;
                    rg[0] = *reinterpret_cast<const uint4 *>(g + ln.off0);
                    rg[1] = *reinterpret_cast<const uint4 *>(g + ln.off1);
                }
            }
            rope_row<T, TP, kBwd, kInterleaved>(ln, rx, rg, cs, sn, inv_d, p.eps, on);
            if (on) {
                T *out = static_cast<T *>(t.y) + at;
                *reinterpret_cast<uint4 *>(out + ln.off0) = rx[0];
                *reinterpret_cast<uint4 *>(out + ln.off1) = rx[1];
            }
        }
    }
    if constexpr (kBwd) {
        let_next_begin();
        rope_dw<VN, TP>(ln, p);
    }
}

// The streamed form: a unit is kRows consecutive rows of one batch entry, one
// contiguous piece of memory per head.  A producer thread copies these pieces
// (x, backward also g) with bulk copies into a ring of shared memory, far
// ahead of the threads that work on them, so that the bytes in flight do not
// depend on how many registers a row takes.
template <typename T, int TP, bool kBwd>
struct RopeRing {
    static constexpr int kRows = kRopeThreads / TP;
    static constexpr int kPiece = kRows * TP * 32;           // bytes of a full piece (32 a thread)
    static constexpr int kStage = kPiece * (kBwd ? 2 : 1);
    static constexpr int NS = 4;
    static constexpr size_t kSmem = (size_t)NS * kStage;
};

template <typename T, int TP, bool kBwd, bool kInterleaved>
__global__ void __launch_bounds__(kRopeThreads + 32, kBwd ? 3 : 4) norm_rope_stream_kernel(const RopeParams p) {
    using Ring = RopeRing<T, TP, kBwd>;
    constexpr int VN = Vec<T>::n, kRows = Ring::kRows, NS = Ring::NS;
    extern __shared__ __align__(128) uint8_t ring[];
    __shared__ uint64_t freq[VN * TP];
    __shared__ uint64_t full[NS], empty[NS];
    const int which = (int)blockIdx.y >= p.t[0].chunks;
    const RopeTensor &t = p.t[which];
    const int chunk = (int)blockIdx.y - (which ? p.t[0].chunks : 0);
    const int h0 = chunk * p.hc, h1 = min(t.heads, h0 + p.hc);
    const int64_t per = (p.S + kRows - 1) / kRows, units = per * (p.rows / p.S);
    const int64_t head = p.S * p.D;  // elements of a head
    if (threadIdx.x == 0) {
        for (int s = 0; s < NS; ++s) {
            mbar_init(smem_u32(&full[s]), 1);
            mbar_init(smem_u32(&empty[s]), kRopeThreads / 32);
        }
        fence_barrier_init();
    }
    rope_freq(freq, p, VN * TP, kRopeThreads + 32);
    __syncthreads();
    if (threadIdx.x >= kRopeThreads) {
        // ---------------- producer
        if (threadIdx.x != kRopeThreads) return;
        int j = 0;
        bool ok = true;
        for (int64_t u = blockIdx.x; u < units && ok; u += gridDim.x) {
            const int64_t b = u / per, s0 = (u - b * per) * kRows;
            const uint32_t bytes = (uint32_t)(min((int64_t)kRows, p.S - s0) * p.D * sizeof(T));
            const int64_t base = (b * t.heads * p.S + s0) * p.D;
            for (int h = h0; h < h1; ++h, ++j) {
                const int s = j % NS;
                if (j >= NS && !mbar_wait(smem_u32(&empty[s]), ((j / NS) + 1) & 1, p.wc)) {
                    ok = false;
                    break;
                }
                const uint32_t fb = smem_u32(&full[s]), dst = smem_u32(ring) + s * Ring::kStage;
                mbar_arrive_expect_tx(fb, bytes * (kBwd ? 2 : 1));
                bulk_load(dst, static_cast<const T *>(t.x) + base + h * head, bytes, fb);
                if (kBwd) bulk_load(dst + Ring::kPiece, static_cast<const T *>(t.g) + base + h * head, bytes, fb);
            }
        }
        // the last piece of every stage has landed before the block may end
        for (int i = j > NS ? j - NS : 0; i < j; ++i) mbar_wait(smem_u32(&full[i % NS]), (i / NS) & 1, p.wc);
        return;
    }
    // ---------------- a group of TP threads per row
    const int c = threadIdx.x % TP, slot = threadIdx.x / TP, lane = threadIdx.x % 32;
    RopeLane<VN, kBwd> ln;
    rope_lane<VN, kBwd, kInterleaved>(ln, p, t.w, c);
    const float inv_d = 1.f / (float)p.D;
    int j = 0;
    bool ok = true;
    for (int64_t u = blockIdx.x; u < units && ok; u += gridDim.x) {
        const int64_t b = u / per, s = (u - b * per) * kRows + slot;
        const bool on = ln.live && s < p.S;
        float cs[VN], sn[VN];
        if (s < p.S) rope_angles<T, VN>(freq + VN * c, (uint64_t)position_of(p, b * p.S + s, s), cs, sn);
        T *out = static_cast<T *>(t.y) + (b * t.heads * p.S + s) * p.D + h0 * head;
        for (int h = h0; h < h1; ++h, ++j, out += head) {
            const int st = j % NS;
            ok = __all_sync(0xffffffffu, mbar_wait(smem_u32(&full[st]), (j / NS) & 1, p.wc));
            if (!ok) break;
            const T *x = reinterpret_cast<const T *>(ring + st * Ring::kStage) + slot * p.D;
            const T *g = reinterpret_cast<const T *>(ring + st * Ring::kStage + Ring::kPiece) + slot * p.D;
            uint4 rx[2] = {make_uint4(0u, 0u, 0u, 0u), make_uint4(0u, 0u, 0u, 0u)}, rg[2] = {rx[0], rx[0]};
            if (on) {
                rx[0] = *reinterpret_cast<const uint4 *>(x + ln.off0);
                rx[1] = *reinterpret_cast<const uint4 *>(x + ln.off1);
                if (kBwd) {
                    rg[0] = *reinterpret_cast<const uint4 *>(g + ln.off0);
                    rg[1] = *reinterpret_cast<const uint4 *>(g + ln.off1);
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&empty[st]));
            rope_row<T, TP, kBwd, kInterleaved>(ln, rx, rg, cs, sn, inv_d, p.eps, on);
            if (on) {
                *reinterpret_cast<uint4 *>(out + ln.off0) = rx[0];
                *reinterpret_cast<uint4 *>(out + ln.off1) = rx[1];
            }
        }
    }
    if constexpr (kBwd) {
        let_next_begin();
        rope_dw<VN, TP>(ln, p);
    }
}

// dw = sum of the blocks' shares, in a fixed order.  One block per 8 columns
// of one weight: 32 threads a column, each adding every 32nd share.
__global__ void __launch_bounds__(256)
    norm_rope_dw_kernel(const float *parts, float *dqw, float *dkw, int nq,
                        int nk, int D) {
    wait_for_previous();
    const int which = blockIdx.y;
    const int col = blockIdx.x * 8 + threadIdx.x % 8, part = threadIdx.x / 8;
    const float *src = parts + (which ? (int64_t)nq * D : 0);
    const int n = which ? nk : nq;
    float v = 0.f;
    if (col < D)
#pragma unroll 8
        for (int i = part; i < n; i += 32) v += src[(int64_t)i * D + col];
    __shared__ float s[32][9];
    s[part][threadIdx.x % 8] = v;
    __syncthreads();
    if (threadIdx.x < 8 && col < D) {
        float t = 0.f;
#pragma unroll
        for (int i = 0; i < 32; ++i) t += s[i][threadIdx.x];
        (which ? dkw : dqw)[col] = t;
    }
}

// Grid: blockIdx.y = a chunk of up to 8 heads of q or of k (a chunk shares one
// computation of the angles; smaller where that leaves multiprocessors
// without work), blockIdx.x strides over the rows.  Never a few blocks more
// than fit at once, which would cost a whole further round (H = 32 + 8, S =
// 65536: 285 us with 1220 blocks, 222 with 605 of 608); long sequences take
// four rounds of shorter blocks, whose ends overlap (201 us; at S = 8192 they
// cost 5 us in set-up).  "At once" is counted for 152 multiprocessors, not
// asked of the device: the backward's shares, and with them the last bits of
// dw, so depend on the sizes only.
//
// Rows are streamed through shared memory by bulk copies when a sequence fills
// at least one block's rows; shorter ones (decoding: one row a request) are
// read by the threads themselves (64 requests of one token, 40 heads: 2.9 us,
// streamed 5.8; S = 65536: 246 us forward and 394 backward, streamed 202 and
// 300).
struct RopeGrid {
    bool stream;
    int hc, cq, ck, gx;
};

RopeGrid rope_grid(int64_t B, int64_t S, int64_t H, int64_t Hkv, int tp, bool bwd) {
    const int64_t per = kRopeThreads / tp;
    RopeGrid g{};
    g.stream = S >= per;
    const int64_t blocks = g.stream ? B * ((S + per - 1) / per) : (B * S + per - 1) / per;
    const int64_t fill = 152 * (bwd ? 3 : 4);  // resident blocks
    g.hc = 8;
    auto chunks = [&](int64_t heads) { return (heads + g.hc - 1) / g.hc; };
    while (g.hc > 1 && blocks * (chunks(H) + chunks(Hkv)) < fill) g.hc /= 2;
    g.cq = (int)chunks(H);
    g.ck = (int)chunks(Hkv);
    int64_t most = fill / (g.cq + g.ck) > 0 ? fill / (g.cq + g.ck) : 1;
    if (blocks >= 32 * most) most *= 4;
    g.gx = (int)(blocks < most ? blocks : most);
    return g;
}

int rope_tp(int64_t D, int dtype) {
    const int64_t need = D / (dtype == STRIPED_BF16 ? 16 : 8);
    int tp = 1;
    while (tp < need) tp *= 2;
    return tp;
}

template <typename T, int TP, bool kBwd, bool kInterleaved>
int launch_rope(const RopeParams &p, const RopeGrid &g, cudaStream_t stream) {
    const dim3 grid((unsigned)g.gx, (unsigned)(g.cq + g.ck));
    if (!g.stream) {
        norm_rope_kernel<T, TP, kBwd, kInterleaved><<<grid, kRopeThreads, 0, stream>>>(p);
        return cuda_status(cudaGetLastError());
    }
    constexpr size_t smem = RopeRing<T, TP, kBwd>::kSmem;
    static PerDeviceOnce once;
    const int attr = once.get([] {
        return cuda_status(cudaFuncSetAttribute(norm_rope_stream_kernel<T, TP, kBwd, kInterleaved>,
                                                cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem));
    });
    if (attr != STRIPED_OK) return attr;
    norm_rope_stream_kernel<T, TP, kBwd, kInterleaved><<<grid, kRopeThreads + 32, smem, stream>>>(p);
    return cuda_status(cudaGetLastError());
}

template <typename T, int TP, bool kBwd>
int launch_tp(const RopeParams &p, const RopeGrid &g, cudaStream_t stream) {
    return p.interleaved ? launch_rope<T, TP, kBwd, true>(p, g, stream) : launch_rope<T, TP, kBwd, false>(p, g, stream);
}

template <typename T, bool kBwd>
int launch_t(const RopeParams &p, const RopeGrid &g, int tp, cudaStream_t stream) {
    switch (tp) {
        case 1: return launch_tp<T, 1, kBwd>(p, g, stream);
        case 2: return launch_tp<T, 2, kBwd>(p, g, stream);
        case 4: return launch_tp<T, 4, kBwd>(p, g, stream);
        case 8: return launch_tp<T, 8, kBwd>(p, g, stream);
        case 16: return launch_tp<T, 16, kBwd>(p, g, stream);
        default: return launch_tp<T, 32, kBwd>(p, g, stream);
    }
}

}  // namespace

size_t rope_bwd_workspace(int64_t B, int64_t H, int64_t Hkv, int64_t S, int64_t D, int dtype) {
    const RopeGrid g = rope_grid(B, S, H, Hkv, rope_tp(D, dtype), true);
    return (size_t)g.gx * (size_t)(g.cq + g.ck) * (size_t)D * 4;
}

int launch_norm_rope(const RopeArgs &a, cudaStream_t stream) {
    RopeParams p{};
    p.t[0].x = a.q, p.t[0].g = a.dq_out, p.t[0].y = a.q_res, p.t[0].w = a.q_weight, p.t[0].heads = (int)a.H;
    p.t[1].x = a.k, p.t[1].g = a.dk_out, p.t[1].y = a.k_res, p.t[1].w = a.k_weight, p.t[1].heads = (int)a.Hkv;
    p.inv_freq = a.inv_freq;
    p.positions = a.positions;
    p.rows = a.B * a.S;
    p.S = a.S;
    p.L = a.positions || a.stripe >= 0 ? a.S : a.S / a.N;
    p.D = (int)a.D;
    p.rot = a.rot;
    p.interleaved = a.interleaved;
    p.N = a.N;
    p.layout = a.layout;
    p.stripe = a.stripe;
    p.eps = a.eps;
    p.parts = static_cast<float *>(a.workspace);
    p.wc = device_wait_ctl();
    const int tp = rope_tp(a.D, a.dtype);
    const RopeGrid g = rope_grid(a.B, a.S, a.H, a.Hkv, tp, a.dq_out != nullptr);
    p.hc = g.hc;
    p.t[0].chunks = g.cq;
    p.t[1].chunks = g.ck;
    int st;
    if (!a.dq_out)
        return a.dtype == STRIPED_BF16 ? launch_t<__nv_bfloat16, false>(p, g, tp, stream)
                                       : launch_t<float, false>(p, g, tp, stream);
    st = a.dtype == STRIPED_BF16 ? launch_t<__nv_bfloat16, true>(p, g, tp, stream)
                                 : launch_t<float, true>(p, g, tp, stream);
    if (st != STRIPED_OK) return st;
    return launch_after(norm_rope_dw_kernel, dim3((unsigned)((a.D + 7) / 8), 2), 256, 0, stream, p.parts, a.dq_weight,
                        a.dk_weight, g.gx * g.cq, g.gx * g.ck, (int)a.D);
}

}  // namespace striped
