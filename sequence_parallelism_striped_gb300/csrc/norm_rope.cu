// norm_rope.cu -- RMS norm of every query and key head and the rotary
// position rotation in one pass over the data, and their gradient.
//
// For a row x of D elements at position p (one head of one token):
//   r = 1 / sqrt(mean(x^2) + eps),  n = x r,  y = n w,
//   (y_a, y_b) -> (y_a cos t - y_b sin t, y_b cos t + y_a sin t),
//   t = p * inv_freq[j] for the pair j = (a, b): (j, j + rot/2), or
//   (2j, 2j + 1) when interleaved; elements from rot on are not rotated.
// Gradient: with g the cotangent turned back by the same angle, h = g w,
//   dw = sum over rows of g n,   dx = r h - x r^3 mean(h x).
//
// The position of a row is the one the placement puts there (striped:
// i*N + d; research.elamur.ai summary page, §Summary "every N-th token"), or
// given.  Angles: inv_freq is turned once per thread into a 64-bit fraction
// of a turn, F = 2^64 * frac(inv_freq / 2 pi); p * F modulo 2^64 is then the
// exact phase of any position (one integer multiplication, no range
// reduction that loses bits at far positions), and its top 32 bits go to
// sincospi, whose error is one ulp of fp32.
//
// Bound by HBM (read and write each element once: 2 or 3 element sizes an
// element).  A group of TP threads owns a row; each thread holds two 16-byte
// vectors of it that contain both members of every pair, so the only
// exchange is the sum for the mean.  The angles of a row are computed once
// and serve every head of the thread's chunk.
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

// kInterleaved is a template parameter so that every register array is
// indexed by constants.
template <typename T, int TP, bool kBwd, bool kInterleaved>
__global__ void __launch_bounds__(kRopeThreads) norm_rope_kernel(const RopeParams p) {
    constexpr int VN = Vec<T>::n;
    constexpr int kRows = kRopeThreads / TP;  // rows a block works on at a time
    constexpr int kU = kBwd ? 1 : 2;          // heads in flight per thread
    const int c = threadIdx.x % TP, slot = threadIdx.x / TP;
    const bool live = c < p.D / (2 * VN);
    const int which = (int)blockIdx.y >= p.t[0].chunks;
    const RopeTensor &t = p.t[which];
    const int chunk = (int)blockIdx.y - (which ? p.t[0].chunks : 0);
    const int h0 = chunk * p.hc, h1 = min(t.heads, h0 + p.hc);

    // the two vectors of this thread, and their pairs' frequencies
    const int nrot = p.rot / (2 * VN);
    int off0, off1;
    if (c < nrot) {
        off0 = kInterleaved ? 2 * VN * c : VN * c;
        off1 = kInterleaved ? off0 + VN : p.rot / 2 + VN * c;
    } else {
        off0 = p.rot + 2 * VN * (c - nrot);
        off1 = off0 + VN;
    }
    uint64_t freq[VN];
    float w[2 * VN];
#pragma unroll
    for (int j = 0; j < VN; ++j) {
        freq[j] = 0;
        if (live && c < nrot) {
            const double turns = p.inv_freq[VN * c + j] * 0.15915494309189533577;
            freq[j] = (uint64_t)((turns - floor(turns)) * 18446744073709551616.0);
        }
        w[j] = live ? t.w[off0 + j] : 0.f;
        w[VN + j] = live ? t.w[off1 + j] : 0.f;
    }
    float dw[2 * VN];
    if (kBwd)
#pragma unroll
        for (int j = 0; j < 2 * VN; ++j) dw[j] = 0.f;

    const float inv_d = 1.f / (float)p.D;
    for (int64_t row0 = (int64_t)blockIdx.x * kRows; row0 < p.rows; row0 += (int64_t)gridDim.x * kRows) {
        const int64_t row = row0 + slot;
        const bool on = live && row < p.rows;
        int64_t base = 0;
        float cs[VN], sn[VN];
        if (row < p.rows) {
            const int64_t b = row / p.S, s = row - b * p.S;
            base = (b * t.heads * p.S + s) * p.D;
            const uint64_t pos = (uint64_t)position_of(p, row, s);
#pragma unroll
            for (int j = 0; j < VN; ++j) {
                const int32_t top = (int32_t)((pos * freq[j]) >> 32);
                sincospif((float)top * 4.656612873077393e-10f, &sn[j], &cs[j]);  // top / 2^31 half turns
            }
        }
        for (int h = h0; h < h1; h += kU) {
            uint4 rx[kU][2], rg[kU][2];
#pragma unroll
            for (int u = 0; u < kU; ++u) {
                rx[u][0] = rx[u][1] = make_uint4(0u, 0u, 0u, 0u);
                rg[u][0] = rg[u][1] = rx[u][0];
                if (on && h + u < h1) {
                    const int64_t at = base + (int64_t)(h + u) * p.S * p.D;
                    const T *x = static_cast<const T *>(t.x) + at;
                    rx[u][0] = *reinterpret_cast<const uint4 *>(x + off0);
                    rx[u][1] = *reinterpret_cast<const uint4 *>(x + off1);
                    if (kBwd) {
                        const T *g = static_cast<const T *>(t.g) + at;
                        rg[u][0] = *reinterpret_cast<const uint4 *>(g + off0);
                        rg[u][1] = *reinterpret_cast<const uint4 *>(g + off1);
                    }
                }
            }
#pragma unroll
            for (int u = 0; u < kU; ++u) {
                if (h + u >= h1) break;  // uniform across the block
                float x[2 * VN], g[2 * VN];
                Vec<T>::unpack(rx[u][0], x);
                Vec<T>::unpack(rx[u][1], x + VN);
                float sum = 0.f, dot = 0.f;
#pragma unroll
                for (int j = 0; j < 2 * VN; ++j) sum = fmaf(x[j], x[j], sum);
                if (kBwd) {
                    Vec<T>::unpack(rg[u][0], g);
                    Vec<T>::unpack(rg[u][1], g + VN);
                    if (row < p.rows) turn<VN>(g, cs, sn, -1.f, kInterleaved);
#pragma unroll
                    for (int j = 0; j < 2 * VN; ++j) dot = fmaf(g[j] * w[j], x[j], dot);
                }
#pragma unroll
                for (int o = TP / 2; o; o >>= 1) {
                    sum += __shfl_xor_sync(0xffffffffu, sum, o);
                    if (kBwd) dot += __shfl_xor_sync(0xffffffffu, dot, o);
                }
                const float r = rsqrtf(sum * inv_d + p.eps);
                if (!on) continue;
                float y[2 * VN];
                if (kBwd) {
                    const float m = r * r * r * (dot * inv_d);
#pragma unroll
                    for (int j = 0; j < 2 * VN; ++j) {
                        dw[j] = fmaf(g[j], x[j] * r, dw[j]);
                        y[j] = r * (g[j] * w[j]) - x[j] * m;
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < 2 * VN; ++j) y[j] = x[j] * r * w[j];
                    turn<VN>(y, cs, sn, 1.f, kInterleaved);
                }
                T *out = static_cast<T *>(t.y) + base + (int64_t)(h + u) * p.S * p.D;
                *reinterpret_cast<uint4 *>(out + off0) = Vec<T>::pack(y);
                *reinterpret_cast<uint4 *>(out + off1) = Vec<T>::pack(y + VN);
            }
        }
    }
    if (kBwd) {
        // the block's share of dw: its rows are summed in a fixed order
        // (within a warp by exchange, over the warps in turn), so the result
        // does not change from run to run
        __shared__ float sum[kRopeThreads / 32][2 * VN * TP];
        const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
#pragma unroll
        for (int j = 0; j < 2 * VN; ++j) {
#pragma unroll
            for (int o = 16; o >= TP; o >>= 1) dw[j] += __shfl_xor_sync(0xffffffffu, dw[j], o);
            if (lane < TP) sum[warp][c * 2 * VN + j] = dw[j];
        }
        __syncthreads();
        if (threadIdx.x < TP && live) {
            float *out = p.parts + ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * p.D;
#pragma unroll
            for (int j = 0; j < 2 * VN; ++j) {
                float v = 0.f;
#pragma unroll
                for (int k = 0; k < kRopeThreads / 32; ++k) v += sum[k][c * 2 * VN + j];
                out[(j < VN ? off0 : off1 - VN) + j] = v;
            }
        }
    }
}

// dw = sum of the blocks' shares, in a fixed order.  One block per 8 columns
// of one weight: 32 threads a column, each adding every 32nd share.
__global__ void __launch_bounds__(256)
    norm_rope_dw_kernel(const float *__restrict__ parts, float *__restrict__ dqw, float *__restrict__ dkw, int nq,
                        int nk, int D) {
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

// Grid: head chunks as large as still give every multiprocessor blocks to
// run (a chunk shares one computation of the angles), then as many row
// blocks as fill the machine.  The block count depends on the sizes only, so
// the backward's shares, and with them dw, do not depend on the device.
constexpr int kRopeBlocks = 152 * 8;

struct RopeGrid {
    int hc, cq, ck, gx;
};

RopeGrid rope_grid(int64_t rows, int64_t H, int64_t Hkv, int tp) {
    const int64_t per = kRopeThreads / tp;
    const int64_t blocks = (rows + per - 1) / per;
    RopeGrid g{};
    g.hc = 8;
    auto chunks = [&](int64_t heads) { return (heads + g.hc - 1) / g.hc; };
    while (g.hc > 1 && blocks * (chunks(H) + chunks(Hkv)) < kRopeBlocks / 2) g.hc /= 2;
    g.cq = (int)chunks(H);
    g.ck = (int)chunks(Hkv);
    const int64_t most = (kRopeBlocks + g.cq + g.ck - 1) / (g.cq + g.ck);
    g.gx = (int)(blocks < most ? blocks : most);
    return g;
}

int rope_tp(int64_t D, int dtype) {
    const int64_t need = D / (dtype == STRIPED_BF16 ? 16 : 8);
    int tp = 1;
    while (tp < need) tp *= 2;
    return tp;
}

template <typename T, int TP, bool kBwd>
int launch_tp(const RopeParams &p, const RopeGrid &g, cudaStream_t stream) {
    const dim3 grid((unsigned)g.gx, (unsigned)(g.cq + g.ck));
    if (p.interleaved) norm_rope_kernel<T, TP, kBwd, true><<<grid, kRopeThreads, 0, stream>>>(p);
    else norm_rope_kernel<T, TP, kBwd, false><<<grid, kRopeThreads, 0, stream>>>(p);
    return cuda_status(cudaGetLastError());
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
    const RopeGrid g = rope_grid(B * S, H, Hkv, rope_tp(D, dtype));
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
    p.L = a.stripe >= 0 ? a.S : a.S / a.N;
    p.D = (int)a.D;
    p.rot = a.rot;
    p.interleaved = a.interleaved;
    p.N = a.N;
    p.layout = a.layout;
    p.stripe = a.stripe;
    p.eps = a.eps;
    p.parts = static_cast<float *>(a.workspace);
    const int tp = rope_tp(a.D, a.dtype);
    const RopeGrid g = rope_grid(p.rows, a.H, a.Hkv, tp);
    if (g.cq + g.ck > 65535) return STRIPED_ERR_UNSUPPORTED;
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
    norm_rope_dw_kernel<<<dim3((unsigned)((a.D + 7) / 8), 2), 256, 0, stream>>>(
        p.parts, a.dq_weight, a.dk_weight, g.gx * g.cq, g.gx * g.ck, (int)a.D);
    return cuda_status(cudaGetLastError());
}

}  // namespace striped
