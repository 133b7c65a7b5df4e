// kv4.cu -- keys and values stored in 4 bits (kv4.cuh) and read back.
//
// Both directions are one pass over memory: 2 bytes a value on one side, 1/2
// and 1/16 on the other.  A lane has 8 channels of a row (16 bytes of bf16, one
// word of codes), so a group is four neighbouring lanes, every access of a warp
// is whole lines, and the group's maximum takes two exchanges.  Measured, 2 x 8
// heads of 131072 rows, D = 128: stored in 107 and read back in 99 us, both at
// 99 % of a copy's rate (that a NaN passes through the maximum costs 0.6 us).
#include <cuda_bf16.h>

#include "common.cuh"
#include "internal.h"
#include "kv4.cuh"

namespace striped {

namespace {

constexpr int kKThreads = 256;
constexpr int kKUnroll = 4;  // vectors of a thread: their loads are in flight together

struct Kv4Args {
    const uint4 *x[2];      // keys, values (load: written)
    uint32_t *codes[2];
    __nv_bfloat16 *scales[2];
    int64_t n;              // vectors of 8 channels in each
};

// x / s to the nearest whole number, + 8, in the low bits: x / s is first
// rounded to a multiple of 2^-11.  A quotient of a number of 8 significant
// bits and one of 5 is either a tie (n + 1/2) or at least 2^-9 away from one
// (255 / 16 times 2^-5 is 1/2 - 2^-9).  Half a step of the rounding, 2^-12, and
// the error of the product with the rounded 1 / s, below 2^-20, are less than
// that: the result falls on the side of the tie, or on the tie, that the
// quotient is on.
__device__ __forceinline__ uint32_t kv4_pack(const float (&x)[8], float inv) {
    constexpr float kSnap = 0x1.8p12f, kRound = 0x1.8p23f + 8.f;
    const uint64_t inv2 = f2(inv, inv), snap = f2(kSnap, kSnap), round = f2(kRound, kRound);
    uint32_t w = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const float2 r = f2_split(add2(sub2(fma2(f2(x[2 * j], x[2 * j + 1]), inv2, snap), snap), round));
        w += ((__float_as_uint(r.x) & 15u) << (4 * j)) + ((__float_as_uint(r.y) & 15u) << (16 + 4 * j));
    }
    return w;
}

// Maxima that a NaN passes through.
__device__ __forceinline__ float fmax_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float fmax3_nan(float a, float b, float c) {
    float r;
    asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

__global__ void __launch_bounds__(kKThreads) kv4_store_kernel(const Kv4Args a) {
    const bool second = blockIdx.y != 0;
    const uint4 *x = second ? a.x[1] : a.x[0];
    uint32_t *codes = second ? a.codes[1] : a.codes[0];
    __nv_bfloat16 *scales = second ? a.scales[1] : a.scales[0];
    const int64_t v0 = (int64_t)blockIdx.x * (kKThreads * kKUnroll) + threadIdx.x;
    uint4 in[kKUnroll];
#pragma unroll
    for (int u = 0; u < kKUnroll; ++u) {
        const int64_t v = v0 + u * kKThreads;
        in[u] = v < a.n ? __ldcs(x + v) : make_uint4(0u, 0u, 0u, 0u);
    }
#pragma unroll
    for (int u = 0; u < kKUnroll; ++u) {
        const int64_t v = v0 + u * kKThreads;
        const uint32_t raw[4] = {in[u].x, in[u].y, in[u].z, in[u].w};
        float f[8], top = 0.f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            f[2 * j] = __uint_as_float(raw[j] << 16);
            f[2 * j + 1] = __uint_as_float(raw[j] & 0xffff0000u);
            top = fmax3_nan(top, fabsf(f[2 * j]), fabsf(f[2 * j + 1]));
        }
        // all lanes of a warp are here: groups never straddle the end (n is a
        // multiple of 4)
        top = fmax_nan(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = fmax_nan(top, __shfl_xor_sync(0xffffffffu, top, 2));
        const uint32_t t = __float_as_uint(top / 7.f);
        // to 5 significant bits: the lowest 19 of the 23 fraction bits go (a NaN
        // stays one: the group's values are NaN, whatever their codes)
        float s = top < 0x1p-100f ? 0.f : __uint_as_float((t + 0x3ffffu + ((t >> 19) & 1u)) & 0xfff80000u);
        if (top != top) s = top;
        const uint32_t w = kv4_pack(f, s > 0.f ? 1.f / s : 0.f);
        if (v < a.n) {
            codes[v] = w;
            if ((threadIdx.x & 3) == 0) scales[v >> 2] = __float2bfloat16_rn(s);
        }
    }
}

__global__ void __launch_bounds__(kKThreads) kv4_load_kernel(const Kv4Args a) {
    const bool second = blockIdx.y != 0;
    uint4 *y = const_cast<uint4 *>(second ? a.x[1] : a.x[0]);
    const uint32_t *codes = second ? a.codes[1] : a.codes[0];
    const unsigned short *scales = reinterpret_cast<const unsigned short *>(second ? a.scales[1] : a.scales[0]);
    const int64_t v0 = (int64_t)blockIdx.x * (kKThreads * kKUnroll) + threadIdx.x;
    uint32_t w[kKUnroll], s[kKUnroll];
#pragma unroll
    for (int u = 0; u < kKUnroll; ++u) {
        const int64_t v = v0 + u * kKThreads;
        w[u] = v < a.n ? __ldcs(codes + v) : 0u;
        s[u] = v < a.n ? __ldcs(scales + (v >> 2)) : 0u;
    }
#pragma unroll
    for (int u = 0; u < kKUnroll; ++u) {
        const int64_t v = v0 + u * kKThreads;
        if (v >= a.n) continue;
        const uint32_t s2 = s[u] | (s[u] << 16);
        __stcs(y + v, make_uint4(bf16x2_mul(kv4_codes(w[u], 0), s2), bf16x2_mul(kv4_codes(w[u], 1), s2),
                                 bf16x2_mul(kv4_codes(w[u], 2), s2), bf16x2_mul(kv4_codes(w[u], 3), s2)));
    }
}

}  // namespace

int launch_kv4(void *k, void *k_codes, void *k_scales, void *v, void *v_codes, void *v_scales, int64_t rows, int64_t D,
               bool store, cudaStream_t stream) {
    Kv4Args a{};
    a.x[0] = static_cast<const uint4 *>(k);
    a.x[1] = static_cast<const uint4 *>(v);
    a.codes[0] = static_cast<uint32_t *>(k_codes);
    a.codes[1] = static_cast<uint32_t *>(v_codes);
    a.scales[0] = static_cast<__nv_bfloat16 *>(k_scales);
    a.scales[1] = static_cast<__nv_bfloat16 *>(v_scales);
    a.n = rows * (D / 8);
    const int64_t per = kKThreads * kKUnroll, blocks = (a.n + per - 1) / per;
    if (blocks > 0x7fffffff) return STRIPED_ERR_UNSUPPORTED;
    const dim3 grid((unsigned)blocks, 2);
    if (store) kv4_store_kernel<<<grid, kKThreads, 0, stream>>>(a);
    else kv4_load_kernel<<<grid, kKThreads, 0, stream>>>(a);
    return cuda_status(cudaGetLastError());
}

}  // namespace striped
