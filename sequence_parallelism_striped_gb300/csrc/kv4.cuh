// kv4.cuh -- rows of a key/value cache held in 4 bits.
//
// A group of 32 channels of one row has the scale
//     s = amax / 7 rounded to 5 significant bits (to nearest, ties to even),
// 0 where amax < 2^-100, and the codes c = x / s rounded to nearest (ties to
// even), -7 .. 7.  A value c * s has 3 + 5 significant bits: it IS a bf16
// number, so that a product on the tensor cores takes a stored row without a
// further rounding, whether the scale is multiplied in before it or after.
// (5 bits instead of the 8 that bf16 has: the scale is at most 3 % too large
// or too small, which costs nothing: over normal values, groups of 32, the
// error is 9.6 % of their root mean square, with 8 bits 9.5 %.)
//
// A 32-bit word holds 8 consecutive channels, code + 8 of channel c at bit
// 16 (c mod 2) + 4 (c / 2): (w >> 4 j) & 0x000f000f is the pair of channels 2 j
// and 2 j + 1, in the halves that a bf16 pair has.
#pragma once

#include <stdint.h>

namespace striped {

constexpr int kKv4Group = 32;

// Codes + 8 of pair j (0 .. 3) of a word as bf16 numbers 128 + code + 8:
// 0x4300 is 128, one unit in its last place is 1.
__device__ __forceinline__ uint32_t kv4_biased(uint32_t w, int j) {
    return ((w >> (4 * j)) & 0x000f000fu) | 0x43004300u;
}
__device__ __forceinline__ uint32_t bf16x2_sub(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ uint32_t bf16x2_mul(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
// The codes of pair j as whole bf16 numbers (exact: 128 + 15 has 8 bits).
__device__ __forceinline__ uint32_t kv4_codes(uint32_t w, int j) { return bf16x2_sub(kv4_biased(w, j), 0x43084308u); }

// The codes of all four pairs, times 2^-6, at 5 operations of the integer pipe
// instead of 7 (it has half the rate of the others and bounds what reads 4-bit
// rows).  A bf16 number whose bits are the whole number n < 256 is n * 2^-133:
// the first normal binade goes on where the subnormals end.  So codes + 8 in
// the low or in the high nibble of a byte are numbers as they stand, and one
// fused multiply-add makes (code + 8 - 8) * 2^-6 of them, exactly.
constexpr float kKv4Unit = 64.f;  // undoes the 2^-6
__device__ __forceinline__ uint32_t bf16x2_fma(uint32_t a, uint32_t b, uint32_t c) {
    uint32_t r;
    asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
    return r;
}
// Scores of keys made so are 2^-6 of themselves.  The scale of the softmax undoes
// that, up to where 64 of it times log2(e) is still a number; beyond it (1e38 is
// allowed) the queries do, 64 of them, which is exact below 2^122.
constexpr float kKv4MostScale = 3.6e36f;
constexpr uint32_t kKv4Query = 0x42804280u;  // 64, 64
__device__ __forceinline__ void kv4_pairs(uint32_t w, uint32_t (&c)[4]) {
    constexpr uint32_t k2e127 = 0x7f007f00u, k2e123 = 0x7d007d00u, kMinus8th = 0xbe00be00u;
    const uint32_t h = w >> 8;
    c[0] = bf16x2_fma(w & 0x000f000fu, k2e127, kMinus8th);
    c[1] = bf16x2_fma(w & 0x00f000f0u, k2e123, kMinus8th);
    c[2] = bf16x2_fma(h & 0x000f000fu, k2e127, kMinus8th);
    c[3] = bf16x2_fma(h & 0x00f000f0u, k2e123, kMinus8th);
}

}  // namespace striped
