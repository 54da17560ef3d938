// frames_common.cuh -- device code shared by the frame-aware attention kernels: the bias by
// frame distance, the frames that a tile of keys covers, and the reading of e4m3 codes as bf16.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "attn_common.cuh"
#include "frames_internal.cuh"

namespace skiparse {

constexpr float kLog2E = 1.4426950408889634f;

// Bias of distance index u (0..2D) for one head in units of log2, -inf where masked.
__device__ __forceinline__ float bias_log2(const FrameBias& fb, int heads, int u, int head) {
    if (!fb.table) return 0.f;
    const int g = fb.buckets[u];
    if (g < 0 || g >= fb.NB) return -INFINITY;
    const float b = __uint_as_float(static_cast<uint32_t>(fb.table[static_cast<size_t>(g) * heads + head]) << 16);
    return b < kBiasMasked ? -INFINITY : b * kLog2E;
}

__device__ __forceinline__ int clamp_dist(int u, int D) { return min(max(u, -D), D); }

// The four e4m3 codes of a word as bf16, times a power of two m (as a bf16 pair): an e4m3 code's
// exponent and mantissa, moved to the low bits of bf16's fields, are its value times 2^-120 (a
// subnormal code becomes a bf16 subnormal), so with m = 2^(120 + e) the product is code * 2^e,
// exactly: three mantissa bits fit bf16's seven.
__device__ __forceinline__ uint32_t bf16x2_mul(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ uint32_t e4m3_pair_raw(uint32_t x) {  // codes in bytes 1 and 3 of x
    return ((x >> 4) & 0x07f007f0u) | (x & 0x80008000u);
}
__device__ __forceinline__ void e4m3x4_to_bf16(uint32_t w, uint32_t m, uint32_t& lo, uint32_t& hi) {
    lo = bf16x2_mul(e4m3_pair_raw(__byte_perm(w, 0u, 0x1404)), m);
    hi = bf16x2_mul(e4m3_pair_raw(__byte_perm(w, 0u, 0x3424)), m);
}
// The bf16 pair 2^(120 + e) of a scale byte e + 127, for e <= 7; beyond, the largest power, and
// the caller multiplies by scale_rest() too. 255 is NaN.
__device__ __forceinline__ uint32_t scale_mul(uint32_t byte) {
    const uint32_t f = byte >= 255u ? 0x7fc0u : (min(byte, 134u) + 120u) << 7;
    return f | (f << 16);
}
__device__ __forceinline__ uint32_t scale_rest(uint32_t byte) {
    const uint32_t f = byte > 134u ? (byte - 134u + 127u) << 7 : 127u << 7;
    return (f | (f << 16)) & 0x7fff7fffu;
}

}  // namespace skiparse
