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

// e4m3 codes as f16 pairs: every code is an f16 value exactly.
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint16_t codes) {
    uint32_t r;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(codes));
    return r;
}
__device__ __forceinline__ uint32_t f16x2_mul(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
// 2^(byte - ref) as an f16 pair, byte <= ref: exact down to 2^-24, 0 below; NaN for byte 255.
__device__ __forceinline__ uint32_t scale_f16x2(uint32_t byte, int ref) {
    const int down = ref - static_cast<int>(byte);
    uint32_t h = down <= 14 ? static_cast<uint32_t>(15 - down) << 10 : down <= 24 ? 1u << (24 - down) : 0u;
    if (byte == 255u) h = 0x7e00u;
    return h | (h << 16);
}
// 2^e in fp32, e clamped to its normal range.
__device__ __forceinline__ float exp2_int(int e) {
    return __uint_as_float(static_cast<uint32_t>(min(max(e, -126), 127) + 127) << 23);
}
// Byte offset of 16-byte chunk c of row r in a tile of TileGeom<D>'s swizzled layout.
template <int D>
__device__ __forceinline__ uint32_t tile_chunk(int r, int c) {
    using C = TileGeom<D>;
    const uint32_t box = static_cast<uint32_t>(c * 16) / C::SW, cb = static_cast<uint32_t>(c * 16) % C::SW / 16;
    const uint32_t sw = C::SW == 128 ? static_cast<uint32_t>(r & 7) : static_cast<uint32_t>((r >> 1) & 3);
    return box * C::BOX_BYTES + static_cast<uint32_t>(r) * C::SW + ((cb ^ sw) << 4);
}

}  // namespace skiparse
