// frames_common.cuh -- device code shared by the frame-aware attention kernels: the bias by
// frame distance, the frames that a tile of keys covers, and the reading of e4m3 codes as f16.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "frames_internal.cuh"

namespace skiparse {

constexpr float kLog2E = 1.4426950408889634f;

// Bias of distance index u (0..2D) for one head as the table's bf16, kBiasNone (-inf) where masked.
constexpr uint16_t kBiasNone = 0xff80;
__device__ __forceinline__ uint16_t bias_bf16(const FrameBias& fb, int heads, int u, int head) {
    const int g = fb.buckets[u];
    if (g < 0 || g >= fb.NB) return kBiasNone;
    const uint16_t b = fb.table[static_cast<size_t>(g) * heads + head];
    return __uint_as_float(static_cast<uint32_t>(b) << 16) < kBiasMasked ? kBiasNone : b;
}
// The same in units of log2, -inf where masked; 0 without a table.
__device__ __forceinline__ float bias_log2(const FrameBias& fb, int heads, int u, int head) {
    return fb.table ? __uint_as_float(static_cast<uint32_t>(bias_bf16(fb, heads, u, head)) << 16) * kLog2E : 0.f;
}

__device__ __forceinline__ int clamp_dist(int u, int D) { return min(max(u, -D), D); }

// The frames that hold keys for a call whose newest frame is end-1, in a ring of cap slots (cap
// = end for keys that do not lie in a ring), and the frame number of each slot.
struct FrameRing {
    int nframes;   // slots with keys: [0, nframes)
    int newest;    // slot of the newest frame; a slot beyond it is one turn of the ring older
    int base;      // frame number of slot f <= newest: f + base
    int cap;
    bool wrapped;  // every slot is in use, in no order of time
    __device__ __forceinline__ void init(int end, int cap_) {
        cap = cap_;
        wrapped = end > cap;
        nframes = wrapped ? cap : end;
        newest = wrapped ? (end - 1) % cap : nframes;
        base = wrapped ? end - 1 - newest : 0;
    }
    __device__ __forceinline__ int time(int slot) const { return slot + base - (slot > newest ? cap : 0); }
    // Slots [f_lo, f_hi] that some query of frames [ta, tb] can see when the visible distances lie
    // in [dlo, dhi] (the end distances +-D stand for all beyond them; dlo > dhi: none is visible).
    // All slots of a wrapped ring are taken, hidden ones too: they lie in no order of time.
    __device__ __forceinline__ void visible(int ta, int tb, int dlo, int dhi, int D, int& f_lo, int& f_hi) const {
        f_lo = 0;
        f_hi = nframes - 1;
        if (!wrapped) {
            if (dhi < D) f_lo = max(f_lo, ta - dhi);
            if (dlo > -D) f_hi = min(f_hi, tb - dlo);
        }
        if (dlo > dhi) f_hi = f_lo - 1;
    }
};

// Fills tab[0..2D] with the bias of one head by distance index, in log2; returns this thread's first
// and last visible distance in dlo, dhi.
__device__ __forceinline__ void fill_bias(float* tab, const FrameBias& fb, int heads, int head, int nthreads, int& dlo,
                                          int& dhi) {
    dlo = fb.D + 1;
    dhi = -fb.D - 1;
    for (int u = threadIdx.x; u <= 2 * fb.D; u += nthreads) {
        const float v = bias_log2(fb, heads, u, head);
        tab[u] = v;
        if (v != -INFINITY) {
            dlo = min(dlo, u - fb.D);
            dhi = max(dhi, u - fb.D);
        }
    }
}

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
// 2^(byte - ref) as an f16 pair, byte <= ref: exact down to 2^-24, 0 below (where the codes enter unscaled and this
// is not used); NaN for byte 255.
__device__ __forceinline__ uint32_t scale_f16x2(uint32_t byte, int ref) {
    const int down = ref - static_cast<int>(byte);
    uint32_t h = down <= 14 ? static_cast<uint32_t>(15 - down) << 10 : down <= 24 ? 1u << (24 - down) : 0u;
    if (byte == 255u) h = 0x7e00u;
    return h | (h << 16);
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
// P is kept as 2^7 p in f16: the lazy rescale lets p grow to 2^8, and 2^15 < 65504.
constexpr float kPShift = 7.f;

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
