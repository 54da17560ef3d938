// cache_append.cu -- writes new frames' keys and values into the e4m3 frame cache.
//
// For every class, head and new frame, each block of 64 class tokens x d values shares a scale
// 2^e, e the smallest whole number with max|x| <= 448 * 2^e (448: e4m3's largest value; e at
// least -110), and is stored as codes RNE(x / 2^e): one rounding, of half a step of e4m3. A
// power of two makes the scaling exact in both directions, and the attention kernels can give
// the codes to the tensor cores as f16 without a second rounding. A block that holds an
// infinity or a NaN is stored with a NaN scale.
//
// 2 bytes read and 1 written per value. One CTA of 256 threads per block and head of
// K or V holds the block's 64 * d values in registers (16-byte loads; a token's d values are one
// contiguous row of its head) between the maximum and the conversion, so the input is read once.
// Heads are the fastest grid dimension: CTAs that run together read the neighbouring heads of
// the same tokens, and write 64 * d contiguous bytes each. Eight CTAs an SM, which takes at most 32
// registers a thread: at 36, one CTA fewer, both cases below took a third longer. Measured: two 480p clips of 21
// frames (604 MB in and out) 96 to 104 us, bound by HBM as much as by its issue slots (83 % busy; 403 MB read from
// DRAM, 141 written by its end); a 720p frame (111 MB) 18 to 20 us, of which DRAM has 74 MB read and 4 written (the
// rest stays in L2): there the issue slots (65 to 69 % busy) and the launch bound it, not HBM.
#include <cuda_runtime.h>

#include "frames_common.cuh"

namespace skiparse {
namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ uint16_t e4m3x2(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

template <int D>
__global__ void __launch_bounds__(kThreads, 8) skiparse_cache_append_kernel(const AppendParams p) {
    constexpr int CPR = D / 8;                       // 16-byte chunks of a row
    constexpr int PER = kCacheBlock * CPR / kThreads;  // chunks of a thread (1, 2, 4)
    static_assert(PER >= 1, "block too small");
    const int head = blockIdx.x % p.g.heads;
    const int blk = blockIdx.x / p.g.heads % p.nblk;
    const int t = blockIdx.x / p.g.heads / p.nblk;
    const int seq = blockIdx.y;
    const bool is_v = blockIdx.z;
    ClassView cls;
    cls.init(p.g, seq);
    const int nF = cls.nF;
    const int first = blk * kCacheBlock;
    if (first >= nF) return;
    const int start = p.cache.start[cls.b];
    if (start < 0 || start > kMaxStart) return;
    const int slot = (start + t) % p.cache.cap;
    const uint16_t* src = is_v ? p.v : p.k;
    // rows of the block's tokens, each computed once
    __shared__ int row_of[kCacheBlock];
    if (threadIdx.x < kCacheBlock && first + threadIdx.x < nF) {
        const RowMap rows = cls.rows(p.g, head);
        row_of[threadIdx.x] = static_cast<int>(load_row(rows(t * nF + first + threadIdx.x), p.nrows, p.status));
    }
    __syncthreads();

    uint4 x[PER];
    uint32_t top = 0;  // bits of the largest magnitude, two at a time
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int ch = threadIdx.x + i * kThreads;
        const int tok = first + ch / CPR;
        x[i] = make_uint4(0u, 0u, 0u, 0u);
        if (tok < nF) {
            const uint4* at = reinterpret_cast<const uint4*>(src + static_cast<size_t>(row_of[ch / CPR]) * D) + ch % CPR;
            asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(x[i].x), "=r"(x[i].y), "=r"(x[i].z), "=r"(x[i].w)
                         : "l"(at));
        }
    }
#pragma unroll
    for (int i = 0; i < PER; ++i) {  // bf16 magnitudes compare as integers
        const uint32_t a = __vmaxu2(x[i].x & 0x7fff7fffu, x[i].y & 0x7fff7fffu);
        const uint32_t e = __vmaxu2(x[i].z & 0x7fff7fffu, x[i].w & 0x7fff7fffu);
        top = __vmaxu2(top, __vmaxu2(a, e));
    }
    top = max(top & 0xffffu, top >> 16);
    __shared__ uint32_t warp_top[kThreads / 32];
    top = __reduce_max_sync(0xffffffffu, top);
    if ((threadIdx.x & 31) == 0) warp_top[threadIdx.x >> 5] = top;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kThreads / 32; ++i) top = max(top, warp_top[i]);

    // top = 2^(E-127) * (1 + M/128): the scale's exponent is E - 127 - 8, one more where
    // 1 + M/128 > 448 / 256 = 1.75
    const int E = top >> 7, M = top & 127;
    const bool bad = E == 255;
    const int byte = bad ? 255 : max(E - 8 + (M > 96 ? 1 : 0), kScaleLow);
    const float f = __uint_as_float(bad ? 0x7fc00000u : static_cast<uint32_t>(254 - byte) << 23);  // 2^-e
    const long long sh = static_cast<long long>(seq) * p.g.heads + head;
    uint8_t* dst = (is_v ? p.cache.v : p.cache.k) + ((sh * p.cache.cap + slot) * p.cache.F + first) * D;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int ch = threadIdx.x + i * kThreads;
        if (first + ch / CPR >= nF) continue;
        const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
        uint32_t r[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const float a0 = __uint_as_float(w[2 * j] << 16) * f;
            const float a1 = __uint_as_float(w[2 * j] & 0xffff0000u) * f;
            const float a2 = __uint_as_float(w[2 * j + 1] << 16) * f;
            const float a3 = __uint_as_float(w[2 * j + 1] & 0xffff0000u) * f;
            r[j] = e4m3x2(a0, a1) | (static_cast<uint32_t>(e4m3x2(a2, a3)) << 16);
        }
        *reinterpret_cast<uint2*>(dst + ch * 8) = make_uint2(r[0], r[1]);
    }
    if (threadIdx.x == 0)
        (is_v ? p.cache.vs : p.cache.ks)[(sh * p.cache.cap + slot) * p.cache.NBk + blk] = static_cast<uint8_t>(byte);
}

}  // namespace

int launch_cache_append(const AppendParams& p, const Geometry& g, int d, void* stream) {
    const dim3 grid(static_cast<unsigned>(g.heads) * p.nblk * g.T, g.B * g.Ph * g.Pw, 2);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    switch (d) {
        case 32: skiparse_cache_append_kernel<32><<<grid, kThreads, 0, st>>>(p); break;
        case 64: skiparse_cache_append_kernel<64><<<grid, kThreads, 0, st>>>(p); break;
        case 128: skiparse_cache_append_kernel<128><<<grid, kThreads, 0, st>>>(p); break;
        default: return static_cast<int>(cudaErrorInvalidValue);
    }
    return static_cast<int>(cudaGetLastError());
}

}  // namespace skiparse
