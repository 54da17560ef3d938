// attn_cached_small.cu -- attention of few queries per class over the e4m3 frame cache (sm_100a).
//
// Frame by frame, a class of a small latent has one or a few dozen queries, and what bounds the
// call is reading the cache: two codes per key and value of d. The tcgen05 kernel would expand
// every key into shared memory for tiles that are mostly empty. Here a warp keeps 8 to 32 queries in
// registers and walks over groups of 16 keys with m16n8k16 products (legacy tensor-core path;
// the codes never leave registers after their copy), keys as the products' 16 rows and queries as
// their 8 columns, so that a call of up to 8 queries a class wastes no product:
//   * S^T = K Q^T. The product does not care in which order d is summed, so a lane takes 16
//     consecutive codes of its key as four K-steps, and Q's fragments are loaded in the same order.
//   * O^T += V^T P^T. P^T is S^T's accumulators as f16, each 8 x 8 block transposed by movmatrix.
//     V^T's operand pairs two keys of one column: two byte permutations and four conversions per
//     four columns of two keys; columns are dealt to the product's rows so that a lane needs one
//     chunk of each of its four keys.
//   * Scales. K's is a factor of the score. V's, 2^e, joins the exponent of the weight:
//     w = 2^(s + e - mv) with a running maximum mv of s + e of its own, beside p = 2^(s - m) for the
//     row sum. So P V needs no common scale, and f16 holds every weight down to 2^-31 of the
//     largest; out = O 2^(mv - m) / l.
//   * Copies go by cp.async into a ring of three stages per warp that only the copying lane
//     reads: no barrier in the loop, 8 KB in flight per warp at d = 128.
// What bounds it: reading the cache, as long as a step's instructions (conversions foremost: 64 per
// lane and step at d = 128, 4 clocks each) keep below the 180 clocks in which an SM's share
// of HBM delivers its 4 KB. Measured, d = 128, one query a class, 192 classes and heads of 8000 keys (396 MB):
// 87 to 90 us, 4.4 to 4.5 TB/s; d = 64, 12 to 20 queries a class, 64 of 4000 to 6700 keys (43 MB): 29 to 32 us, the
// latency of 12 warps an SM; d = 128, 20 queries a class, 48 of 58,000 keys (713 MB): 340 us, 2.1 TB/s.
// Key groups are dealt to the warps of a CTA and, over long caches, to `splits` CTAs; warps join
// through shared memory, CTAs through the join kernel of attn_frames_fwd_sm100.cu. A CTA has
// 8, 16, 24 or 32 queries.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <atomic>

#include "frames_common.cuh"

namespace skiparse {
namespace {

constexpr int kWarps = 4;
constexpr int kKeys = 16;      // keys of a warp step
constexpr int kStages = 3;
constexpr int kMaxRows = 32;   // queries per class up to which this kernel is used (measured, 57,000 keys,
                               // d = 128: 30 queries 0.49 ms against the tcgen05 kernel's 0.80, 64: 0.89, 0.52)
constexpr float kRescaleLog2 = 8.0f;

template <int D, int NQ>  // NQ: tiles of 8 queries of a CTA
struct SmallCfg {
    static constexpr int ROWS = 8 * NQ;
    static constexpr int KL = D == 128 ? 2 : 1;       // copies of a key by a lane
    static constexpr int STAGE_BYTES = (2 * KL + 4) * 512;           // of one warp: 16 keys of K and of V
    static constexpr int STAGES_BYTES = kWarps * kStages * STAGE_BYTES;
    static constexpr int MERGE_BYTES = kWarps * ROWS * (D + 3) * 4;  // over the stages, after the loop
    static constexpr int OFF_TABLE = STAGES_BYTES > MERGE_BYTES ? STAGES_BYTES : MERGE_BYTES;
    static constexpr int OFF_RANGE = OFF_TABLE + 4 * (kMaxDistEntries + 1);
    static constexpr int SMEM_BYTES = OFF_RANGE + 8;
    static constexpr int KB = D == 128 ? 16 : D / 4;  // bytes of such a copy
    static constexpr int VB = D / 8;                  // bytes of a lane's copy of a value
    static constexpr int KSTEPS = D / 16;
    static constexpr int MT = D / 16;                 // row tiles of O^T
    // per SM, by registers: at d = 64 and 32 these counts spill nothing; at d = 128, three tiles (held to 168
    // registers) spill 260 bytes a thread and four (255) 180, which other counts were not measured against
    static constexpr int CTAS = NQ == 4 ? 2 : NQ == 1 ? 4 : 3;
};

template <int BYTES>
__device__ __forceinline__ void cp_async_n(uint32_t dst, const void* src) {
    if (BYTES == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(dst), "l"(src), "n"(BYTES) : "memory");
}

// BYTES of this lane's staged data as words.
template <int BYTES>
__device__ __forceinline__ void ld_words(uint32_t (&w)[BYTES / 4], uint32_t at) {
    if constexpr (BYTES == 16)
        asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "r"(at));
    else if constexpr (BYTES == 8)
        asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(at));
    else
        asm volatile("ld.shared.b32 %0, [%1];" : "=r"(w[0]) : "r"(at));
}

__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// The 8 x 8 f16 matrix of a warp transposed: a lane's pair is row lane/4, columns 2 (lane%4) and + 1.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

template <int D, int NQ>
__global__ void __launch_bounds__(32 * kWarps, SmallCfg<D, NQ>::CTAS)
    skiparse_cached_small_kernel(const FramesFwdParams p) {
    using C = SmallCfg<D, NQ>;
    const int split = blockIdx.x;
    const int head = blockIdx.y;
    const int seq = blockIdx.z;
    ClassView cls;
    cls.init(p.g, seq);
    const int nF = cls.nF;
    const FastDiv dF = cls.dF;
    const int n_q = p.g.T * nF;  // at most C::ROWS
    if (n_q == 0) return;
    const int start = p.cache.start[cls.b];
    if (start < 0 || start > kMaxStart) return;
    FrameRing ring;
    ring.init(start + p.g.T, p.cache.cap);
    const RowMap rows = cls.rows(p.g, head);

    extern __shared__ __align__(16) uint8_t smem[];
    const uint32_t sbase = ptx::smem_u32(smem);
    float* tab = reinterpret_cast<float*>(smem + C::OFF_TABLE);
    int* range = reinterpret_cast<int*>(smem + C::OFF_RANGE);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g = lane >> 2, c = lane & 3;
    const int dmax = p.bias.D;
    if (threadIdx.x == 0) {
        range[0] = dmax + 1;
        range[1] = -dmax - 1;
    }
    __syncthreads();
    int dlo, dhi;
    fill_bias(tab, p.bias, p.g.heads, head, 32 * kWarps, dlo, dhi);
    dlo = __reduce_min_sync(0xffffffffu, dlo);
    dhi = __reduce_max_sync(0xffffffffu, dhi);
    if (lane == 0 && dlo <= dhi) {
        atomicMin(&range[0], dlo);
        atomicMax(&range[1], dhi);
    }
    __syncthreads();
    int f_lo, f_hi;
    ring.visible(start, start + p.g.T - 1, range[0], range[1], dmax, f_lo, f_hi);
    const int groups = f_hi >= f_lo ? ((f_hi - f_lo + 1) * nF + kKeys - 1) / kKeys : 0;
    const int per_split = (groups + p.plan.splits - 1) / p.plan.splits;
    const int jend = (f_hi + 1) * nF;
    const int jbeg = f_lo * nF + split * per_split * kKeys;
    const int mygroups = max(0, min(per_split, groups - split * per_split));
    const int steps = (mygroups - warp + kWarps - 1) / kWarps;  // groups warp, warp + kWarps, ...

    const long long sh = static_cast<long long>(seq) * p.g.heads + head;
    const int crows = p.cache.cap * p.cache.F;  // rows of a (subsequence, head); at most 2^30
    const uint8_t* kc = p.cache.k + sh * crows * D + c * C::KB;
    const uint8_t* vc = p.cache.v + sh * crows * D + g * C::VB;
    const uint8_t* ks = p.cache.ks + sh * p.cache.cap * p.cache.NBk;
    const uint8_t* vs = p.cache.vs + sh * p.cache.cap * p.cache.NBk;
    const uint32_t my_stage = sbase + warp * kStages * C::STAGE_BYTES + lane * 16;
    const int gap = p.cache.F - nF;  // unused places of a slot

    // row in the cache of the class's key j
    auto key_row = [&](int j) -> long long {
        return load_row(j + static_cast<long long>(dF.div(j)) * gap, crows, p.status);
    };
    auto copy_key = [&](uint32_t at, int n, const uint8_t* src) {
#pragma unroll
        for (int l = 0; l < C::KL; ++l) cp_async_n<C::KB>(at + (n * C::KL + l) * 512, src + l * 64);
    };
    // Copies the group of a step: lane's keys g and g + 8, lane's values 2c, 2c + 1, 2c + 8, 2c + 9. Every
    // copy has 16 bytes of a stage to itself per lane, whatever its size.
    auto fetch = [&](int step) {
        if (step < steps) {
            const int j0 = jbeg + (step * kWarps + warp) * kKeys;
            const uint32_t at = my_stage + (step % kStages) * C::STAGE_BYTES;
            const int slot0 = dF.div(j0);
            if (j0 + kKeys <= jend && (gap == 0 || j0 + kKeys <= (slot0 + 1) * nF)) {  // consecutive rows
                const long long last = load_row(j0 + kKeys - 1 + static_cast<long long>(slot0) * gap, crows, p.status);
                const long long r0 = max(last - (kKeys - 1), 0ll);
                const uint8_t* ksrc = kc + (r0 + g) * D;
                const uint8_t* vsrc = vc + (r0 + 2 * c) * D;
                copy_key(at, 0, ksrc);
                copy_key(at, 1, ksrc + 8 * D);
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    cp_async_n<C::VB>(at + (2 * C::KL + k) * 512, vsrc + ((k & 1) + 8 * (k >> 1)) * D);
            } else {
                copy_key(at, 0, kc + key_row(min(j0 + g, jend - 1)) * D);
                copy_key(at, 1, kc + key_row(min(j0 + g + 8, jend - 1)) * D);
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    cp_async_n<C::VB>(at + (2 * C::KL + k) * 512, vc + key_row(min(j0 + 2 * c + (k & 1) + 8 * (k >> 1), jend - 1)) * D);
            }
        }
        cp_async_commit();
    };
#pragma unroll
    for (int s = 0; s < kStages - 1; ++s) fetch(s);

    // Q's fragments as f16, each row times a power of two (its largest magnitude to [2^7, 2^8)), in the
    // order of d in which the lane holds its keys; then the factor and frame of this lane's queries
    // 2c and 2c + 1 of each tile
    uint32_t qb[NQ][C::KSTEPS][2];
    float mul[NQ][2];
    int tq[NQ][2];
#pragma unroll
    for (int t = 0; t < NQ; ++t) {
        const int qi = min(8 * t + g, n_q - 1);
        const uint16_t* src = p.q + static_cast<size_t>(load_row(rows(qi), p.nrows, p.status)) * D;
        uint32_t w[C::KL][C::KB / 2];
        uint32_t top = 0;
#pragma unroll
        for (int l = 0; l < C::KL; ++l)
#pragma unroll
            for (int e = 0; e < C::KB / 8; ++e) {
                const uint4 x = *reinterpret_cast<const uint4*>(src + l * 64 + c * C::KB + 8 * e);
                w[l][4 * e] = x.x; w[l][4 * e + 1] = x.y; w[l][4 * e + 2] = x.z; w[l][4 * e + 3] = x.w;
            }
#pragma unroll
        for (int l = 0; l < C::KL; ++l)
#pragma unroll
            for (int e = 0; e < C::KB / 2; ++e) top = __vmaxu2(top, w[l][e] & 0x7fff7fffu);
        top = max(top & 0xffffu, top >> 16);
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
        const int up = top == 0 ? 0 : max(static_cast<int>(top >> 7), 8) - 134;
        const float f = exp2_int(-up), back = p.scale_log2 * exp2_int(up);
#pragma unroll
        for (int l = 0; l < C::KL; ++l)
#pragma unroll
            for (int e = 0; e < C::KB / 2; ++e)  // words 2s and 2s+1 of a chunk are K-step s's rows 2c.. and 2c+8..
                qb[t][l * 4 + e / 2][e & 1] =
                    pack_f16x2(__uint_as_float(w[l][e] << 16) * f, __uint_as_float(w[l][e] & 0xffff0000u) * f);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            mul[t][e] = __shfl_sync(0xffffffffu, back, 4 * (2 * c + e));
            tq[t][e] = start + dF.div(min(8 * t + 2 * c + e, n_q - 1)) + dmax;
        }
    }

    float o[NQ][C::MT][4];  // O^T: columns g VB + 2 mt (0, 1) and + 1 (2, 3), queries 2c and 2c + 1
    float m[NQ][2], mv[NQ][2], l[NQ][2];  // references of p and of the weights, this lane's part of the row sum
#pragma unroll
    for (int t = 0; t < NQ; ++t) {
#pragma unroll
        for (int i = 0; i < C::MT; ++i) o[t][i][0] = o[t][i][1] = o[t][i][2] = o[t][i][3] = 0.f;
        m[t][0] = m[t][1] = mv[t][0] = mv[t][1] = -INFINITY;
        l[t][0] = l[t][1] = 0.f;
    }

    // scale bytes and slots of this lane's keys of a step, g and g + 8
    uint32_t kb[2], vb[2];
    int kslot[2];
    auto fetch_keys = [&](int step) {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const int j = jbeg + (step * kWarps + warp) * kKeys + g + 8 * k;
            const int jc = min(j, jend - 1), slot = dF.div(jc);
            const int at = slot * p.cache.NBk + (jc - slot * nF) / kCacheBlock;
            kb[k] = __ldg(ks + at);
            vb[k] = __ldg(vs + at);
            kslot[k] = j < jend ? slot : -1;  // -1: past the end
        }
    };
    if (steps > 0) fetch_keys(0);
    for (int step = 0; step < steps; ++step) {
        fetch(step + kStages - 1);
        cp_async_wait<kStages - 1>();
        const uint32_t at = my_stage + (step % kStages) * C::STAGE_BYTES;
        float s[NQ][4];  // S^T: key g, queries 2c, 2c + 1; key g + 8, the same
#pragma unroll
        for (int t = 0; t < NQ; ++t) s[t][0] = s[t][1] = s[t][2] = s[t][3] = 0.f;
#pragma unroll
        for (int kl = 0; kl < C::KL; ++kl) {
            uint32_t w0[C::KB / 4], w1[C::KB / 4];
            ld_words<C::KB>(w0, at + kl * 512);
            ld_words<C::KB>(w1, at + (C::KL + kl) * 512);
#pragma unroll
            for (int i = 0; i < C::KB / 4; ++i) {
                const uint32_t a[4] = {
                    e4m3x2_to_f16x2(static_cast<uint16_t>(w0[i])), e4m3x2_to_f16x2(static_cast<uint16_t>(w1[i])),
                    e4m3x2_to_f16x2(static_cast<uint16_t>(w0[i] >> 16)), e4m3x2_to_f16x2(static_cast<uint16_t>(w1[i] >> 16))};
#pragma unroll
                for (int t = 0; t < NQ; ++t) mma16816(s[t], a, qb[t][kl * 4 + i][0], qb[t][kl * 4 + i][1]);
            }
        }
        // scores in log2; ev is added to them for the weights
        float ev[2];
        bool grow = false;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const float kscale = kb[k] == 255u ? __uint_as_float(0x7fc00000u) : exp2_int(static_cast<int>(kb[k]) - 127);
            ev[k] = vb[k] == 255u ? __uint_as_float(0x7fc00000u) : static_cast<float>(static_cast<int>(vb[k]) - 127);
            const int tk = ring.time(kslot[k]);
#pragma unroll
            for (int t = 0; t < NQ; ++t)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float& x = s[t][2 * k + e];
                    const float bias = tab[min(max(tq[t][e] - tk, 0), 2 * dmax)];
                    x = fmaf(x, mul[t][e] * kscale, bias);
                    if (kslot[k] < 0 || bias == -INFINITY) x = -INFINITY;
                    grow = grow || x > m[t][e] + kRescaleLog2 || x + ev[k] > mv[t][e] + kRescaleLog2;
                }
        }
        if (step + 1 < steps) fetch_keys(step + 1);
        if (__any_sync(0xffffffffu, grow)) {  // rare after the first keys: new references
#pragma unroll
            for (int t = 0; t < NQ; ++t)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float top = fmaxf(s[t][e], s[t][2 + e]), topv = fmaxf(s[t][e] + ev[0], s[t][2 + e] + ev[1]);
#pragma unroll
                    for (int d = 4; d < 32; d <<= 1) {
                        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
                        topv = fmaxf(topv, __shfl_xor_sync(0xffffffffu, topv, d));
                    }
                    if (top > m[t][e]) {
                        l[t][e] *= ptx::ex2_approx(m[t][e] - top);  // m = -inf: l is 0
                        m[t][e] = top;
                    }
                    if (topv > mv[t][e]) {
                        const float a = ptx::ex2_approx(mv[t][e] - topv);
#pragma unroll
                        for (int i = 0; i < C::MT; ++i) {
                            o[t][i][e] *= a;
                            o[t][i][2 + e] *= a;
                        }
                        mv[t][e] = topv;
                    }
                }
        }
        uint32_t pb[NQ][2];  // P^T
#pragma unroll
        for (int t = 0; t < NQ; ++t) {
            float w[4];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const float ref = m[t][e] == -INFINITY ? 0.f : m[t][e];
                const float refv = (mv[t][e] == -INFINITY ? 0.f : mv[t][e]) - kPShift;
                l[t][e] += ptx::ex2_approx(s[t][e] - ref) + ptx::ex2_approx(s[t][2 + e] - ref);
                w[e] = ptx::ex2_approx(s[t][e] + ev[0] - refv);
                w[2 + e] = ptx::ex2_approx(s[t][2 + e] + ev[1] - refv);
            }
            pb[t][0] = transpose8x8(pack_f16x2(w[0], w[1]));
            pb[t][1] = transpose8x8(pack_f16x2(w[2], w[3]));
        }
        // four columns of each of the lane's four keys at a time
        uint32_t vw[4][C::VB / 4];
#pragma unroll
        for (int k = 0; k < 4; ++k) ld_words<C::VB>(vw[k], at + (2 * C::KL + k) * 512);
#pragma unroll
        for (int i = 0; i < C::VB / 4; ++i) {
            const uint32_t x0 = __byte_perm(vw[0][i], vw[1][i], 0x5140), x1 = __byte_perm(vw[0][i], vw[1][i], 0x7362);
            const uint32_t y0 = __byte_perm(vw[2][i], vw[3][i], 0x5140), y1 = __byte_perm(vw[2][i], vw[3][i], 0x7362);
            const uint32_t a0[4] = {
                e4m3x2_to_f16x2(static_cast<uint16_t>(x0)), e4m3x2_to_f16x2(static_cast<uint16_t>(x0 >> 16)),
                e4m3x2_to_f16x2(static_cast<uint16_t>(y0)), e4m3x2_to_f16x2(static_cast<uint16_t>(y0 >> 16))};
            const uint32_t a1[4] = {
                e4m3x2_to_f16x2(static_cast<uint16_t>(x1)), e4m3x2_to_f16x2(static_cast<uint16_t>(x1 >> 16)),
                e4m3x2_to_f16x2(static_cast<uint16_t>(y1)), e4m3x2_to_f16x2(static_cast<uint16_t>(y1 >> 16))};
#pragma unroll
            for (int t = 0; t < NQ; ++t) {
                mma16816(o[t][2 * i], a0, pb[t][0], pb[t][1]);
                mma16816(o[t][2 * i + 1], a1, pb[t][0], pb[t][1]);
            }
        }
    }
    cp_async_wait<0>();  // only empty groups are left; nothing outlives the thread
    __syncthreads();     // the stages become the merge buffer

    // warps' results: O as [warp][query][d], then m, mv, l as [warp][query]
    float* mo = reinterpret_cast<float*>(smem);
    float* mm = mo + kWarps * C::ROWS * D;
    float* mmv = mm + kWarps * C::ROWS;
    float* ml = mmv + kWarps * C::ROWS;
#pragma unroll
    for (int t = 0; t < NQ; ++t)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            float sum = l[t][e];
#pragma unroll
            for (int d = 4; d < 32; d <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
            const int row = warp * C::ROWS + 8 * t + 2 * c + e;
            if (g == 0) {
                mm[row] = m[t][e];
                mmv[row] = mv[t][e];
                ml[row] = sum;
            }
#pragma unroll
            for (int i = 0; i < C::MT; i += 2)
                *reinterpret_cast<float4*>(mo + row * D + g * C::VB + 2 * i) =
                    make_float4(o[t][i][e], o[t][i][2 + e], o[t][i + 1][e], o[t][i + 1][2 + e]);
        }
    __syncthreads();
    // each warp joins every fourth query; a lane takes D/32 columns
    constexpr int PER = D / 32;
    for (int row = warp; row < C::ROWS; row += kWarps) {
        if (row >= n_q) break;
        float top = -INFINITY, topv = -INFINITY;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            top = fmaxf(top, mm[w * C::ROWS + row]);
            topv = fmaxf(topv, mmv[w * C::ROWS + row]);
        }
        top = top == -INFINITY ? 0.f : top;  // no key seen, or NaNs alone, which have to stay
        topv = topv == -INFINITY ? 0.f : topv;
        float total = 0.f, acc[PER] = {};
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            total += ml[w * C::ROWS + row] * ptx::ex2_approx(mm[w * C::ROWS + row] - top);
            const float a = ptx::ex2_approx(mmv[w * C::ROWS + row] - topv);
#pragma unroll
            for (int e = 0; e < PER; ++e) acc[e] = fmaf(a, mo[(w * C::ROWS + row) * D + lane * PER + e], acc[e]);
        }
        // a row without a visible key: 0, and -inf for its log-sum-exp
        const float scale = total == 0.f ? 0.f : ptx::ex2_approx(topv - top - kPShift) / total;
        const float l2 = total == 0.f ? -INFINITY : top + ptx::lg2_approx(total);
        const long long grow = rows(row);
        if (!row_ok(grow, p.nrows, p.status)) continue;
        if (p.plan.splits > 1) {
            float* dst = p.part_o + (grow * p.plan.splits + split) * D + lane * PER;
#pragma unroll
            for (int e = 0; e < PER; ++e) dst[e] = acc[e] * scale;
            if (lane == 0) p.part_l[grow * p.plan.splits + split] = l2;
        } else {
            uint16_t* dst = p.out + grow * D + lane * PER;
#pragma unroll
            for (int e = 0; e < PER; ++e) dst[e] = __bfloat16_as_ushort(__float2bfloat16_rn(acc[e] * scale));
            if (lane == 0 && p.lse) p.lse[grow] = l2 * 0.6931471805599453f;
        }
    }
}

// Tiles of 8 queries of a CTA for classes of up to n queries, n <= kMaxRows.
int query_tiles(int n) { return (n + 7) / 8; }

template <int D, int NQ>
int launch_small_d(const FramesFwdParams& p, const Geometry& g, cudaStream_t stream) {
    using C = SmallCfg<D, NQ>;
    static std::atomic<int> attr_done_dev[64];  // as in attn_frames_fwd_sm100.cu
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return static_cast<int>(e);
    if (dev < 0 || dev >= 64 || !attr_done_dev[dev].load(std::memory_order_acquire)) {
        e = cudaFuncSetAttribute(skiparse_cached_small_kernel<D, NQ>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 C::SMEM_BYTES);
        if (e != cudaSuccess) return static_cast<int>(e);
        if (dev >= 0 && dev < 64) attr_done_dev[dev].store(1, std::memory_order_release);
    }
    const dim3 grid(p.plan.splits, g.heads, g.B * g.Ph * g.Pw);
    skiparse_cached_small_kernel<D, NQ><<<grid, 32 * kWarps, C::SMEM_BYTES, stream>>>(p);
    return static_cast<int>(cudaGetLastError());
}

template <int D>
int launch_small(const FramesFwdParams& p, const Geometry& g, cudaStream_t stream) {
    switch (query_tiles(g.T * max_class_tokens(g))) {
        case 1: return launch_small_d<D, 1>(p, g, stream);
        case 2: return launch_small_d<D, 2>(p, g, stream);
        case 3: return launch_small_d<D, 3>(p, g, stream);
        default: return launch_small_d<D, 4>(p, g, stream);
    }
}

}  // namespace

bool cached_small(const Geometry& g) { return static_cast<long long>(g.T) * max_class_tokens(g) <= kMaxRows; }

// One wave of CTAs for up to 24 queries a class, two for more, of at least 512 keys each (measured:
// more CTAs cost up to a quarter in small calls and gain nothing in large ones).
int cached_small_splits(const Geometry& g, int cap) {
    const int tiles = query_tiles(g.T * max_class_tokens(g));
    const long long keys = static_cast<long long>(cap) * max_class_tokens(g);
    const long long ctas = static_cast<long long>(g.heads) * g.B * g.Ph * g.Pw;
    long long s = 148LL * (tiles == 2 || tiles == 3 ? 3 : 4) / ctas;
    if (s > keys / 512) s = keys / 512;
    return static_cast<int>(s < 1 ? 1 : s);
}

int launch_cached_small(const FramesFwdParams& p, const Geometry& g, void* stream) {
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    switch (g.d) {
        case 32: return launch_small<32>(p, g, st);
        case 64: return launch_small<64>(p, g, st);
        case 128: return launch_small<128>(p, g, st);
        default: return static_cast<int>(cudaErrorInvalidValue);
    }
}

}  // namespace skiparse
