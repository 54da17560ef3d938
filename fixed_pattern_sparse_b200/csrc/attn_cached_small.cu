// attn_cached_small.cu -- attention of few queries per class over the e4m3 frame cache (sm_100a).
//
// Frame by frame, a class of a small latent has one or a few dozen queries, and what bounds the
// call is reading the cache: two codes per key and value of d. The tcgen05 kernel would expand
// every key into shared memory for tiles that are mostly empty. Here a warp keeps 16 query rows in
// registers and walks over groups of 16 keys with m16n8k16 products (legacy tensor-core path;
// the codes never leave registers after their copy):
//   * S = Q K^T. The product does not care in which order d is summed, so a lane takes 16
//     consecutive codes of its key as four K-steps, and Q's fragments are loaded in the same order.
//   * O += P V. S's accumulators are P's operand layout. V's operand pairs two keys of one
//     column: two byte permutations and four conversions per four columns of two keys; columns are
//     dealt to the product's n index so that a lane needs one chunk of each of its four keys.
//   * Scales. K's is a factor of the score. V's, 2^e, joins the exponent of the weight:
//     w = 2^(s + e - mv) with a running maximum mv of s + e of its own, beside p = 2^(s - m) for the
//     row sum. So P V needs no common scale, and f16 holds every weight down to 2^-31 of the
//     largest; out = O 2^(mv - m) / l.
//   * Copies go by cp.async into a ring of four stages per warp that only the copying lane
//     reads: no barrier in the loop, 16 KB in flight per warp.
// Key groups are dealt to the warps of a CTA and, over long caches, to `splits` CTAs; warps join
// through shared memory, CTAs through the join kernel of attn_frames_fwd_sm100.cu. Rows beyond 16
// go to further CTAs that re-read the keys, from L2 when they run together.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <atomic>

#include "frames_common.cuh"

namespace skiparse {
namespace {

constexpr int kWarps = 4;
constexpr int kRows = 16;      // query rows of a CTA
constexpr int kKeys = 16;      // keys of a warp step
constexpr int kStages = 4;
constexpr int kMaxRows = 64;   // queries per class up to which this kernel is used
constexpr float kRescaleLog2 = 8.0f;

template <int D>
struct SmallCfg {
    static constexpr int STAGE_BYTES = 2 * kKeys * D;              // of one warp: 16 keys of K and of V
    static constexpr int OFF_TAB = kWarps * kStages * STAGE_BYTES;
    static constexpr int MERGE_BYTES = kWarps * kRows * (D + 3) * 4;  // over the stages, after the loop
    static constexpr int SMEM_BYTES = (OFF_TAB > MERGE_BYTES ? OFF_TAB : MERGE_BYTES) + 4 * (kMaxDistEntries + 1) + 8;
    static constexpr int OFF_TABLE = OFF_TAB > MERGE_BYTES ? OFF_TAB : MERGE_BYTES;
    static constexpr int OFF_RANGE = OFF_TABLE + 4 * (kMaxDistEntries + 1);
    static constexpr int KB = D == 128 ? 16 : D / 4;  // bytes of a lane's copy of a key (D = 128: two of them)
    static constexpr int KL = D == 128 ? 2 : 1;
    static constexpr int VB = D / 8;                  // bytes of a lane's copy of a value
    static constexpr int KSTEPS = D / 16;
    static constexpr int NT = D / 8;                  // n tiles of O
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

template <int D>
__global__ void __launch_bounds__(32 * kWarps, 3) skiparse_cached_small_kernel(const FramesFwdParams p, int row_tiles) {
    using C = SmallCfg<D>;
    const int split = blockIdx.x / row_tiles, tile = blockIdx.x % row_tiles;
    const int head = blockIdx.y;
    const int seq = blockIdx.z;
    const int q2 = p.g.Ph * p.g.Pw;
    const int b = seq / q2, c2 = seq % q2, ci = c2 / p.g.Pw, cj = c2 % p.g.Pw;
    const int Rc = p.g.Rc[ci], Sc = p.g.Sc[cj], nF = Rc * Sc;
    const int n_q = p.g.T * nF;
    const int q_first = tile * kRows;
    if (q_first >= n_q) return;
    const int start = p.cache.start[b];
    if (start < 0 || start > kMaxStart) return;
    FrameRing ring;
    ring.init(start + p.g.T, p.cache.cap);
    FastDiv dF;
    dF.init(nF);
    RowMap rows;
    rows.init(p.g.T, p.g.H, p.g.W, p.g.heads, p.g.Ph, p.g.Pw, p.g.mode, ci, cj, Rc, Sc, b, head);

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
    ring.visible(start + dF.div(q_first), start + dF.div(min(q_first + kRows, n_q) - 1), range[0], range[1], dmax, f_lo, f_hi);
    const int groups = f_hi >= f_lo ? ((f_hi - f_lo + 1) * nF + kKeys - 1) / kKeys : 0;
    const int per_split = (groups + p.splits - 1) / p.splits;
    const int jend = (f_hi + 1) * nF;
    const int jbeg = f_lo * nF + split * per_split * kKeys;
    const int mygroups = max(0, min(per_split, groups - split * per_split));
    const int steps = (mygroups - warp + kWarps - 1) / kWarps;  // groups warp, warp + kWarps, ...

    const long long sh = static_cast<long long>(seq) * p.g.heads + head;
    const long long crows = static_cast<long long>(p.cache.cap) * p.cache.F;
    const uint8_t* kc = p.cache.k + sh * crows * D;
    const uint8_t* vc = p.cache.v + sh * crows * D;
    const uint8_t* ks = p.cache.ks + sh * p.cache.cap * p.cache.NBk;
    const uint8_t* vs = p.cache.vs + sh * p.cache.cap * p.cache.NBk;
    const uint32_t my_stage = sbase + warp * kStages * C::STAGE_BYTES;

    // the key of index j of this CTA's range, its row in the cache and its scales' place
    auto key_row = [&](int j, int& slot) -> long long {
        j = min(j, jend - 1);
        slot = dF.div(j);
        return load_row(static_cast<long long>(slot) * p.cache.F + (j - slot * nF), crows, p.status);
    };
    auto fetch = [&](int step) {
        if (step < steps) {
            const int j0 = jbeg + (step * kWarps + warp) * kKeys;
            const uint32_t at = my_stage + (step % kStages) * C::STAGE_BYTES;
            int slot;
#pragma unroll
            for (int n = 0; n < 2; ++n) {
                const uint8_t* src = kc + key_row(j0 + 8 * n + g, slot) * D;
#pragma unroll
                for (int l = 0; l < C::KL; ++l)
                    cp_async_n<C::KB>(at + ((n * C::KL + l) * 32 + lane) * C::KB, src + l * 64 + c * C::KB);
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const uint8_t* src = vc + key_row(j0 + 2 * c + (k & 1) + 8 * (k >> 1), slot) * D;
                cp_async_n<C::VB>(at + kKeys * D + (k * 32 + lane) * C::VB, src + g * C::VB);
            }
        }
        cp_async_commit();
    };
#pragma unroll
    for (int s = 0; s < kStages - 1; ++s) fetch(s);

    // Q's fragments as f16, each row times a power of two (its largest magnitude to [2^7, 2^8)); rows
    // g and g + 8 of the tile, in the order of d in which the lane holds its keys
    uint32_t qa[C::KSTEPS][4];
    float mul[2];
    int tq[2];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        const int qi = min(q_first + g + 8 * r, n_q - 1);
        tq[r] = start + dF.div(qi);
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
        const float f = exp2_int(-up);
        mul[r] = p.scale_log2 * exp2_int(up);
#pragma unroll
        for (int l = 0; l < C::KL; ++l)
#pragma unroll
            for (int e = 0; e < C::KB / 2; ++e)
                // words 2t and 2t+1 of a chunk are K-step t's columns 2c.. and 2c+8..
                qa[l * 4 + e / 2][r + 2 * (e & 1)] =
                    pack_f16x2(__uint_as_float(w[l][e] << 16) * f, __uint_as_float(w[l][e] & 0xffff0000u) * f);
    }

    float o[C::NT][4];
#pragma unroll
    for (int n = 0; n < C::NT; ++n) o[n][0] = o[n][1] = o[n][2] = o[n][3] = 0.f;
    // per row g + 8 r: references of p and of the weights, and this lane's part of the row sum
    float m[2] = {-INFINITY, -INFINITY}, mv[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};

    // scale bytes and frames of this lane's four keys of a step (columns 2c, 2c+1 of both halves)
    uint32_t kb[4], vb[4];
    int kf[4];
    auto fetch_keys = [&](int step) {
        const int j0 = jbeg + (step * kWarps + warp) * kKeys;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int j = j0 + 2 * c + (k & 1) + 8 * (k >> 1);
            const int jc = min(j, jend - 1), slot = dF.div(jc);
            const long long at = static_cast<long long>(slot) * p.cache.NBk + (jc - slot * nF) / kCacheBlock;
            kb[k] = __ldg(ks + at);
            vb[k] = __ldg(vs + at);
            kf[k] = j < jend ? slot : -1;  // -1: past the end
        }
    };
    if (steps > 0) fetch_keys(0);
    for (int step = 0; step < steps; ++step) {
        fetch(step + kStages - 1);
        cp_async_wait<kStages - 1>();
        const uint32_t at = my_stage + (step % kStages) * C::STAGE_BYTES;
        float s[2][4];
#pragma unroll
        for (int n = 0; n < 2; ++n) {
            s[n][0] = s[n][1] = s[n][2] = s[n][3] = 0.f;
#pragma unroll
            for (int kl = 0; kl < C::KL; ++kl) {
                uint32_t w[C::KB / 4];
                ld_words<C::KB>(w, at + ((n * C::KL + kl) * 32 + lane) * C::KB);
#pragma unroll
                for (int t = 0; t < C::KB / 4; ++t)
                    mma16816(s[n], qa[kl * 4 + t], e4m3x2_to_f16x2(static_cast<uint16_t>(w[t])),
                             e4m3x2_to_f16x2(static_cast<uint16_t>(w[t] >> 16)));
            }
        }
        // scores in log2, and with V's exponent: index [n][2 r + e] is row g + 8 r, key 2c + e + 8 n
        float xv[2][4];
        float top[2] = {-INFINITY, -INFINITY}, topv[2] = {-INFINITY, -INFINITY};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const float kf32 = kb[k] == 255u ? __uint_as_float(0x7fc00000u) : exp2_int(static_cast<int>(kb[k]) - 127);
            const float ev = vb[k] == 255u ? __uint_as_float(0x7fc00000u) : static_cast<float>(static_cast<int>(vb[k]) - 127);
            const int t = ring.time(kf[k]);
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                float& x = s[k >> 1][2 * r + (k & 1)];
                const float bias = tab[clamp_dist(tq[r] - t, dmax) + dmax];
                x = fmaf(x, mul[r] * kf32, bias);
                if (kf[k] < 0 || bias == -INFINITY) x = -INFINITY;
                xv[k >> 1][2 * r + (k & 1)] = x + ev;
                top[r] = fmaxf(top[r], x);
                topv[r] = fmaxf(topv[r], x + ev);
            }
        }
        if (step + 1 < steps) fetch_keys(step + 1);
        bool grow = false;
#pragma unroll
        for (int r = 0; r < 2; ++r) grow = grow || top[r] > m[r] + kRescaleLog2 || topv[r] > mv[r] + kRescaleLog2;
        if (__any_sync(0xffffffffu, grow)) {  // rare after the first keys: new references for the rows
#pragma unroll
            for (int r = 0; r < 2; ++r) {
#pragma unroll
                for (int d = 1; d < 4; d <<= 1) {
                    top[r] = fmaxf(top[r], __shfl_xor_sync(0xffffffffu, top[r], d));
                    topv[r] = fmaxf(topv[r], __shfl_xor_sync(0xffffffffu, topv[r], d));
                }
                if (top[r] > m[r]) {
                    l[r] *= ptx::ex2_approx(m[r] - top[r]);  // m = -inf: l is 0
                    m[r] = top[r];
                }
                if (topv[r] > mv[r]) {
                    const float a = ptx::ex2_approx(mv[r] - topv[r]);
#pragma unroll
                    for (int n = 0; n < C::NT; ++n) {
                        o[n][2 * r] *= a;
                        o[n][2 * r + 1] *= a;
                    }
                    mv[r] = topv[r];
                }
            }
        }
        uint32_t pa[4];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const float ref = m[r] == -INFINITY ? 0.f : m[r], refv = (mv[r] == -INFINITY ? 0.f : mv[r]) - kPShift;
#pragma unroll
            for (int n = 0; n < 2; ++n) {
                l[r] += ptx::ex2_approx(s[n][2 * r] - ref) + ptx::ex2_approx(s[n][2 * r + 1] - ref);
                pa[r + 2 * n] = pack_f16x2(ptx::ex2_approx(xv[n][2 * r] - refv), ptx::ex2_approx(xv[n][2 * r + 1] - refv));
            }
        }
        // four columns of each of the lane's four keys at a time
        uint32_t vw[4][C::VB / 4];
#pragma unroll
        for (int k = 0; k < 4; ++k) ld_words<C::VB>(vw[k], at + kKeys * D + (k * 32 + lane) * C::VB);
#pragma unroll
        for (int q = 0; q < C::VB / 4; ++q) {
            const uint32_t a0 = __byte_perm(vw[0][q], vw[1][q], 0x5140), a1 = __byte_perm(vw[0][q], vw[1][q], 0x7362);
            const uint32_t b0 = __byte_perm(vw[2][q], vw[3][q], 0x5140), b1 = __byte_perm(vw[2][q], vw[3][q], 0x7362);
            mma16816(o[4 * q], pa, e4m3x2_to_f16x2(static_cast<uint16_t>(a0)), e4m3x2_to_f16x2(static_cast<uint16_t>(b0)));
            mma16816(o[4 * q + 1], pa, e4m3x2_to_f16x2(static_cast<uint16_t>(a0 >> 16)),
                     e4m3x2_to_f16x2(static_cast<uint16_t>(b0 >> 16)));
            mma16816(o[4 * q + 2], pa, e4m3x2_to_f16x2(static_cast<uint16_t>(a1)), e4m3x2_to_f16x2(static_cast<uint16_t>(b1)));
            mma16816(o[4 * q + 3], pa, e4m3x2_to_f16x2(static_cast<uint16_t>(a1 >> 16)),
                     e4m3x2_to_f16x2(static_cast<uint16_t>(b1 >> 16)));
        }
    }
    cp_async_wait<0>();  // only empty groups are left; nothing outlives the thread
    __syncthreads();     // the stages become the merge buffer

    // warps' results: O as [warp][row][d], then m, mv, l as [warp][row]
    float* mo = reinterpret_cast<float*>(smem);
    float* mm = mo + kWarps * kRows * D;
    float* mmv = mm + kWarps * kRows;
    float* ml = mmv + kWarps * kRows;
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
        l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
        const int row = warp * kRows + g + 8 * r;
        if (c == 0) {
            mm[row] = m[r];
            mmv[row] = mv[r];
            ml[row] = l[r];
        }
        // column 2c + e of n tile n is value column (2c + e) * NT + n
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
            for (int n = 0; n < C::NT; n += 4)
                *reinterpret_cast<float4*>(mo + row * D + (2 * c + e) * C::NT + n) =
                    make_float4(o[n][2 * r + e], o[n + 1][2 * r + e], o[n + 2][2 * r + e], o[n + 3][2 * r + e]);
    }
    __syncthreads();
    // each warp joins four rows; a lane takes D/32 columns
    constexpr int PER = D / 32;
    for (int row = warp; row < kRows; row += kWarps) {
        const int qi = q_first + row;
        if (qi >= n_q) break;
        float top = -INFINITY, topv = -INFINITY;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            top = fmaxf(top, mm[w * kRows + row]);
            topv = fmaxf(topv, mmv[w * kRows + row]);
        }
        top = top == -INFINITY ? 0.f : top;  // no key seen, or NaNs alone, which have to stay
        topv = topv == -INFINITY ? 0.f : topv;
        float total = 0.f, acc[PER] = {};
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            total += ml[w * kRows + row] * ptx::ex2_approx(mm[w * kRows + row] - top);
            const float a = ptx::ex2_approx(mmv[w * kRows + row] - topv);
#pragma unroll
            for (int e = 0; e < PER; ++e) acc[e] = fmaf(a, mo[(w * kRows + row) * D + lane * PER + e], acc[e]);
        }
        // a row without a visible key: 0, and -inf for its log-sum-exp
        const float scale = total == 0.f ? 0.f : ptx::ex2_approx(topv - top - kPShift) / total;
        const float l2 = total == 0.f ? -INFINITY : top + ptx::lg2_approx(total);
        const long long grow = rows(qi);
        if (!row_ok(grow, p.nrows, p.status)) continue;
        if (p.splits > 1) {
            float* dst = p.part_o + (grow * p.splits + split) * D + lane * PER;
#pragma unroll
            for (int e = 0; e < PER; ++e) dst[e] = acc[e] * scale;
            if (lane == 0) p.part_l[grow * p.splits + split] = l2;
        } else {
            uint16_t* dst = p.out + grow * D + lane * PER;
#pragma unroll
            for (int e = 0; e < PER; ++e) dst[e] = __bfloat16_as_ushort(__float2bfloat16_rn(acc[e] * scale));
            if (lane == 0 && p.lse) p.lse[grow] = l2 * 0.6931471805599453f;
        }
    }
}

template <int D>
int launch_small_d(const FramesFwdParams& p, const Geometry& g, cudaStream_t stream) {
    using C = SmallCfg<D>;
    static std::atomic<int> attr_done_dev[64];  // as in attn_frames_fwd_sm100.cu
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return static_cast<int>(e);
    if (dev < 0 || dev >= 64 || !attr_done_dev[dev].load(std::memory_order_acquire)) {
        e = cudaFuncSetAttribute(skiparse_cached_small_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM_BYTES);
        if (e != cudaSuccess) return static_cast<int>(e);
        if (dev >= 0 && dev < 64) attr_done_dev[dev].store(1, std::memory_order_release);
    }
    const int row_tiles = (g.T * max_class_tokens(g) + kRows - 1) / kRows;
    const dim3 grid(static_cast<unsigned>(row_tiles) * p.splits, g.heads, g.B * g.Ph * g.Pw);
    skiparse_cached_small_kernel<D><<<grid, 32 * kWarps, C::SMEM_BYTES, stream>>>(p, row_tiles);
    return static_cast<int>(cudaGetLastError());
}

}  // namespace

bool cached_small(const Geometry& g) { return static_cast<long long>(g.T) * max_class_tokens(g) <= kMaxRows; }

// At least 512 keys a CTA, and no more CTAs than some four waves of three per SM.
int cached_small_splits(const Geometry& g, int cap) {
    const long long keys = static_cast<long long>(cap) * max_class_tokens(g);
    const long long ctas = (static_cast<long long>(g.T) * max_class_tokens(g) + kRows - 1) / kRows * g.heads * g.B * g.Ph * g.Pw;
    long long s = 4LL * 3 * 148 / ctas;
    if (s > keys / 512) s = keys / 512;
    return static_cast<int>(s < 1 ? 1 : s);
}

int launch_cached_small(const FramesFwdParams& p, const Geometry& g, void* stream) {
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    switch (g.d) {
        case 32: return launch_small_d<32>(p, g, st);
        case 64: return launch_small_d<64>(p, g, st);
        case 128: return launch_small_d<128>(p, g, st);
        default: return static_cast<int>(cudaErrorInvalidValue);
    }
}

}  // namespace skiparse
