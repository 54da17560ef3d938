// attn_frames_bwd_sm100.cu -- backward pass of the class attention with a learned bias by frame
// distance (sm_100a).
//
// For one (b, class, head) subsequence, with P = exp(s - L) recomputed from the biased, masked
// scores s = q.k/sqrt(d) + bias[t_q - t_k] and the forward's log-sum-exp L, and D_i = dO_i . O_i:
//   dV = P^T dO,  dP = dO V^T,  dS = P o (dP - D),  dQ = dS K / sqrt(d),  dK = dS^T Q / sqrt(d),
//   dtable[g][head] = sum of dS_ij over all pairs (i, j) whose distance lies in bucket g.
// The schedule is that of the unbiased backward pass (attn_bwd_sm100.cu): a key-major kernel for dK
// and dV and a query-major one for dQ, seven tile products per pair of tiles, no atomics on
// results. What the bias adds:
//   * Frames. Within 32 columns of one frame the bias is one number per row: in the query-major
//     kernel it joins the row's log-sum-exp in the existing FMA (no instruction per score), in
//     the key-major one it is added to each column's. A chunk that holds a frame's border
//     chooses between two; frames of fewer than 32 tokens look the bias up where it changes.
//     Streamed tiles that no stationary row can see are skipped.
//   * D. Every row of dS sums to zero over its keys, so an error of D_i enters the bias gradient
//     through all of the row's keys with one sign, and D from the forward's output, which carries
//     the roundings of P and of the output itself, would dominate that gradient's error. The
//     query-major kernel therefore runs first, with that D, and sums its rows of dS: what is left
//     is D's error, and the key-major kernel gets D without it. (dQ keeps D's error, the smaller
//     for a stored rounding residual of the output, out_lo.)
//   * Bias gradient. The key-major kernel sums dS, in fp32, before its rounding to bf16, in a
//     register per key row for as long as the streamed queries stay in one frame; when the
//     frame changes, the warp adds its rows of equal distance by shuffles and one lane adds the
//     sum to the warp's own table of distances in shared memory. A CTA writes the sum of its
//     eight tables, in a fixed order, to the workspace, and the last kernel adds those rows and
//     joins distances to buckets, in a fixed order too: the result does not depend on timing.
//     Per score this costs one addition (half of one packed instruction).
// Launches: dQ, which first takes D and L from its rows of out, dO and lse; dK/dV; dtable. (Row statistics
// by a kernel of their own took the same at 480p and 7 us longer, of 183 and of 94, in small steps.)
// What bounds it, 480p (21 frames of 390 tokens a class, d = 128, 12 heads): dQ 2.2 ms, dK and dV 3.3 ms at
// 1965 MHz, 1.1 and 1.0 PFLOP/s; 2.4 and 3.6 in training steps back to back, under the power cap. As in the unbiased backward pass, a key step waits on its chain of products and
// exponentials (2500 and 3600 clocks at d = 64, where the tensor core needs 770 and 1020 of them); the
// frames add 7 % more streamed rows to dK and dV, and the sums of dS.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <atomic>

#include "frames_common.cuh"

namespace skiparse {
namespace {

// 13 warps: softmax 0-7, producers 8-11 (warps 8-9 copy the first streamed tensor and the
// statistics, warps 10-11 the second, each pair splitting a tile's rows), MMA issuer 12.
constexpr int kBwdThreads = 416;
constexpr int kBwdProd0 = 8;
constexpr int kBwdProducers = 128;
constexpr int kBwdMma = 12;
constexpr int kBwdSoftmax = 256;
constexpr int kMaxSmem = 232448;  // 227 KB, the most a CTA may have

template <int D, bool KV>
struct BwdCfg : TileGeom<D> {
    using G = TileGeom<D>;
    using G::TILE_BYTES;
    // ring slots of the two streamed tensors: B1 = Q (key-major) or K (query-major), B2 = dO or V
    static constexpr int NS1 = KV ? 2 : 3, NS2 = 2;
    static constexpr int OFF_A1 = 0;
    static constexpr int OFF_A2 = TILE_BYTES;
    static constexpr int OFF_B1 = 2 * TILE_BYTES;
    static constexpr int OFF_B2 = OFF_B1 + NS1 * TILE_BYTES;
    static constexpr int OFF_VEC = OFF_B2 + NS2 * TILE_BYTES;  // [B1 slot or stationary][L,D][128] fp32
    static constexpr int VEC_BYTES = (KV ? NS1 : 1) * 2 * kTileRows * 4;
    static constexpr int OFF_HIST = OFF_VEC + VEC_BYTES;       // key-major: 8 warps x distances
    static constexpr int OFF_TAB = OFF_HIST + (KV ? 8 * (kMaxDistEntries + 1) * 4 : 0);  // the bias by distance, bf16
    static constexpr int OFF_BAR = OFF_TAB + 2 * (kMaxDistEntries + 1);
    static constexpr int B_STAT = 0, B_FULL1 = 1, B_EMPTY1 = B_FULL1 + NS1, B_FULL2 = B_EMPTY1 + NS1,
                         B_EMPTY2 = B_FULL2 + NS2, B_X1 = B_EMPTY2 + NS2, B_X2 = B_X1 + 1, B_X1FREE = B_X2 + 1,
                         B_P = B_X1FREE + 1, B_DS = B_P + 1, B_ACC = B_DS + 1,
                         B_DRAIN = B_ACC + 1, NBARS = B_DRAIN + 1;
    static constexpr int OFF_TMEM_SLOT = OFF_BAR + 8 * NBARS;
    static constexpr int OFF_ABORT = OFF_TMEM_SLOT + 4;
    static constexpr int OFF_RANGE = OFF_ABORT + 4;            // first and last visible distance
    static constexpr int SMEM_USED = OFF_RANGE + 8;
    // + slack for 1024-byte alignment where it fits (the kernel checks the slack it got); at least
    // 116 KB so that one CTA (and its 512 TMEM columns) owns an SM even for small d
    static constexpr int SMEM_BYTES =
        SMEM_USED + 1024 > kMaxSmem ? kMaxSmem : (SMEM_USED + 1024 > 118784 ? SMEM_USED + 1024 : 118784);
    static_assert(SMEM_USED + 256 <= kMaxSmem, "shared memory overflow");
    // TMEM: X1 = S (or S^T), X2 = dP (or dP^T); P^T (key-major) and dS (both kernels) are written
    // in bf16 over the first half of each warpgroup's 64 columns of X1 and X2
    static constexpr uint32_t COL_X1 = 0, COL_X2 = 128, COL_ACC1 = 256, COL_ACC2 = 256 + D, NCOLS = 512;
    static_assert(COL_ACC2 + D <= NCOLS, "TMEM overflow");
};

// TMEM column of K-step kk (16 streamed rows) of a bf16 operand written by the two softmax
// warpgroups over their own halves of a 128-column score region: rows 0..63 -> columns 0..31,
// rows 64..127 -> columns 64..95.
__device__ __forceinline__ uint32_t half_packed_col(int kk) { return kk < 4 ? 8 * kk : 64 + 8 * (kk - 4); }

// 4-byte cp.async of one fp32 per tile row (L or D of the row's token and head); tr holds the
// token rows of this lane's two tile rows 64*pw + lane and 64*pw + 32 + lane.
__device__ __forceinline__ void load_vec(uint32_t dst, const float* __restrict__ src, const TileRows& tr,
                                         int pw, int lane) {
#pragma unroll
    for (int half = 0; half < 2; ++half) {
        const int r = 64 * pw + 32 * half + lane;
        asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst + 4u * r),
                     "l"(src + (half ? tr.rb : tr.ra))
                     : "memory");
    }
}

// dS of two columns, p (dP - D), two per instruction (packed f32x2); dP - D exactly, as an FMA with -1.
__device__ __forceinline__ float2 ds_pair(float2 p, float2 d, uint32_t dp0, uint32_t dp1) {
    return __fmul2_rn(p, __ffma2_rn(d, make_float2(-1.f, -1.f), make_float2(__uint_as_float(dp0), __uint_as_float(dp1))));
}

// sum_e dO[e] * (O[e] + O_lo[e]) over a row that `lanes` neighbouring lanes hold, eight elements each, this
// lane's from element `at` of the tensors.
__device__ __forceinline__ float dot_of_row(const uint16_t* out, const uint16_t* out_lo, const uint16_t* dout, long long at,
                                            int lanes) {
    const uint4 a = __ldg(reinterpret_cast<const uint4*>(out + at));
    const uint4 g = __ldg(reinterpret_cast<const uint4*>(dout + at));
    uint4 lo = make_uint4(0u, 0u, 0u, 0u);
    if (out_lo) lo = __ldg(reinterpret_cast<const uint4*>(out_lo + at));
    const uint32_t av[4] = {a.x, a.y, a.z, a.w}, gv[4] = {g.x, g.y, g.z, g.w}, lv[4] = {lo.x, lo.y, lo.z, lo.w};
    float acc = 0.f;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        acc = fmaf(__uint_as_float(av[e] << 16) + __uint_as_float(lv[e] << 16), __uint_as_float(gv[e] << 16), acc);
        acc = fmaf(__uint_as_float(av[e] & 0xffff0000u) + __uint_as_float(lv[e] & 0xffff0000u),
                   __uint_as_float(gv[e] & 0xffff0000u), acc);
    }
    for (int off = lanes / 2; off > 0; off >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, off);
    return acc;
}

template <int D, bool KV, bool AL>
__global__ void __launch_bounds__(kBwdThreads, 1) skiparse_frames_bwd_kernel(const FramesBwdParams p) {
    using C = BwdCfg<D, KV>;
    // the tiles that see most come first under a causal map: early keys, late queries
    int tile, head, seq;
    p.order.get(blockIdx.x, p.g.heads, tile, seq, head);
    if (!KV) tile = p.tiles - 1 - tile;
    ClassView cls;
    cls.init(p.g, seq);
    const int nF = cls.nF;
    const FastDiv dF = cls.dF;
    const int n_c = p.g.T * nF;
    const int first = tile * kTileRows;
    if (first >= n_c) return;  // uniform over the CTA, before any shared state
    const RowMap rows = cls.rows(p.g, head);

    extern __shared__ __align__(1024) uint8_t smem_raw[];
    const uint32_t raw_base = ptx::smem_u32(smem_raw);
    const uint32_t pad = (1024u - (raw_base & 1023u)) & 1023u;
    if (pad + C::SMEM_USED > static_cast<uint32_t>(C::SMEM_BYTES)) {
        // not aligned well enough for this layout (uniform over the CTA, before any shared state): report
        // it instead of running out of bounds
        if (threadIdx.x == 0) atomicExch(p.status, kErrLaunch);
        return;
    }
    uint8_t* smem = smem_raw + pad;
    const uint32_t sbase = raw_base + pad;
    auto bar = [&](int i) -> uint32_t { return sbase + C::OFF_BAR + 8u * i; };
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::OFF_TMEM_SLOT);
    volatile int* abort = reinterpret_cast<volatile int*>(smem + C::OFF_ABORT);
    int* range = reinterpret_cast<int*>(smem + C::OFF_RANGE);
    const float* vecs = reinterpret_cast<const float*>(smem + C::OFF_VEC);
    float* hist = reinterpret_cast<float*>(smem + C::OFF_HIST);

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const uint64_t lim = p.wait_limit_ns;
    const int dmax = p.bias.D;
    uint16_t* tab = reinterpret_cast<uint16_t*>(smem + C::OFF_TAB) + dmax;  // bias by distance, bf16 as in the table

    if (threadIdx.x == 0) {
        ptx::mbar_init(bar(C::B_STAT), kBwdProducers);
        for (int s = 0; s < C::NS1; ++s) {
            ptx::mbar_init(bar(C::B_FULL1 + s), kBwdProducers / 2);  // one producer pair per tensor
            ptx::mbar_init(bar(C::B_EMPTY1 + s), 1);
        }
        for (int s = 0; s < C::NS2; ++s) {
            ptx::mbar_init(bar(C::B_FULL2 + s), kBwdProducers / 2);
            ptx::mbar_init(bar(C::B_EMPTY2 + s), 1);
        }
        ptx::mbar_init(bar(C::B_X1), 1);
        ptx::mbar_init(bar(C::B_X2), 1);
        ptx::mbar_init(bar(C::B_X1FREE), kBwdSoftmax);
        ptx::mbar_init(bar(C::B_P), kBwdSoftmax);
        ptx::mbar_init(bar(C::B_DS), kBwdSoftmax);
        ptx::mbar_init(bar(C::B_ACC), 1);
        ptx::mbar_init(bar(C::B_DRAIN), 1);
        *abort = 0;
        range[0] = dmax + 1;
        range[1] = -dmax - 1;
        ptx::fence_mbar_init();
    }
    if (warp == kBwdMma) {
        ptx::tmem_alloc(ptx::smem_u32(tmem_slot), C::NCOLS);
        ptx::tmem_relinquish();
    }
    // stationary tiles: (K, V) for the key-major kernel, (Q, dO) for the query-major one. They start
    // to travel before the barriers stand; the copies arrive on theirs below.
    const uint16_t* g_a1 = KV ? p.k : p.q;
    const uint16_t* g_a2 = KV ? p.v : p.dout;
    const uint16_t* g_b1 = KV ? p.q : p.k;
    const uint16_t* g_b2 = KV ? p.dout : p.v;
    if (warp >= kBwdProd0 && warp < kBwdProd0 + 4) {
        const int pair = (warp - kBwdProd0) >> 1, pw = (warp - kBwdProd0) & 1;
        const TileRows ta = tile_rows(rows, first, n_c, pw, lane, p.nrows, p.status);
        load_tile_rows<D>(sbase + (pair ? C::OFF_A2 : C::OFF_A1), pair ? g_a2 : g_a1, ta, pw, lane);
    }
    if (KV)
        for (int i = threadIdx.x; i < 8 * p.ND; i += kBwdThreads) hist[i] = 0.f;
    int dlo = dmax + 1, dhi = -dmax - 1;  // first and last visible distance
    for (int u = static_cast<int>(threadIdx.x) - dmax; u <= dmax; u += kBwdThreads) {
        const uint16_t b = bias_bf16(p.bias, p.g.heads, u + dmax, head);
        tab[u] = b;
        if (b != kBiasNone) {
            dlo = min(dlo, u);
            dhi = max(dhi, u);
        }
    }
    dlo = __reduce_min_sync(0xffffffffu, dlo);
    dhi = __reduce_max_sync(0xffffffffu, dhi);
    ptx::tc_fence_before();
    __syncthreads();
    if (lane == 0 && dlo <= dhi) {
        atomicMin(&range[0], dlo);
        atomicMax(&range[1], dhi);
    }
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    dlo = range[0];
    dhi = range[1];
    // streamed frames that some stationary row sees (the end distances stand for all beyond them)
    int f_lo = 0, f_hi = p.g.T - 1;
    {
        const int ta = dF.div(first), tb = dF.div(min(first + kTileRows, n_c) - 1);
        if (KV) {  // query frame - key frame in [dlo, dhi]
            if (dlo > -dmax) f_lo = max(f_lo, ta + dlo);
            if (dhi < dmax) f_hi = min(f_hi, tb + dhi);
        } else {
            if (dhi < dmax) f_lo = max(f_lo, ta - dhi);
            if (dlo > -dmax) f_hi = min(f_hi, tb - dlo);
        }
        if (dlo > dhi) f_hi = f_lo - 1;
    }
    const int jbeg = f_lo * nF, jend = (f_hi + 1) * nF;
    const int cpf = (nF + 31) / 32, chunks = (f_hi - f_lo + 1) * cpf;  // aligned: of a frame, of the stream
    const FastDiv dC = p.g.dC[cls.c];
    const int nstream = f_hi < f_lo ? 0 : AL ? (chunks + 3) / 4 : (jend - jbeg + kTileRows - 1) / kTileRows;
    // aligned: the class's index of row i of chunk q of the stream (rows past a frame's end, or of
    // chunks past the last, repeat a real one)
    auto chunk_row = [&](int q, int i) {
        q = min(q, chunks - 1);
        const int f = dC.div(q);
        return (f_lo + f) * nF + min((q - f * cpf) * 32 + i, nF - 1);
    };

    if (warp >= kBwdProd0 && warp < kBwdProd0 + 4) {
        // ------------------------------------------------------------------ producers
        // Pair 0 (warps 8-9) copies the first streamed tensor (and the L/D statistics), pair 1
        // (warps 10-11) the second; within a pair, warp pw copies rows [64pw, 64pw+64).
        const int pair = (warp - kBwdProd0) >> 1;
        const int pw = (warp - kBwdProd0) & 1;
        const int ns = pair ? C::NS2 : C::NS1;
        cp_async_arrive_noinc(bar(C::B_STAT));
        bool ok = true;
        for (int j = 0; j < nstream; ++j) {
            const int s = j % ns;
            if (j >= ns) {
                int w_ok = 1;
                if (lane == 0)
                    w_ok = ptx::mbar_wait(bar((pair ? C::B_EMPTY2 : C::B_EMPTY1) + s), ((j / ns) - 1) & 1, abort, lim);
                w_ok = __shfl_sync(0xffffffffu, w_ok, 0);
                if (!w_ok) {
                    ok = false;
                    break;
                }
            }
            const TileRows tr =
                AL ? TileRows{static_cast<int>(load_row(rows(chunk_row(4 * j + 2 * pw, lane)), p.nrows, p.status)),
                              static_cast<int>(load_row(rows(chunk_row(4 * j + 2 * pw + 1, lane)), p.nrows, p.status))}
                   : tile_rows(rows, jbeg + j * kTileRows, jend, pw, lane, p.nrows, p.status);
            load_tile_rows<D>(sbase + (pair ? C::OFF_B2 : C::OFF_B1) + s * C::TILE_BYTES, pair ? g_b2 : g_b1, tr,
                              pw, lane);
            if (KV && pair == 0) {  // the streamed queries' L and D
                const uint32_t v = sbase + C::OFF_VEC + s * 2 * 4 * kTileRows;
                load_vec(v, p.nlse2, tr, pw, lane);
                load_vec(v + 4 * kTileRows, p.delta, tr, pw, lane);
            }
            // completes when this tile has landed; test hook: one thread of the key-major kernel
            // never signals the first streamed tile
            if (!(KV && p.fault == 1 && j == 0 && pair == 0 && pw == 0 && lane == 0))
                cp_async_arrive_noinc(bar((pair ? C::B_FULL2 : C::B_FULL1) + s));
        }
        cp_async_commit();
        cp_async_wait<0>();  // no copy of this thread outlives it
        if (!ok) record_abort(abort, p.status);
    } else if (warp == kBwdMma) {
        // ------------------------------------------------------------------ MMA issuer
        if (lane == 0 && nstream > 0) {
            const uint32_t idesc_x = ptx::idesc_bf16_f32(kTileRows, kTileRows, false);
            const uint32_t idesc_acc = ptx::idesc_bf16_f32(kTileRows, D, true);
            const uint64_t a1 = ptx::smem_desc(sbase + C::OFF_A1, 16, 8 * C::SW, C::LAYOUT);
            const uint64_t a2 = ptx::smem_desc(sbase + C::OFF_A2, 16, 8 * C::SW, C::LAYOUT);
            // streamed tiles read K-major (as the B of S, dP) or MN-major (as the B of dV, dK, dQ)
            auto bk = [&](int off) { return ptx::smem_desc(sbase + off, 16, 8 * C::SW, C::LAYOUT); };
            auto bm = [&](int off) { return ptx::smem_desc(sbase + off, C::BOX_BYTES, 8 * C::SW, C::LAYOUT); };
            auto x_mma = [&](uint64_t a, uint64_t b, uint32_t d_tmem) {   // D = A B^T over d
#pragma unroll
                for (int kk = 0; kk < C::KSTEPS; ++kk) {
                    const uint32_t off = C::kstep_off(kk) >> 4;
                    ptx::mma_ss(d_tmem, a + off, b + off, idesc_x, kk > 0 ? 1u : 0u);
                }
            };
            // D += A B over the 128 streamed rows, A from TMEM (P^T, dS^T or dS, half-packed columns)
            auto acc_mma = [&](uint32_t a_col, uint64_t b, uint32_t d_tmem, bool acc) {
#pragma unroll
                for (int kk = 0; kk < kTileRows / 16; ++kk)
                    ptx::mma_ts(d_tmem, tmem + a_col + half_packed_col(kk), b + ((kk * 16 * C::SW) >> 4),
                                idesc_acc, (acc || kk > 0) ? 1u : 0u);
            };
            auto b1_off = [&](int j) { return C::OFF_B1 + (j % C::NS1) * C::TILE_BYTES; };
            auto b2_off = [&](int j) { return C::OFF_B2 + (j % C::NS2) * C::TILE_BYTES; };
            // S (or S^T) of streamed tile j into X1; dP (or dP^T) into X2
            auto issue_x1 = [&](int j) {
                fence_proxy_async();  // the cp.async data, observed through the barrier, for the MMA
                ptx::tc_fence_after();
                x_mma(a1, bk(b1_off(j)), tmem + C::COL_X1);
                ptx::mma_commit(bar(C::B_X1));
            };
            auto issue_x2 = [&](int j) {
                fence_proxy_async();
                ptx::tc_fence_after();
                x_mma(a2, bk(b2_off(j)), tmem + C::COL_X2);
                ptx::mma_commit(bar(C::B_X2));
                if (!KV) ptx::mma_commit(bar(C::B_EMPTY2 + j % C::NS2));  // V_j: dP was its last reader
            };
            bool ok = ptx::mbar_wait(bar(C::B_STAT), 0, abort, lim);
            if (ok) fence_proxy_async();
            ok = ok && ptx::mbar_wait(bar(C::B_FULL1), 0, abort, lim);
            if (ok) issue_x1(0);
            ok = ok && ptx::mbar_wait(bar(C::B_FULL2), 0, abort, lim);
            if (ok) issue_x2(0);
            auto wait = [&](int b, int parity) { return ptx::mbar_wait(bar(b), parity, abort, lim); };
            // Per streamed tile j, in a fixed order (each wait suspends the thread in hardware until
            // its phase completes):
            //   key-major  : dV(j) once P^T(j) is in TMEM, S^T(j+1) (over the columns dV(j) has just
            //                read), dK(j) once dS^T(j) is in TMEM, dP^T(j+1) (over dS^T(j)'s columns)
            //   query-major: S(j+1) once the softmax has read S(j), dQ(j) once dS(j) is in TMEM,
            //                dP(j+1) (over dS(j)'s columns)
            for (int j = 0; ok && j < nstream; ++j) {
                const bool more = j + 1 < nstream;
                if (KV) {
                    ok = wait(C::B_P, j & 1);
                    if (!ok) break;
                    ptx::tc_fence_after();
                    acc_mma(C::COL_X1, bm(b2_off(j)), tmem + C::COL_ACC1, j > 0);  // dV += P^T dO
                    ptx::mma_commit(bar(C::B_EMPTY2 + j % C::NS2));                 // dO_j: dV was its last reader
                } else {
                    ok = wait(C::B_X1FREE, j & 1);
                    if (!ok) break;
                }
                if (more) {
                    ok = wait(C::B_FULL1 + (j + 1) % C::NS1, ((j + 1) / C::NS1) & 1);
                    if (!ok) break;
                    issue_x1(j + 1);
                }
                ok = wait(C::B_DS, j & 1);
                if (!ok) break;
                ptx::tc_fence_after();
                // key-major: dK += dS^T Q ; query-major: dQ += dS K
                acc_mma(C::COL_X2, bm(b1_off(j)), tmem + (KV ? C::COL_ACC2 : C::COL_ACC1), j > 0);
                ptx::mma_commit(bar(C::B_EMPTY1 + j % C::NS1));  // B1 of tile j: its last reader
                if (more) {
                    ok = wait(C::B_FULL2 + (j + 1) % C::NS2, ((j + 1) / C::NS2) & 1);
                    if (!ok) break;
                    issue_x2(j + 1);
                }
            }
            if (ok) {
                ptx::mma_commit(bar(C::B_ACC));
            } else {
                record_abort(abort, p.status);
            }
            // every MMA issued by this thread must finish before TMEM is released
            ptx::mma_commit(bar(C::B_DRAIN));
            volatile int never = 0;
            ptx::mbar_wait(bar(C::B_DRAIN), 0, &never, lim);
        }
        __syncwarp();
    } else {
        // ------------------------------------------------------------------ softmax halves
        const int h = warp >> 2;                        // streamed columns [64h, 64h+64)
        const int row = threadIdx.x & 127;              // TMEM lane == stationary row
        const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const uint32_t x1 = tmem + lane_base + C::COL_X1 + 64 * h;
        const uint32_t x2 = tmem + lane_base + C::COL_X2 + 64 * h;
        const float sl2 = p.scale_log2;
        const bool row_real = first + row < n_c;
        const int t_row = dF.div(min(first + row, n_c - 1));
        const bool one_frame = __all_sync(0xffffffffu, t_row == __shfl_sync(0xffffffffu, t_row, 0));  // of this warp's rows
        // bias of this row and streamed frame f
        auto bias_of = [&](int f) {
            return __uint_as_float(static_cast<uint32_t>(tab[clamp_dist(KV ? f - t_row : t_row - f, dmax)]) << 16) * kLog2E;
        };
        // Key-major: adds v, this row's sum of dS over queries of frame f, to the warp's table of
        // distances. Rows of equal distance are neighbours: their sum forms in the first of them.
        float* my_hist = hist + warp * p.ND;
        auto add_hist = [&](float v, int f) {
            const int u = clamp_dist(f - t_row, p.Dn) + p.Dn;
            if (!row_real) v = 0.f;
            if (one_frame) {
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
                if (lane == 0) my_hist[u] += v;
            } else {
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const float other = __shfl_down_sync(0xffffffffu, v, o);
                    const int uo = __shfl_down_sync(0xffffffffu, u, o);
                    if (lane + o < 32 && uo == u) v += other;
                }
                const int before = __shfl_up_sync(0xffffffffu, u, 1);
                if (lane == 0 || before != u) my_hist[u] += v;
            }
            __syncwarp();  // the next addition may come from another lane
        };
        float acc = 0.f;   // sum of dS over the queries of frame f_acc so far
        int f_acc = -1;
        float row_l2 = 0.f, row_d = 0.f;  // query-major: -L in log2, and D
        if (!KV) {
            // D of the tile's rows, from memory while the first keys travel: D / 8 lanes a row, 16 rows a warp
            float* d_of = reinterpret_cast<float*>(smem + C::OFF_VEC);
            constexpr int LPR = D / 8, RPW = 32 / LPR;
#pragma unroll 4
            for (int i = 0; i < 16; i += RPW) {
                const int r = warp * 16 + i + lane / LPR;
                const long long at = load_row(rows(min(first + r, n_c - 1)), p.nrows, p.status) * D + (lane % LPR) * 8;
                const float d = dot_of_row(p.out, p.out_lo, p.dout, at, LPR);
                if (lane % LPR == 0) d_of[r] = d;
            }
            const long long at = load_row(rows(min(first + row, n_c - 1)), p.nrows, p.status);
            const float l = __ldg(p.lse + at) * kLog2E;
            row_l2 = l == -INFINITY ? kNoKeys : -l;
            asm volatile("bar.sync 1, 256;" ::: "memory");
            row_d = d_of[row];
            if (h == 0 && row_real) p.nlse2[at] = row_l2;
        }
        float2 row_sum = make_float2(0.f, 0.f);  // query-major: of the row's dS
        bool ok = true;
        // the frame of the next column, the columns until the frame after it starts, and the bias
        int f = AL ? f_lo : dF.div(jbeg + 64 * h), next = (f + 1) * nF - (jbeg + 64 * h);
        float off = bias_of(f);
        for (int j = 0; j < nstream; ++j) {
            const int s1 = j % C::NS1;
            const int j0 = jbeg + j * kTileRows + 64 * h;
            const int valid = jend - j0;               // streamed rows in this half (may be <= 0)
            const int f0 = f, border = next;
            // every wait of a softmax warp is made uniform over the warp: the tcgen05.ld/st below
            // are .sync.aligned and need all 32 lanes
            if (!__all_sync(0xffffffffu, ptx::mbar_wait(bar(C::B_X1), j & 1, abort, lim))) {
                ok = false;
                break;
            }
            ptx::tc_fence_after();
            // the L/D vectors were written by the producers' cp.async: observe their barrier too
            if (KV && !__all_sync(0xffffffffu, ptx::mbar_wait(bar(C::B_FULL1 + s1), (j / C::NS1) & 1, abort, lim))) {
                ok = false;
                break;
            }
            const float* col_l = vecs + s1 * 2 * kTileRows + 64 * h;   // key-major: per column
            const float* col_d = col_l + kTileRows;
            float pr[64];
            int f_of[2];
            {
                uint32_t xv[64];
                ptx::tmem_ld32(x1, *reinterpret_cast<uint32_t(*)[32]>(&xv[0]));
                ptx::tmem_ld32(x1 + 32, *reinterpret_cast<uint32_t(*)[32]>(&xv[32]));
                ptx::tmem_wait_ld();
                if (!KV) {  // S is in registers: the tensor core may compute the next tile's S
                    ptx::tc_fence_before();
                    ptx::mbar_arrive(bar(C::B_X1FREE));
                }
                const float2 sl2x2 = make_float2(sl2, sl2);
#pragma unroll
                for (int g = 0; g < 2; ++g) {
                    int real = 32;      // aligned: columns of this chunk that are tokens
                    if (AL) {
                        const int q = 4 * j + 2 * h + g, fq = dC.div(min(q, chunks - 1));
                        real = q < chunks ? min(32, nF - (q - fq * cpf) * 32) : 0;
                        if (f_lo + fq != f) {
                            f = f_lo + fq;
                            off = bias_of(f);
                        }
                        f_of[g] = f;
                    }
                    if (AL || next >= 32) {  // 32 columns of one frame; two columns per instruction (packed f32x2)
                        const float2 o2 = make_float2(KV ? off : off + row_l2, KV ? off : off + row_l2);
#pragma unroll
                        for (int e4 = 0; e4 < 8; ++e4) {
                            float2 a = o2, b = o2;
                            if (KV) {
                                const float4 l4 = reinterpret_cast<const float4*>(col_l)[8 * g + e4];
                                a = __fadd2_rn(o2, make_float2(l4.x, l4.y));
                                b = __fadd2_rn(o2, make_float2(l4.z, l4.w));
                            }
                            const int e = 32 * g + 4 * e4;
                            a = __ffma2_rn(make_float2(__uint_as_float(xv[e]), __uint_as_float(xv[e + 1])), sl2x2, a);
                            b = __ffma2_rn(make_float2(__uint_as_float(xv[e + 2]), __uint_as_float(xv[e + 3])), sl2x2, b);
                            pr[e] = ptx::ex2_approx(a.x);
                            pr[e + 1] = ptx::ex2_approx(a.y);
                            pr[e + 2] = ptx::ex2_approx(b.x);
                            pr[e + 3] = ptx::ex2_approx(b.y);
                        }
                        if (AL && real < 32) {
#pragma unroll
                            for (int e = 0; e < 32; ++e)
                                if (e >= real) pr[32 * g + e] = 0.f;
                        }
                    } else if (nF >= 32) {  // one border
                        const float o1 = bias_of(++f);
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            pr[32 * g + e] = ptx::ex2_approx(
                                fmaf(__uint_as_float(xv[32 * g + e]), sl2, (e < next ? off : o1) + (KV ? col_l[32 * g + e] : row_l2)));
                        off = o1;
                        next += nF;
                    } else {  // frames of fewer tokens: a lookup per column
                        const int jg = j0 + 32 * g;
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            pr[32 * g + e] = ptx::ex2_approx(fmaf(__uint_as_float(xv[32 * g + e]), sl2,
                                                                  bias_of(dF.div(jg + e)) + (KV ? col_l[32 * g + e] : row_l2)));
                        f = dF.div(jg + 32);
                        next = (f + 1) * nF - jg;
                        off = bias_of(f);
                    }
                    next -= 32;
                }
                next -= 64;  // the other warpgroup's columns
                if (!AL && next <= 0) {
                    f = dF.div(j0 + kTileRows);
                    next = (f + 1) * nF - (j0 + kTileRows);
                    off = bias_of(f);
                }
                if (!AL && valid < 64) {  // the ragged last tile: repeated streamed rows give 0
#pragma unroll
                    for (int e = 0; e < 64; ++e)
                        if (e >= valid) pr[e] = 0.f;
                }
            }
            if (KV) {  // P^T for dV += P^T dO
#pragma unroll
                for (int g = 0; g < 2; ++g) {
                    uint32_t pk[16];
#pragma unroll
                    for (int e = 0; e < 16; ++e) pk[e] = ptx::pack_bf16x2(pr[32 * g + 2 * e], pr[32 * g + 2 * e + 1]);
                    ptx::tmem_st16(x1 + 16 * g, pk);
                }
                ptx::tmem_wait_st();
                ptx::tc_fence_before();
                ptx::mbar_arrive(bar(C::B_P));
                if (!AL && f_acc != f0) {  // uniform over the warp: all rows see the same columns
                    if (f_acc >= 0) add_hist(acc, f_acc);
                    acc = 0.f;
                    f_acc = f0;
                }
            }
            if (!__all_sync(0xffffffffu, ptx::mbar_wait(bar(C::B_X2), j & 1, abort, lim))) {
                ok = false;
                break;
            }
            ptx::tc_fence_after();
            int ends = border;  // key-major: column, from the chunk's first, where the frame changes next
#pragma unroll
            for (int g = 0; g < 2; ++g) {
                // 32 columns at a time: 13 warps leave 128 registers a thread, and P is live
                uint32_t dv[32];
                ptx::tmem_ld32(x2 + 32 * g, dv);
                ptx::tmem_wait_ld();
                uint32_t pk[16];
                float2 sum = make_float2(0.f, 0.f);
#pragma unroll
                for (int e4 = 0; e4 < 4; ++e4) {
                    const int e0 = 32 * g + 8 * e4;
                    float dcol[8];
                    if (KV) {  // key-major: each column's D, four at a time
                        const float4 a = reinterpret_cast<const float4*>(col_d)[e0 / 4];
                        const float4 b = reinterpret_cast<const float4*>(col_d)[e0 / 4 + 1];
                        dcol[0] = a.x; dcol[1] = a.y; dcol[2] = a.z; dcol[3] = a.w;
                        dcol[4] = b.x; dcol[5] = b.y; dcol[6] = b.z; dcol[7] = b.w;
                    } else {
#pragma unroll
                        for (int e = 0; e < 8; ++e) dcol[e] = row_d;
                    }
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int c = 8 * e4 + 2 * e;  // column inside this 32-column chunk
                        const float2 sv = ds_pair(make_float2(pr[32 * g + c], pr[32 * g + c + 1]),
                                                  make_float2(dcol[2 * e], dcol[2 * e + 1]), dv[c], dv[c + 1]);
                        pk[4 * e4 + e] = ptx::pack_bf16x2(sv.x, sv.y);
                        sum = __fadd2_rn(sum, sv);
                        if (KV && !AL) {
                            dv[c] = __float_as_uint(sv.x);
                            dv[c + 1] = __float_as_uint(sv.y);
                        }
                    }
                }
                if (KV && AL) {
                    if (f_acc != f_of[g]) {  // uniform over the warp: all rows see the same columns
                        if (f_acc >= 0) add_hist(acc, f_acc);
                        acc = 0.f;
                        f_acc = f_of[g];
                    }
                    acc += sum.x + sum.y;
                }
                if (KV && !AL) {
                    if (ends >= 32) {
                        acc += sum.x + sum.y;
                    } else {  // frames end in this chunk: sum each one's columns
                        int lo = 0;
#pragma unroll 1
                        while (lo < 32) {
                            const int hi = min(ends, 32);
                            float s = 0.f;
#pragma unroll
                            for (int e = 0; e < 32; ++e)
                                s += (e >= lo && e < hi) ? __uint_as_float(dv[e]) : 0.f;
                            acc += s;
                            if (hi < 32) {
                                add_hist(acc, f_acc);
                                acc = 0.f;
                                ++f_acc;
                                ends += nF;
                            }
                            lo = hi;
                        }
                    }
                    ends -= 32;
                }
                if (!KV) row_sum = __fadd2_rn(row_sum, sum);
                ptx::tmem_st16(x2 + 16 * g, pk);
            }
            ptx::tmem_wait_st();
            ptx::tc_fence_before();
            ptx::mbar_arrive(bar(C::B_DS));
            // a frame that ends with these columns is added when the next tile's frame differs;
            // f_acc is the frame of the last column
        }
        if (KV && ok && f_acc >= 0) add_hist(acc, f_acc);
        if (ok && (nstream == 0 || __all_sync(0xffffffffu, ptx::mbar_wait(bar(C::B_ACC), 0, abort, lim)))) {
            ptx::tc_fence_after();
            const int si = first + row;                 // stationary row (key or query)
            const bool store = si < n_c && row_ok(rows(si), p.nrows, p.status);
            const size_t grow = store ? static_cast<size_t>(rows(si)) : 0;
            if (!KV) {
                // The row's dS ought to sum to zero; what it sums to is D's error, which goes into D
                // for the key-major kernel.
                float* other = reinterpret_cast<float*>(smem + C::OFF_VEC) + kTileRows + row;
                if (h == 1) *other = row_sum.x + row_sum.y;
                asm volatile("bar.sync 1, 256;" ::: "memory");
                if (h == 0 && store) p.delta[grow] = row_d + ((row_sum.x + row_sum.y) + *other);
            }
            constexpr int HALF = D / 2;                 // accumulator columns of this warpgroup
            // key-major: acc1 = dV (unscaled), acc2 = dK ; query-major: acc1 = dQ
#pragma unroll
            for (int which = 0; which < (KV ? 2 : 1); ++which) {
                const uint32_t col = tmem + lane_base + (which ? C::COL_ACC2 : C::COL_ACC1) + HALF * h;
                const float mul = (KV && which == 0) ? 1.f : p.scale;
                uint16_t* out = KV ? (which ? p.dk : p.dv) : p.dq;
#pragma unroll
                for (int g = 0; g < HALF / 16; ++g) {
                    uint32_t av[16];
                    if (nstream > 0) {
                        ptx::tmem_ld16(col + 16 * g, av);
                        ptx::tmem_wait_ld();
                    } else {  // nothing sees this tile
#pragma unroll
                        for (int e = 0; e < 16; ++e) av[e] = 0u;
                    }
                    uint32_t pk[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        pk[e] = ptx::pack_bf16x2(__uint_as_float(av[2 * e]) * mul, __uint_as_float(av[2 * e + 1]) * mul);
                    if (store) {
                        uint4* dst = reinterpret_cast<uint4*>(out + grow * D + HALF * h + 16 * g);
                        dst[0] = make_uint4(pk[0], pk[1], pk[2], pk[3]);
                        dst[1] = make_uint4(pk[4], pk[5], pk[6], pk[7]);
                    }
                }
            }
        } else {
            if (!*abort) record_abort(abort, p.status);
            if (!KV) asm volatile("bar.arrive 1, 256;" ::: "memory");  // for warps that saw no failure
        }
    }

    ptx::tc_fence_before();
    __syncthreads();
    if (warp == kBwdMma) {
        ptx::tc_fence_after();
        ptx::tmem_dealloc(tmem, C::NCOLS);
    }
    if (KV) {  // this CTA's sums by distance, its warps' tables added in order
        const size_t n = static_cast<size_t>(p.seqs) * p.tiles;
        float* part = p.part + static_cast<size_t>(head) * p.ND * n + static_cast<size_t>(seq) * p.tiles + tile;
        for (int u = threadIdx.x; u < p.ND; u += kBwdThreads) {
            float s = 0.f;
#pragma unroll
            for (int w = 0; w < 8; ++w) s += hist[w * p.ND + u];
            part[u * n] = s;
        }
    }
}

// dtable of one head: the CTAs' sums added per distance (one warp each), then the distances of each
// bucket.
constexpr int kTableThreads = 1024;
__global__ void __launch_bounds__(kTableThreads) skiparse_frames_dtable_kernel(const FramesBwdParams p) {
    __shared__ float sums[kMaxDistEntries];
    __shared__ int tiles_of[kMaxAxisClasses];  // key tiles of each class; the others were not launched
    const int head = blockIdx.x;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int q2 = p.g.Ph * p.g.Pw;
    if (threadIdx.x < q2) {
        const int c = threadIdx.x;
        tiles_of[c] = (p.g.T * p.g.Rc[c / p.g.Pw] * p.g.Sc[c % p.g.Pw] + kTileRows - 1) / kTileRows;
    }
    __syncthreads();
    const int n = p.seqs * p.tiles;
    const float* part = p.part + static_cast<size_t>(head) * p.ND * n;
    for (int u = warp; u < p.ND; u += kTableThreads / 32) {
        float s = 0.f;
        for (int i = lane; i < n; i += 32) {
            const int seq = i / p.tiles;
            if (i - seq * p.tiles < tiles_of[seq % q2]) s += part[static_cast<size_t>(u) * n + i];
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        if (lane == 0) sums[u] = s;
    }
    __syncthreads();
    for (int g = threadIdx.x; g < p.bias.NB; g += kTableThreads) {
        float s = 0.f;
        for (int u = 0; u < p.ND; ++u)
            if (p.bias.buckets[u - p.Dn + p.bias.D] == g) s += sums[u];
        p.dtable[static_cast<size_t>(g) * p.g.heads + head] = __bfloat16_as_ushort(__float2bfloat16_rn(s));
    }
}

template <int D, bool KV, bool AL>
int launch_bwd_d(const FramesBwdParams& p, const Geometry& g, cudaStream_t stream) {
    using C = BwdCfg<D, KV>;
    // per device: the kernel's shared-memory attribute is set (host threads may race here;
    // setting it twice is harmless, the flag only has to be a race-free read)
    static std::atomic<int> attr_done_dev[64];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return static_cast<int>(e);
    if (dev < 0 || dev >= 64 || !attr_done_dev[dev].load(std::memory_order_acquire)) {
        e = cudaFuncSetAttribute(skiparse_frames_bwd_kernel<D, KV, AL>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 C::SMEM_BYTES);
        if (e != cudaSuccess) return static_cast<int>(e);
        if (dev >= 0 && dev < 64) attr_done_dev[dev].store(1, std::memory_order_release);
    }
    const dim3 grid(static_cast<unsigned>(p.tiles * g.heads * p.seqs));
    skiparse_frames_bwd_kernel<D, KV, AL><<<grid, kBwdThreads, C::SMEM_BYTES, stream>>>(p);
    return static_cast<int>(cudaGetLastError());
}

// Whether the key-major kernel streams its queries in 32-row chunks of one frame each (the last of
// a frame filled up): no chunk then holds a frame's border, whose handling costs the kernel
// registers everywhere, for up to twice the rows. 480p (390 tokens a frame, 7 % more rows): 3.77 ms
// with borders, 3.45 without; 20 tokens a frame (60 % more), 4 x 16 frames: 84 us with borders, 60 without.
bool aligned_chunks(int nF) { return (nF + 31) / 32 * 32 <= nF * 2; }

template <int D>
int launch_bwd_all(const FramesBwdParams& p, const Geometry& g, cudaStream_t st) {
    int e = launch_bwd_d<D, false, false>(p, g, st);
    if (e) return e;
    e = aligned_chunks(max_class_tokens(g)) ? launch_bwd_d<D, true, true>(p, g, st) : launch_bwd_d<D, true, false>(p, g, st);
    if (e) return e;
    skiparse_frames_dtable_kernel<<<g.heads, kTableThreads, 0, st>>>(p);
    return static_cast<int>(cudaGetLastError());
}

}  // namespace

int launch_frames_bwd(const FramesBwdParams& p, const Geometry& g, void* stream) {
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    switch (g.d) {
        case 32: return launch_bwd_all<32>(p, g, st);
        case 64: return launch_bwd_all<64>(p, g, st);
        case 128: return launch_bwd_all<128>(p, g, st);
        default: return static_cast<int>(cudaErrorInvalidValue);
    }
}

}  // namespace skiparse
