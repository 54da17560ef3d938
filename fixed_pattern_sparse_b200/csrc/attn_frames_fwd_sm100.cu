// attn_frames_fwd_sm100.cu -- class attention with a learned bias by frame distance, forward, over
// bf16 keys and values or over the e4m3 frame cache (sm_100a).
//
// For one (b, class, head) subsequence, a query x at frame t_x and a key y at frame t_y:
//   s_xy = q_x . k_y / sqrt(d) + bias[clamp(t_x - t_y, -D, D)],   out_x = softmax_y(s_xy) v_y,
// where a bias of -inf masks the pair; a row without a visible key gives 0 (lse -inf).
//
// The schedule is that of the unbiased forward (attn_fwd_sm100.cu): a CTA owns 256 queries as two
// 128-row tiles, streams 128-key tiles of K and V through shared-memory rings of two slots,
// S = Q K^T and O += P V run on tcgen05 with S, P and O in TMEM, one thread per query row does
// the online softmax with the lazy rescale. What the frames add:
//   * The bias is constant over the tokens of a frame, so a key tile inside one frame needs one table
//     lookup per row, folded into the softmax's existing FMA: no instruction per score. For tiles
//     that hold a frame's border the bias comes as further columns of Q and K (bf16 keys, frames of
//     64 tokens and more: BiasCols below), or by a pass over S in TMEM before the softmax.
//   * The frames that some row of the CTA can see form a range, from the first and last visible
//     distance of the table; only its keys are loaded. With a causal map that is half the work. (In a
//     cache whose ring has turned over, frames do not lie in order of time: all are loaded, whatever the mask.)
//     Query tiles are launched last frame first, so that the longest ones start first (TileOrder).
//   * Cached keys are e4m3 codes. Three producer warps for K and three for V copy them into
//     a staging buffer, expand them to f16 (one conversion per two codes, exact) and store them
//     into the swizzled tile; the tensor core then works on f16 operands. A block's scale enters
//     as 2^(e - ref), ref the largest e among the keys this CTA reads, so that a single power
//     of two for K (in the softmax's factor) and one for V (in the epilogue) are left. Where the
//     scales of these keys, masked ones included, spread beyond what that holds (kWideK, kWideV), the
//     codes enter unscaled, K's scale multiplies the score and V's joins the exponent of its weight
//     (wide_softmax): a block counts by its own values whatever the others' scales. Q's rows are
//     scaled by a power of two each into f16, and P is kept as 2^7 p, so that f16 holds every p above
//     2^-31: P's rounding is 2^-11 instead of bf16's 2^-8.
//   * Few query tiles over a long cache leave SMs idle, and so does a last wave of few CTAs: the key
//     range of these tiles is cut into parts, each CTA writes its normalised partial output and
//     log-sum-exp in fp32, and a second kernel joins them.
//   * Calls of few query tiles: a CTA may own 128 queries instead, its two softmax groups taking
//     every other key tile each (an own O in TMEM each, joined at the end), which halves the
//     length of a CTA and doubles their number.
// Shared memory at d = 128: Q 64 KB, K and V rings 64 KB each, table 2 KB, staging (cache) 32 KB or bias
// columns (bf16) 32 KB.
// What bounds it, 480p (21 frames of 390 tokens a class, d = 128, 12 heads): 1.45 ms for 1.65 TFLOP, 1140
// TFLOP/s, at 1965 MHz (1.6 in training steps back to back, under the power cap). A key step of 256
// queries takes 3100 to 3500 clocks against 2048 of tensor core and as many of exponentials; the rest is
// the dependency of the two tiles' softmax and products on each other. The cache form adds the expansion
// of the codes: 0.68 ms for three frames over 24 (760 TFLOP/s).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <atomic>
#include <initializer_list>

#include "frames_common.cuh"

namespace skiparse {
namespace {

constexpr int kBM = 128;
constexpr int kBN = 128;
constexpr int kProdWarp0 = 8;
constexpr int kMaxSmem = 232448;      // 227 KB, the most a CTA may have
constexpr float kRescaleLog2 = 8.0f;  // rescale O only when the max grows by more than 2^8
constexpr int kPParts = 2;            // P is released to the tensor core in two halves of the key tile
// Largest spread, as a power of two, of the scales of a CTA's keys at which they enter the codes as f16
// factors. K: a code's last bit is worth 2^-9 or more, f16's 2^-24: the product is exact. V: so is it, but weights
// are off by up to 2^-32 of the row's largest, times 2^spread where that one's block is the smallest.
constexpr int kWideK = 15, kWideV = 8;

// The bias as part of S = Q K^T (bf16 keys): 16 more columns of Q and K. The frames of a CTA's queries, at
// most five, are numbered; a query's row holds ones in the three columns of its frame, a key's row holds,
// for each of these frames, its bias for that frame's queries in units of q.k as the sum of three bf16
// numbers (24 bits), so that the tensor core adds it to each score in fp32. That replaces a pass over S in
// TMEM for every tile that holds a frame's border; a CTA whose queries lie in more frames takes the pass.
// A key's row depends on its distance from the first of the queries' frames only: these rows are made
// once per CTA and copied. Taken by 256-query CTAs and frames of up to 8 d tokens: 390 tokens, d = 128:
// 1.53 -> 1.44 ms, as fast as without a bias; 225, d = 64: 642 -> 598 us; 81, d = 32: 621 -> 511 us. Beyond,
// borders are rare and the MMA step costs more than they do (1296, d = 128: 1.36 -> 1.37 ms; 900, d = 64:
// 1.05 -> 1.09 ms), and in 128-query CTAs, which load twice the keys, so do the producers' copies (144
// tokens, d = 128: 42.5 -> 45.5 us).
struct BiasCols {
    static constexpr int FRAMES = 5, ROW = 32, TILE_BYTES = kBN * ROW;
    static constexpr uint32_t LAYOUT = 6;           // 32-byte swizzle
    static constexpr int MAX_ROWS = kMaxDistEntries + FRAMES - 1;  // distances -D-4 .. D
    // A masked pair: far below any score, and finite, since zeros multiply it for the other frames.
    static constexpr float MASKED = -1.7014118346046923e38f;  // -2^127
    // Scaled scores beyond +-FAR stand for masked keys, or for an entry of the table that is not finite.
    static constexpr float FAR_LOG2 = 1e35f;

    static __device__ __forceinline__ void store16(uint32_t at, const uint32_t (&w)[4]) {
        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]) : "memory");
    }
    // Address of 16-byte half c of row r of a tile.
    static __device__ __forceinline__ uint32_t half_at(uint32_t tile, int r, int c) {
        return tile + r * ROW + ((c ^ ((r >> 2) & 1)) << 4);
    }
    // Row r of a query tile: ones for frame number fi.
    static __device__ __forceinline__ void store_query(uint32_t tile, int r, int fi) {
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            uint32_t w[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int lo = 8 * c + 2 * e - 3 * fi, hi = lo + 1;
                w[e] = (lo >= 0 && lo < 3 ? 0x3f80u : 0u) | (hi >= 0 && hi < 3 ? 0x3f800000u : 0u);
            }
            store16(half_at(tile, r, c), w);
        }
    }
    // The row, at `at`, of keys at distance u from the queries' first frame; tab: the bias by distance in log2.
    static __device__ __forceinline__ void make_row(uint32_t at, const float* tab, int u, int dmax, float sl2) {
        uint32_t t[16];
#pragma unroll
        for (int i = 0; i < FRAMES; ++i) {
            const float l2 = tab[clamp_dist(u + i, dmax) + dmax];
            float x = l2 == -INFINITY ? MASKED : fabsf(l2) < 1e37f ? l2 / sl2 : -MASKED;
#pragma unroll
            for (int e = 0; e < 3; ++e) {
                t[3 * i + e] = __bfloat16_as_ushort(__float2bfloat16_rn(x));
                x -= __uint_as_float(t[3 * i + e] << 16);
            }
        }
        t[15] = 0u;
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            const uint32_t w[4] = {t[8 * c] | t[8 * c + 1] << 16, t[8 * c + 2] | t[8 * c + 3] << 16,
                                   t[8 * c + 4] | t[8 * c + 5] << 16, t[8 * c + 6] | t[8 * c + 7] << 16};
            store16(at + 16 * c, w);
        }
    }
    // Row r of a key tile, for a key at distance u from the queries' first frame.
    static __device__ __forceinline__ void store_key(uint32_t tile, int r, uint32_t rows, int u, int dmax) {
        const uint32_t at = rows + (min(max(u, -dmax - FRAMES + 1), dmax) + dmax + FRAMES - 1) * ROW;
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            uint32_t w[4];
            asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "r"(at + 16 * c));
            store16(half_at(tile, r, c), w);
        }
    }
};

template <int D, bool CACHE>
struct Cfg : TileGeom<D> {
    using G = TileGeom<D>;
    using G::TILE_BYTES;
    // bf16: producers 8-9, MMA 10. Cache: producers of K 8-10 and of V 12-14, MMA 15, so that the
    // MMA issuer's sub-partition has no producer; 11 idles.
    static constexpr int MMA_WARP = CACHE ? 15 : kProdWarp0 + 2;
    static constexpr int THREADS = 32 * (MMA_WARP + 1);
    static constexpr int FULL_COUNT = CACHE ? 3 : 64;  // arrivals per tile
    static constexpr int KST = 2, VST = 2;
    static constexpr uint32_t COL_S0 = 0, COL_S1 = 128, COL_O0 = 256, COL_O1 = 256 + D;
    static constexpr uint32_t NCOLS = 512;
    static constexpr int OFF_Q = 0;
    static constexpr int OFF_K = 2 * TILE_BYTES;
    static constexpr int OFF_V = OFF_K + KST * TILE_BYTES;
    static constexpr int OFF_STAGE = OFF_V + VST * TILE_BYTES;  // cache: a tile of codes of K and of V
    // bf16: the bias columns of the two query tiles and of the K ring's slots (see BiasCols)
    static constexpr int OFF_QB = OFF_STAGE;
    static constexpr int OFF_KB = OFF_QB + 2 * BiasCols::TILE_BYTES;
    static constexpr int OFF_ROWS = OFF_KB + KST * BiasCols::TILE_BYTES;
    static constexpr int OFF_TAB =                                // bias by distance index
        CACHE ? OFF_STAGE + 2 * kBN * D : OFF_ROWS + BiasCols::MAX_ROWS * BiasCols::ROW;
    static constexpr int OFF_BAR = OFF_TAB + 4 * (kMaxDistEntries + 1);
    static constexpr int B_Q = 0;
    static constexpr int B_KFULL = 1;
    static constexpr int B_KEMPTY = B_KFULL + KST;
    static constexpr int B_VFULL = B_KEMPTY + KST;
    static constexpr int B_VEMPTY = B_VFULL + VST;
    static constexpr int B_SFULL = B_VEMPTY + VST;
    static constexpr int B_PFULL = B_SFULL + 2;
    static constexpr int B_OFULL = B_PFULL + 2 * kPParts;
    static constexpr int B_DRAIN = B_OFULL + 1;
    static constexpr int B_QF16 = B_DRAIN + 1;               // cache: Q has been turned into f16
    static constexpr int NBARS = B_QF16 + 1;
    static constexpr int OFF_TMEM_SLOT = OFF_BAR + 8 * NBARS;
    static constexpr int OFF_ABORT = OFF_TMEM_SLOT + 4;
    static constexpr int OFF_RANGE = OFF_ABORT + 4;  // first and last visible distance
    static constexpr int OFF_REF = OFF_RANGE + 8;    // cache: largest scale bytes of K and V, then smallest
    static constexpr int SMEM_USED = OFF_REF + 16;
    // + slack for 1024-byte alignment where it fits (the kernel checks the slack it got); at
    // least 116 KB so that one CTA (and its 512 TMEM columns) owns an SM even for small d
    static constexpr int SMEM_BYTES =
        SMEM_USED + 1024 > kMaxSmem ? kMaxSmem : (SMEM_USED + 1024 > 118784 ? SMEM_USED + 1024 : 118784);
    static_assert(COL_O1 + D <= NCOLS, "TMEM overflow");
    static_assert(SMEM_USED + 256 <= kMaxSmem, "shared memory overflow");
};

// Instruction descriptor of kind::f16 with f16 (instead of bf16) A and B.
constexpr uint32_t f16_operands(uint32_t idesc) { return idesc & ~((1u << 7) | (1u << 10)); }

// One producer lane's part of the tiles of codes of K or V: a 16-byte chunk (16 codes) of every third
// row group. The chunks travel by cp.async through a staging buffer in shared memory that only
// the lane itself reads, the scale bytes through registers.
template <int D>
struct CacheTile {
    static constexpr int CPR = D / 16;            // chunks per row of codes
    static constexpr int RPI = 32 / CPR;          // rows per warp instruction
    static constexpr int NG = kBN / RPI;          // row groups of a tile
    static constexpr int PER = (NG + 2) / 3;      // row groups of a warp
    static constexpr int STAGE_BYTES = NG * 512;  // a tile of codes
    uint32_t byte[PER < 3 ? 3 : PER];             // scale bytes, then factors
    int at0;                                      // of the tile whose bytes these are: its first token's
    bool inside;                                  // place in its frame, and whether it lies in one
    const uint8_t* codes;                         // of this (subsequence, head)
    const uint8_t* scales;
    uint32_t stage;                               // this lane's first chunk
    int pw, lane;

    static __device__ __forceinline__ bool mine(int i, int pw) { return 3 * i + 2 < NG || pw + 3 * i < NG; }
    __device__ __forceinline__ void init(const uint8_t* codes_, const uint8_t* scales_, uint32_t stage_base, int pw_, int lane_) {
        codes = codes_;
        scales = scales_;
        pw = pw_;
        lane = lane_;
        stage = stage_base + pw * 512 + lane * 16;
    }
    // Starts the copies of the keys j0..j0+127 of the class, those from jend on repeating the last, and
    // loads their scale bytes: of a tile inside one frame the three that it can meet, else one a row.
    __device__ __forceinline__ void fetch(int j0, int jend, const FastDiv& dF, int nF, const CacheView& cv, int* status) {
        const int c = lane % CPR, rsub = lane / CPR;
        const int slot0 = dF.div(j0);
        at0 = j0 - slot0 * nF;
        inside = at0 + kBN <= nF && j0 + kBN <= jend;
        const long long rows = static_cast<long long>(cv.cap) * cv.F;
        const int gap = cv.F - nF;  // unused places of a slot
        if (inside) {
            const long long row0 = load_row(j0 + static_cast<long long>(slot0) * gap + pw * RPI + rsub, rows, status);
            const uint8_t* src = codes + row0 * D + c * 16;
#pragma unroll
            for (int i = 0; i < PER; ++i)
                if (mine(i, pw)) cp_async_16(stage + i * 3 * 512, src + i * 3 * RPI * D);
            const uint8_t* sc = scales + static_cast<long long>(slot0) * cv.NBk;
            const int last = (at0 + kBN - 1) / kCacheBlock;
#pragma unroll
            for (int i = 0; i < 3; ++i) byte[i] = __ldg(sc + min(at0 / kCacheBlock + i, last));
        } else {
#pragma unroll
            for (int i = 0; i < PER; ++i)
                if (mine(i, pw)) {
                    const int j = min(j0 + (pw + 3 * i) * RPI + rsub, jend - 1);
                    const int slot = dF.div(j);
                    const long long row = load_row(j + static_cast<long long>(slot) * gap, rows, status);
                    cp_async_16(stage + i * 3 * 512, codes + row * D + c * 16);
                    byte[i] = __ldg(scales + slot * cv.NBk + (j - slot * nF) / kCacheBlock);
                }
        }
        cp_async_commit();
    }
    // Whether every scale of the warp's rows is the reference; if not, byte[] becomes the factors
    // 2^(scale - ref) row by row.
    __device__ __forceinline__ bool all_ref(int ref) {
        const uint32_t r = static_cast<uint32_t>(ref);
        if (inside) {
            const uint32_t b0 = byte[0], b1 = byte[1], b2 = byte[2];
            if (b0 == r && b1 == r && b2 == r) return true;
            const uint32_t m0 = scale_f16x2(b0, ref), m1 = scale_f16x2(b1, ref), m2 = scale_f16x2(b2, ref);
            const int r0 = at0 % kCacheBlock + pw * RPI + lane / CPR;
#pragma unroll
            for (int i = 0; i < PER; ++i)
                byte[i] = r0 + 3 * i * RPI < kCacheBlock ? m0 : r0 + 3 * i * RPI < 2 * kCacheBlock ? m1 : m2;
            return false;
        }
        bool one = true;
#pragma unroll
        for (int i = 0; i < PER; ++i)
            if (mine(i, pw)) one = one && byte[i] == r;
        if (__all_sync(0xffffffffu, one)) return true;
#pragma unroll
        for (int i = 0; i < PER; ++i)
            if (mine(i, pw)) byte[i] = scale_f16x2(byte[i], ref);
        return false;
    }
    // Expands the staged tile into the swizzled f16 tile at dst, times byte[] if SCALED.
    template <bool SCALED>
    __device__ __forceinline__ void expand(uint32_t dst) const {
        using C = TileGeom<D>;
        const int c = lane % CPR, rsub = lane / CPR;
        // A chunk gives two 16-byte stores; the lanes of a row's second box start with their second
        // half, so that the lanes of a row never meet in a bank. The rows of a lane are 3 * RPI
        // apart: their swizzles repeat after two (D = 128) or do not change.
        const int flip = (c * 32 / C::SW) & 1;
        const int r0 = pw * RPI + rsub;
        const uint32_t even[2] = {dst + tile_chunk<D>(r0, 2 * c + flip), dst + tile_chunk<D>(r0, 2 * c + 1 - flip)};
        const uint32_t odd[2] = {dst + tile_chunk<D>(r0 + 3 * RPI, 2 * c + flip) - 3 * RPI * C::SW,
                                 dst + tile_chunk<D>(r0 + 3 * RPI, 2 * c + 1 - flip) - 3 * RPI * C::SW};
        const uint32_t half_at[2] = {stage + 8 * flip, stage + 8 - 8 * flip};
        // loads in batches, ahead of the conversions that use them (all of them at once, to free the
        // staging buffer for the next tile earlier, was slower: the registers do not suffice)
        constexpr int BATCH = 4;
#pragma unroll
        for (int i0 = 0; i0 < PER; i0 += BATCH) {
            uint32_t w[2 * BATCH][2];
#pragma unroll
            for (int i = i0; i < i0 + BATCH && i < PER; ++i)
#pragma unroll
                for (int half = 0; half < 2; ++half)
                    if (mine(i, pw))
                        asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];"
                                     : "=r"(w[2 * (i - i0) + half][0]), "=r"(w[2 * (i - i0) + half][1])
                                     : "r"(half_at[half] + i * 3 * 512));
#pragma unroll
            for (int i = i0; i < i0 + BATCH && i < PER; ++i)
                if (mine(i, pw)) {
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        const uint32_t* x = w[2 * (i - i0) + half];
                        uint32_t y[4];
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            y[2 * e] = e4m3x2_to_f16x2(static_cast<uint16_t>(x[e]));
                            y[2 * e + 1] = e4m3x2_to_f16x2(static_cast<uint16_t>(x[e] >> 16));
                        }
                        if (SCALED) {
#pragma unroll
                            for (int e = 0; e < 4; ++e) y[e] = f16x2_mul(y[e], byte[i]);
                        }
                        const uint32_t at = ((i & 1) ? odd[half] : even[half]) + i * 3 * RPI * C::SW;
                        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(y[0]), "r"(y[1]), "r"(y[2]),
                                     "r"(y[3])
                                     : "memory");
                    }
                }
        }
    }
};

// Turns one row of a Q tile in shared memory from bf16 into f16, times the power of two that puts
// the row's largest magnitude in [2^7, 2^8): exact for values down to 2^-22 of it, within 2^-33 of
// it below. Returns that power's exponent (the row is 2^exponent times what is stored).
template <int D>
__device__ __forceinline__ int q_row_to_f16(uint32_t tile, int row) {
    uint32_t top = 0;
#pragma unroll
    for (int c = 0; c < D / 8; ++c) {
        uint32_t v[4];
        asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
                     : "r"(tile + tile_chunk<D>(row, c)));
#pragma unroll
        for (int e = 0; e < 4; ++e) top = __vmaxu2(top, v[e] & 0x7fff7fffu);
    }
    top = max(top & 0xffffu, top >> 16);
    const int up = top == 0 ? 0 : max(static_cast<int>(top >> 7), 8) - 134;  // 127 + 7
    const float f = exp2_int(-up);
#pragma unroll
    for (int c = 0; c < D / 8; ++c) {
        const uint32_t at = tile + tile_chunk<D>(row, c);
        uint32_t v[4];
        asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
                     : "r"(at));
#pragma unroll
        for (int e = 0; e < 4; ++e)
            v[e] = pack_f16x2(__uint_as_float(v[e] << 16) * f, __uint_as_float(v[e] & 0xffff0000u) * f);
        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3])
                     : "memory");
    }
    return up;
}

// The softmax of a query tile over keys whose scales spread (see kWideK): what it needs, as its caller has it.
struct WideArgs {
    int jbeg, jend, nF, step, first, tiles;  // key tile j of this query tile starts at jbeg + first + j * step
    int tq, dmax, NBk;
    uint32_t s_addr, o_addr, sfull, pfull;
    float sl2;
    const float* tab;
    const uint8_t* k_scales;
    const uint8_t* v_scales;
    FastDiv dF;
    FrameRing ring;
    volatile int* abort;
    uint64_t lim;
};
// S becomes the score plus the exponent of its value's block, whose running maximum m_w is the reference of the
// weights; the row sum l and its reference m are taken from the scores alone. Returns m, l, m_w and whether
// every wait ended. Such calls take 3 times as long (480p chunk 0.70 -> 2.3 ms, 720p frame 1.65 -> 5.1; d = 64 and 32
// twice: 333 -> 665 us, 288 -> 628). A function
// of its own: inlined, they take 2.3 to 2.5 times as long, but its presence costs the others 4 to 14 % (720p
// frame 1.59 ms without it, 1.64 so, 1.67 to 1.81 inlined in several ways).
template <int D>
__device__ __noinline__ float4 wide_softmax(const WideArgs& a) {
    float m_w = -INFINITY, m = -INFINITY, l = 0.f;
    bool ok = true;
    const auto bias_of = [&](int f) { return a.tab[clamp_dist(a.tq - a.ring.time(f), a.dmax) + a.dmax]; };
    for (int j = 0; ok && j < a.tiles; ++j) {
        const int j0 = a.jbeg + j * a.step + a.first;
        ok = __all_sync(0xffffffffu, ptx::mbar_wait(a.sfull, j & 1, a.abort, a.lim));
        if (!ok) break;
        ptx::tc_fence_after();
        float mx = -INFINITY;
#pragma unroll 1
        for (int g = 0; g < kBN / 16; ++g) {
            const int jg = j0 + 16 * g;
            uint32_t sv[16];
            ptx::tmem_ld16(a.s_addr + 16 * g, sv);
            ptx::tmem_wait_ld();
            // scale of K, exponent of V and bias of key i, past the end those of the last
            auto of_key = [&](int i, float& ks, float& ev, float& bias) {
                i = min(i, a.jend - 1);
                const int f = a.dF.div(i);
                const long long at = static_cast<long long>(f) * a.NBk + (i - f * a.nF) / kCacheBlock;
                const int kb = __ldg(a.k_scales + at), vb = __ldg(a.v_scales + at);
                ks = kb == 255 ? NAN : exp2_int(kb - 127);
                ev = vb == 255 ? NAN : static_cast<float>(vb - 127);
                bias = bias_of(f);
            };
            float ev[16], top = m;
            const int at0 = jg - a.dF.div(min(jg, a.jend - 1)) * a.nF;
            if (jg + 16 <= a.jend && at0 + 16 <= a.nF && at0 % kCacheBlock + 16 <= kCacheBlock) {  // one block
                float ks, bias;
                of_key(jg, ks, ev[0], bias);
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    const float x = bias == -INFINITY ? bias : fmaf(__uint_as_float(sv[e]) * a.sl2, ks, bias);
                    sv[e] = __float_as_uint(x);
                    ev[e] = ev[0];
                    top = fmaxf(top, x);
                }
            } else {
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    float ks, bias;
                    of_key(jg + e, ks, ev[e], bias);
                    const bool hidden = jg + e >= a.jend || bias == -INFINITY;
                    const float x = hidden ? -INFINITY : fmaf(__uint_as_float(sv[e]) * a.sl2, ks, bias);
                    sv[e] = __float_as_uint(x);
                    top = fmaxf(top, x);
                }
            }
            const float ref = top == -INFINITY ? 0.f : top;  // no key seen yet, or NaNs alone
            l *= ptx::ex2_approx(m - ref);
            m = top;
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                const float x = __uint_as_float(sv[e]);
                l += ptx::ex2_approx(x - ref);
                sv[e] = __float_as_uint(x + ev[e]);
                mx = fmaxf(mx, x + ev[e]);
            }
            ptx::tmem_st16(a.s_addr + 16 * g, sv);
        }
        ptx::tmem_wait_st();
        float alpha = 1.f;
        if (j == 0 || mx > m_w + kRescaleLog2) {
            alpha = j == 0 ? 0.f : ptx::ex2_approx(m_w - mx);
            m_w = mx;
        }
        if (j > 0 && __any_sync(0xffffffffu, alpha != 1.f)) {
#pragma unroll 1
            for (int go = 0; go < D / 16; ++go) {
                uint32_t ov[16];
                const uint32_t o_addr = a.o_addr + 16 * go;
                ptx::tmem_ld16(o_addr, ov);
                ptx::tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 16; ++e) ov[e] = __float_as_uint(__uint_as_float(ov[e]) * alpha);
                ptx::tmem_st16(o_addr, ov);
            }
        }
        const float neg = kPShift - (m_w == -INFINITY ? 0.f : m_w);
#pragma unroll 1
        for (int g = 0; g < 4; ++g) {  // the weights over columns that have been read
            uint32_t sv[32], pk[16];
            ptx::tmem_ld32(a.s_addr + 32 * g, sv);
            ptx::tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 16; ++e)
                pk[e] = pack_f16x2(ptx::ex2_approx(__uint_as_float(sv[2 * e]) + neg),
                                   ptx::ex2_approx(__uint_as_float(sv[2 * e + 1]) + neg));
            ptx::tmem_st16(a.s_addr + 16 * g, pk);
            if (g & 1) {
                ptx::tmem_wait_st();
                ptx::tc_fence_before();
                ptx::mbar_arrive(a.pfull + 8 * (g >> 1));
            }
        }
    }
    return make_float4(m, l, m_w, ok ? 1.f : 0.f);
}

template <int D, bool CACHE>
__global__ void __launch_bounds__(Cfg<D, CACHE>::THREADS, 1) skiparse_attn_frames_kernel(const FramesFwdParams p) {
    using C = Cfg<D, CACHE>;
    int pair, head, seq;
    if (!CACHE) {
        p.order.get(blockIdx.x, p.g.heads, pair, seq, head);
        pair = p.npairs - 1 - pair;
    }
    // cache: this CTA's number among those of the items that are cut, negative for a whole item
    const int over = CACHE ? static_cast<int>(blockIdx.x) - static_cast<int>(p.plan.whole) : -1;
    const int splits = over >= 0 ? p.plan.splits : 1;
    if (CACHE) {
        const int item = blockIdx.x - (over >= 0 ? over - p.dSplits.div(over) : 0);
        seq = p.dPairs.div(item);
        pair = p.npairs - 1 - (item - seq * p.npairs);
        head = seq;
        seq = p.dHeads.div(seq);
        head -= seq * p.g.heads;
    }
    ClassView cls;
    cls.init(p.g, seq);
    const int nF = cls.nF;
    const FastDiv dF = cls.dF;
    const int n_q = p.g.T * nF;
    const int q_first = pair * (p.halves ? kBM : 2 * kBM);
    if (q_first >= n_q) return;  // uniform over the CTA, before any shared state
    // both tiles are the same 128 queries, each over half of the key tiles; so is a class's rest
    const bool halves = p.halves || n_q - q_first <= kBM;
    int start = 0;
    if (CACHE) {
        start = p.cache.start[cls.b];
        if (start < 0 || start > kMaxStart) return;  // a sequence without new frames
    }
    FrameRing ring;
    ring.init(start + p.g.T, CACHE ? p.cache.cap : p.g.T);

    extern __shared__ __align__(1024) uint8_t smem_raw[];
    const uint32_t raw_base = ptx::smem_u32(smem_raw);
    const uint32_t pad = (1024u - (raw_base & 1023u)) & 1023u;
    if (pad + C::SMEM_USED > static_cast<uint32_t>(C::SMEM_BYTES)) {
        // the dynamic shared memory is not aligned well enough for this layout (uniform over the
        // CTA, before any shared state): report it instead of running out of bounds
        if (threadIdx.x == 0) atomicExch(p.status, kErrLaunch);
        return;
    }
    uint8_t* smem = smem_raw + pad;
    const uint32_t sbase = raw_base + pad;
    auto bar = [&](int i) -> uint32_t { return sbase + C::OFF_BAR + 8u * i; };
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::OFF_TMEM_SLOT);
    volatile int* abort = reinterpret_cast<volatile int*>(smem + C::OFF_ABORT);
    float* tab = reinterpret_cast<float*>(smem + C::OFF_TAB);
    int* range = reinterpret_cast<int*>(smem + C::OFF_RANGE);
    int* refs = reinterpret_cast<int*>(smem + C::OFF_REF);

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const uint64_t lim = p.wait_limit_ns;
    const int dmax = p.bias.D;
    const RowMap rows = cls.rows(p.g, head);

    // bf16: the frames of this CTA's queries, and whether the bias comes with the scores
    const int q_frame = dF.div(q_first);
    const int q_frames = dF.div(min(q_first + (halves ? kBM : 2 * kBM), n_q) - 1) - q_frame + 1;
    const bool cols = !CACHE && !p.halves && nF <= 8 * D && q_frames <= BiasCols::FRAMES;

    if (threadIdx.x == 0) {
        ptx::mbar_init(bar(C::B_Q), 64);
        for (int s = 0; s < C::KST; ++s) {
            ptx::mbar_init(bar(C::B_KFULL + s), C::FULL_COUNT + (cols ? 2 : 0));
            ptx::mbar_init(bar(C::B_KEMPTY + s), 1);
        }
        for (int s = 0; s < C::VST; ++s) {
            ptx::mbar_init(bar(C::B_VFULL + s), C::FULL_COUNT);
            ptx::mbar_init(bar(C::B_VEMPTY + s), 1);
        }
        for (int i = 0; i < 2; ++i) {
            ptx::mbar_init(bar(C::B_SFULL + i), 1);
            for (int h = 0; h < kPParts; ++h) ptx::mbar_init(bar(C::B_PFULL + kPParts * i + h), kBM);
        }
        ptx::mbar_init(bar(C::B_OFULL), 1);
        ptx::mbar_init(bar(C::B_DRAIN), 1);
        ptx::mbar_init(bar(C::B_QF16), 2 * kBM);
        *abort = 0;
        refs[0] = refs[1] = 0;
        refs[2] = refs[3] = 255;
        range[0] = dmax + 1;
        range[1] = -dmax - 1;
        ptx::fence_mbar_init();
    }
    if (warp == C::MMA_WARP) {
        ptx::tmem_alloc(ptx::smem_u32(tmem_slot), C::NCOLS);
        ptx::tmem_relinquish();
    }
    // Q starts to travel before the barriers stand; its copies arrive on theirs below
    const bool q_producer = warp == kProdWarp0 || warp == kProdWarp0 + 1;
    if (q_producer) {
        const int pw = warp - kProdWarp0;
        load_tile<D>(sbase + C::OFF_Q, p.q, rows, q_first, n_q, pw, lane, p.nrows, p.status);
        load_tile<D>(sbase + C::OFF_Q + C::TILE_BYTES, p.q, rows, halves ? q_first : q_first + kBM, n_q, pw, lane, p.nrows,
                     p.status);
    }
    // the bias by distance, and the first and last distance that is visible
    int dlo, dhi;
    fill_bias(tab, p.bias, p.g.heads, head, C::THREADS, dlo, dhi);
    if (!CACHE && cols) {
        if (threadIdx.x < 2 * kBM) {
            const int t = threadIdx.x / kBM, r = threadIdx.x % kBM;
            BiasCols::store_query(sbase + C::OFF_QB + t * BiasCols::TILE_BYTES, r,
                                  dF.div(min(q_first + (halves ? 0 : t * kBM) + r, n_q - 1)) - q_frame);
            fence_proxy_async();
        }
    }
    ptx::tc_fence_before();
    __syncthreads();
    if (!CACHE && cols)
        for (int i = threadIdx.x; i < 2 * dmax + BiasCols::FRAMES; i += C::THREADS)
            BiasCols::make_row(sbase + C::OFF_ROWS + i * BiasCols::ROW, tab, i - dmax - BiasCols::FRAMES + 1, dmax, p.scale_log2);
    dlo = __reduce_min_sync(0xffffffffu, dlo);
    dhi = __reduce_max_sync(0xffffffffu, dhi);
    if (lane == 0 && dlo <= dhi) {
        atomicMin(&range[0], dlo);
        atomicMax(&range[1], dhi);
    }
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    dlo = range[0];
    dhi = range[1];
    int f_lo, f_hi;  // frames that some row of this CTA can see
    ring.visible(start + dF.div(q_first), start + dF.div(min(q_first + (halves ? kBM : 2 * kBM), n_q) - 1), dlo, dhi, dmax, f_lo, f_hi);
    const int nkv_all = f_hi >= f_lo ? ((f_hi - f_lo + 1) * nF + kBN - 1) / kBN : 0;
    const int per_split = (nkv_all + splits - 1) / splits;
    const int jend = (f_hi + 1) * nF;                          // end of the visible keys
    const int first_tile = over >= 0 ? (over - p.dSplits.div(over) * splits) * per_split : 0;
    const int jbeg = f_lo * nF + first_tile * kBN;             // this CTA's first key
    const int nkv = max(0, min(per_split, nkv_all - first_tile));
    // cache: the largest and smallest scales among the keys read. Codes enter the tensor core as f16
    // values code * 2^(e - ref), so that one power of two for K and one for V remain to be applied, or
    // (wide) as they are.
    const long long sh = static_cast<long long>(seq) * p.g.heads + head;
    const uint8_t* k_scales = CACHE ? p.cache.ks + sh * p.cache.cap * p.cache.NBk : nullptr;
    const uint8_t* v_scales = CACHE ? p.cache.vs + sh * p.cache.cap * p.cache.NBk : nullptr;
    if (CACHE && nkv > 0) {
        const int s_lo = dF.div(jbeg), s_hi = dF.div(min(jbeg + nkv * kBN, jend) - 1);
        const int used = (nF + kCacheBlock - 1) / kCacheBlock, count = (s_hi - s_lo + 1) * used;
        int kr = 0, vr = 0, kl = 255, vl = 255;
        for (int i = threadIdx.x; i < count; i += C::THREADS) {
            const long long at = static_cast<long long>(s_lo + i / used) * p.cache.NBk + i % used;
            const int kb = __ldg(k_scales + at), vb = __ldg(v_scales + at);
            kr = max(kr, kb == 255 ? 0 : kb);
            vr = max(vr, vb == 255 ? 0 : vb);
            kl = min(kl, kb);
            vl = min(vl, vb);
        }
        kr = __reduce_max_sync(0xffffffffu, kr);
        vr = __reduce_max_sync(0xffffffffu, vr);
        kl = __reduce_min_sync(0xffffffffu, kl);
        vl = __reduce_min_sync(0xffffffffu, vl);
        if (lane == 0) {
            atomicMax(&refs[0], kr);
            atomicMax(&refs[1], vr);
            atomicMin(&refs[2], kl);
            atomicMin(&refs[3], vl);
        }
        __syncthreads();
    }
    const bool wide = CACHE && nkv > 0 && (refs[0] - refs[2] > kWideK || refs[1] - refs[3] > kWideV);

    if (CACHE) {
        // 512 threads start with 128 registers each; the softmax needs 168: 2 * 168 + 2 * 88 = 4 * 128
        if (warp < kProdWarp0)
            asm volatile("setmaxnreg.inc.sync.aligned.u32 168;");
        else
            asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
    }
    if (warp >= kProdWarp0) {
        if (warp < C::MMA_WARP) {
            // ------------------------------------------------------------------ producers
            const bool of_v = warp >= 12;                       // cache: K by warps 8-10, V by 12-14
            const int pw = warp - (of_v ? 12 : kProdWarp0);
            const int fault_skip = (p.fault == 1 && pw == 0 && lane == 0);
            bool ok = true;
            auto wait_empty = [&](bool is_v, int j) {  // the slot of key step j is free
                const int nst = is_v ? C::VST : C::KST;
                if (j < nst) return true;
                int w_ok = 1;
                if (lane == 0)
                    w_ok = ptx::mbar_wait(bar((is_v ? C::B_VEMPTY : C::B_KEMPTY) + j % nst), ((j / nst) - 1) & 1, abort, lim);
                return __shfl_sync(0xffffffffu, w_ok, 0) != 0;
            };
            if (q_producer) cp_async_arrive_noinc(bar(C::B_Q));
            if constexpr (CACHE) {
                static_assert(C::KST == C::VST, "one slot index for both rings");
                CacheTile<D> t;
                t.init((of_v ? p.cache.v : p.cache.k) + sh * p.cache.cap * p.cache.F * D, of_v ? v_scales : k_scales,
                       sbase + C::OFF_STAGE + (of_v ? CacheTile<D>::STAGE_BYTES : 0), pw, lane);
                const int ref = refs[of_v];
                const uint32_t slots = sbase + (of_v ? C::OFF_V : C::OFF_K);
                const int steps = pw < 3 ? nkv : 0;
                if (steps > 0) t.fetch(jbeg, jend, dF, nF, p.cache, p.status);
                for (int j = 0; j < steps; ++j) {
                    cp_async_wait<0>();
                    const bool one = t.all_ref(ref) || wide;
                    if (!(ok = wait_empty(of_v, j))) break;
                    const uint32_t dst = slots + (j % C::KST) * C::TILE_BYTES;
                    if (one)
                        t.template expand<false>(dst);
                    else
                        t.template expand<true>(dst);
                    fence_proxy_async();  // these stores, for the tensor core
                    __syncwarp();
                    // test hook: one warp never signals the first K tile
                    if (lane == 0 && !(fault_skip && !of_v && j == 0))
                        ptx::mbar_arrive(bar((of_v ? C::B_VFULL : C::B_KFULL) + j % C::KST));
                    if (j + 1 < steps) t.fetch(jbeg + (j + 1) * kBN, jend, dF, nF, p.cache, p.status);
                }
            } else {
                TileRows kv{0, 0};  // token rows of key step j, shared by its K and V tiles
                for (int L = 0; L < 2 * nkv; ++L) {
                    const int j = L >> 1;
                    const bool is_v = L & 1;
                    if (!is_v) kv = tile_rows(rows, jbeg + j * kBN, jend, pw, lane, p.nrows, p.status);
                    if (!(ok = wait_empty(is_v, j))) break;
                    const int s = j % (is_v ? C::VST : C::KST);
                    load_tile_rows<D>(sbase + (is_v ? C::OFF_V : C::OFF_K) + s * C::TILE_BYTES, is_v ? p.v : p.k, kv, pw, lane);
                    if (cols && !is_v) {
#pragma unroll
                        for (int half = 0; half < 2; ++half) {
                            const int r = 64 * pw + 32 * half + lane;
                            BiasCols::store_key(sbase + C::OFF_KB + s * BiasCols::TILE_BYTES, r, sbase + C::OFF_ROWS,
                                                q_frame - dF.div(min(jbeg + j * kBN + r, jend - 1)), dmax);
                        }
                        fence_proxy_async();  // these stores, for the tensor core
                        __syncwarp();
                        if (lane == 0) ptx::mbar_arrive(bar(C::B_KFULL + s));
                    }
                    // test hook: one thread never signals the first K tile
                    if (!(fault_skip && L == 0)) cp_async_arrive_noinc(bar((is_v ? C::B_VFULL : C::B_KFULL) + s));
                }
            }
            cp_async_commit();
            cp_async_wait<0>();  // no copy of this thread outlives it
            if (!ok) record_abort(abort, p.status);
        } else {
            // ------------------------------------------------------------------ MMA issuer
            if (lane == 0 && nkv > 0) {
                constexpr uint32_t bf16_s = ptx::idesc_bf16_f32(kBM, kBN, false), bf16_o = ptx::idesc_bf16_f32(kBM, D, true);
                constexpr uint32_t idesc_s = CACHE ? f16_operands(bf16_s) : bf16_s;
                constexpr uint32_t idesc_o = CACHE ? f16_operands(bf16_o) : bf16_o;
                const uint32_t q0 = sbase + C::OFF_Q, q1 = q0 + C::TILE_BYTES;
                const uint64_t qd0 = ptx::smem_desc(q0, 16, 8 * C::SW, C::LAYOUT);
                const uint64_t qd1 = ptx::smem_desc(q1, 16, 8 * C::SW, C::LAYOUT);
                const uint64_t kd0 = ptx::smem_desc(sbase + C::OFF_K, 16, 8 * C::SW, C::LAYOUT);
                const uint64_t vd0 = ptx::smem_desc(sbase + C::OFF_V, C::BOX_BYTES, 8 * C::SW, C::LAYOUT);
                auto bias_desc = [&](int off) { return ptx::smem_desc(sbase + off, 16, 8 * BiasCols::ROW, BiasCols::LAYOUT); };
                auto issue_s = [&](int qt, int kslot, uint32_t d_tmem) {
                    const uint64_t qd = qt ? qd1 : qd0;
                    const uint64_t kd = kd0 + ((kslot * C::TILE_BYTES) >> 4);
#pragma unroll
                    for (int kk = 0; kk < C::KSTEPS; ++kk) {
                        const uint32_t off = C::kstep_off(kk) >> 4;
                        ptx::mma_ss(d_tmem, qd + off, kd + off, idesc_s, kk > 0 ? 1u : 0u);
                    }
                    if (!CACHE && cols) {
                        ptx::mma_ss(d_tmem, bias_desc(C::OFF_QB + qt * BiasCols::TILE_BYTES),
                                    bias_desc(C::OFF_KB + kslot * BiasCols::TILE_BYTES), idesc_s, 1u);
                    }
                };
                auto issue_o = [&](int qt, int vslot, bool acc, int phase) -> bool {
                    const uint32_t p_tmem = tmem + (qt ? C::COL_S1 : C::COL_S0);
                    const uint32_t d_tmem = tmem + (qt ? C::COL_O1 : C::COL_O0);
                    const uint64_t vd = vd0 + ((vslot * C::TILE_BYTES) >> 4);
                    constexpr int KPP = kBN / 16 / kPParts;  // K-steps per part
                    for (int h = 0; h < kPParts; ++h) {
                        if (!ptx::mbar_wait(bar(C::B_PFULL + kPParts * qt + h), phase, abort, lim)) return false;
                        ptx::tc_fence_after();
#pragma unroll
                        for (int k4 = 0; k4 < KPP; ++k4) {
                            const int kk = h * KPP + k4;
                            ptx::mma_ts(d_tmem, p_tmem + kk * 8, vd + ((kk * 16 * C::SW) >> 4), idesc_o,
                                        (acc || kk > 0) ? 1u : 0u);
                        }
                    }
                    return true;
                };
                bool ok = ptx::mbar_wait(bar(CACHE ? C::B_QF16 : C::B_Q), 0, abort, lim) &&
                          ptx::mbar_wait(bar(C::B_KFULL + 0), 0, abort, lim);
                if (ok) {
                    fence_proxy_async();  // cp.async data observed through the barriers, for the MMA
                    ptx::tc_fence_after();
                    issue_s(0, 0, tmem + C::COL_S0);
                    ptx::mma_commit(bar(C::B_SFULL + 0));
                }
                if (halves) {
                    // query tile qt works on the key tiles 2 i + qt, each tile's slots released by its
                    // one reader
                    auto next_s = [&](int qt, int j) {  // S of key tile j, whose slot it releases
                        if (!ptx::mbar_wait(bar(C::B_KFULL + j % C::KST), (j / C::KST) & 1, abort, lim)) return false;
                        fence_proxy_async();
                        ptx::tc_fence_after();
                        issue_s(qt, j % C::KST, tmem + (qt ? C::COL_S1 : C::COL_S0));
                        ptx::mma_commit(bar(C::B_SFULL + qt));
                        ptx::mma_commit(bar(C::B_KEMPTY + j % C::KST));
                        return true;
                    };
                    if (ok) ptx::mma_commit(bar(C::B_KEMPTY + 0));
                    if (ok && nkv > 1) ok = next_s(1, 1);
                    for (int j = 0; ok && j < nkv; ++j) {
                        const int qt = j & 1, i = j >> 1, vs = j % C::VST;
                        ok = ptx::mbar_wait(bar(C::B_VFULL + vs), (j / C::VST) & 1, abort, lim);
                        if (ok) fence_proxy_async();
                        ok = ok && issue_o(qt, vs, i > 0, i & 1);
                        if (ok) ptx::mma_commit(bar(C::B_VEMPTY + vs));
                        if (ok && j + 2 < nkv) ok = next_s(qt, j + 2);
                    }
                } else {
                    if (ok) {
                        issue_s(1, 0, tmem + C::COL_S1);
                        ptx::mma_commit(bar(C::B_SFULL + 1));
                        ptx::mma_commit(bar(C::B_KEMPTY + 0));
                    }
                    for (int j = 0; ok && j < nkv; ++j) {
                        const int vs = j % C::VST;
                        const bool v_ok = ptx::mbar_wait(bar(C::B_VFULL + vs), (j / C::VST) & 1, abort, lim);
                        if (v_ok) fence_proxy_async();
                        if (!v_ok || !issue_o(0, vs, j > 0, j & 1)) {
                            ok = false;
                            break;
                        }
                        const bool more = j + 1 < nkv;
                        const int ks = (j + 1) % C::KST;
                        if (more) {
                            if (!ptx::mbar_wait(bar(C::B_KFULL + ks), ((j + 1) / C::KST) & 1, abort, lim)) {
                                ok = false;
                                break;
                            }
                            fence_proxy_async();
                            ptx::tc_fence_after();
                            issue_s(0, ks, tmem + C::COL_S0);
                            ptx::mma_commit(bar(C::B_SFULL + 0));
                        }
                        if (!issue_o(1, vs, j > 0, j & 1)) {
                            ok = false;
                            break;
                        }
                        ptx::mma_commit(bar(C::B_VEMPTY + vs));
                        if (more) {
                            issue_s(1, ks, tmem + C::COL_S1);
                            ptx::mma_commit(bar(C::B_SFULL + 1));
                            ptx::mma_commit(bar(C::B_KEMPTY + ks));
                        }
                    }
                }
                if (ok) {
                    ptx::mma_commit(bar(C::B_OFULL));
                } else {
                    record_abort(abort, p.status);
                }
                // every MMA issued by this thread must finish before TMEM is released
                ptx::mma_commit(bar(C::B_DRAIN));
                volatile int never = 0;
                ptx::mbar_wait(bar(C::B_DRAIN), 0, &never, lim);
            }
            __syncwarp();
        }
    } else {
        // ------------------------------------------------------------------ softmax (WG 0/1)
        const int qt = warp >> 2;                       // query tile 0 or 1
        const int row = threadIdx.x & 127;              // TMEM lane == row in the tile
        const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const uint32_t s_addr = tmem + lane_base + (qt ? C::COL_S1 : C::COL_S0);
        const uint32_t o_col = qt ? C::COL_O1 : C::COL_O0;
        const uint32_t sfull = bar(C::B_SFULL + qt);
        const int qi = q_first + (halves ? 0 : qt * kBM) + row;
        const int tq = start + dF.div(min(qi, n_q - 1));
        auto bias_of = [&](int f) { return tab[clamp_dist(tq - ring.time(f), dmax) + dmax]; };
        float m_run = -INFINITY, l_run = 0.f;  // in units of log2
        bool ok = true;
        float sl2 = p.scale_log2;
        if (CACHE && nkv > 0) {
            ok = __all_sync(0xffffffffu, ptx::mbar_wait(bar(C::B_Q), 0, abort, lim));
            if (ok) {
                const int up = q_row_to_f16<D>(sbase + C::OFF_Q + qt * C::TILE_BYTES, row);
                sl2 *= exp2_int(wide ? up : up + refs[0] - 127);
                fence_proxy_async();
                ptx::mbar_arrive(bar(C::B_QF16));
            }
        }
        // The row's results from its reference and sum of weights (in log2), and the power of two left in V
        auto finish = [&](bool ok, float m_run, float l_run, float v_scale) __attribute__((always_inline)) {
            if (ok && (nkv == 0 || __all_sync(0xffffffffu, ptx::mbar_wait(bar(C::B_OFULL), 0, abort, lim)))) {
                ptx::tc_fence_after();
                // a row without a visible key: 0, and -inf for its log-sum-exp
                if (!CACHE && m_run > BiasCols::FAR_LOG2) l_run = NAN;  // a bias that is not finite
                float inv_l = l_run == 0.f ? 0.f : v_scale / l_run;
                float l2 = l_run == 0.f ? -INFINITY : m_run + ptx::lg2_approx(l_run) - (CACHE ? kPShift : 0.f);
                float* other = reinterpret_cast<float*>(smem + C::OFF_K) + row;  // [d][128], over the finished K ring
                float join = 0.f;  // weight of the other half's result
                if (halves && nkv > 1) {
                    // the second half's result and log-sum-exp go through shared memory to the first
                    if (qt == 1) {
#pragma unroll
                        for (int g = 0; g < D / 32; ++g) {
                            uint32_t ov[32];
                            ptx::tmem_ld32(tmem + lane_base + o_col + 32 * g, ov);
                            ptx::tmem_wait_ld();
#pragma unroll
                            for (int e = 0; e < 32; ++e) other[(32 * g + e) * kBM] = __uint_as_float(ov[e]) * inv_l;
                        }
                        tab[row] = l2;  // the softmax is done with the bias
                    }
                    asm volatile("bar.sync 1, 256;" ::: "memory");
                    const float l2b = tab[row], top = fmaxf(l2, l2b) == -INFINITY ? 0.f : fmaxf(l2, l2b);
                    const float wa = ptx::ex2_approx(l2 - top), wb = ptx::ex2_approx(l2b - top), sum = wa + wb;
                    inv_l *= sum == 0.f ? 0.f : wa / sum;
                    join = sum == 0.f ? 0.f : wb / sum;
                    l2 = sum == 0.f ? -INFINITY : top + ptx::lg2_approx(sum);
                }
                const bool real = qi < n_q && !(halves && qt == 1) && row_ok(rows(qi), p.nrows, p.status);
                const size_t grow = real ? static_cast<size_t>(rows(qi)) : 0;
                const bool partial = CACHE && splits > 1;
                size_t part = 0;  // its place
                if (partial) {
                    const int cut = p.dSplits.div(over);
                    part = (static_cast<size_t>(cut) * (p.halves ? kBM : 2 * kBM) + (qi - q_first)) * splits + (over - cut * splits);
                }
                if (real) {
                    if (partial)
                        p.part_l[part] = l2;
                    else if (p.lse)
                        p.lse[grow] = l2 * 0.6931471805599453f;
                }
#pragma unroll
                for (int g = 0; g < D / 32; ++g) {
                    uint32_t ov[32];
                    if (nkv > 0) {
                        ptx::tmem_ld32(tmem + lane_base + o_col + 32 * g, ov);
                        ptx::tmem_wait_ld();
                    } else {
#pragma unroll
                        for (int e = 0; e < 32; ++e) ov[e] = 0u;
                    }
                    if (halves && nkv > 1) {
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            ov[e] = __float_as_uint(fmaf(__uint_as_float(ov[e]), inv_l, join * other[(32 * g + e) * kBM]));
                    }
                    const float inv = halves && nkv > 1 ? 1.f : inv_l;
                    if (partial) {
                        if (real) {
                            float4* dst = reinterpret_cast<float4*>(p.part_o + part * D + 32 * g);
#pragma unroll
                            for (int e = 0; e < 8; ++e)
                                dst[e] = make_float4(__uint_as_float(ov[4 * e]) * inv, __uint_as_float(ov[4 * e + 1]) * inv,
                                                     __uint_as_float(ov[4 * e + 2]) * inv, __uint_as_float(ov[4 * e + 3]) * inv);
                        }
                    } else {
                        auto store = [&](uint16_t* to, const uint32_t(&w)[16]) {
                            uint4* dst = reinterpret_cast<uint4*>(to + grow * D);
#pragma unroll
                            for (int v4 = 0; v4 < 4; ++v4)
                                dst[4 * g + v4] = make_uint4(w[4 * v4], w[4 * v4 + 1], w[4 * v4 + 2], w[4 * v4 + 3]);
                        };
                        uint32_t pkd[16];
#pragma unroll
                        for (int e = 0; e < 16; ++e)
                            pkd[e] = ptx::pack_bf16x2(__uint_as_float(ov[2 * e]) * inv, __uint_as_float(ov[2 * e + 1]) * inv);
                        if (real) store(p.out, pkd);
                        if (!CACHE && p.out_lo) {  // what the rounding took: exact in fp32, rounded once
#pragma unroll
                            for (int e = 0; e < 16; ++e)
                                pkd[e] = ptx::pack_bf16x2(
                                    fmaf(__uint_as_float(ov[2 * e]), inv, -__uint_as_float(pkd[e] << 16)),
                                    fmaf(__uint_as_float(ov[2 * e + 1]), inv, -__uint_as_float(pkd[e] & 0xffff0000u)));
                            if (real) store(p.out_lo, pkd);
                        }
                    }
                }
            } else {
                if (!*abort) record_abort(abort, p.status);
                if (halves && nkv > 1) asm volatile("bar.arrive 1, 256;" ::: "memory");  // for warps that saw no failure
            }
        };
        const int tiles = halves ? (nkv - qt + 1) / 2 : nkv;  // of this query tile
        if (CACHE && wide) {
            const WideArgs wa{jbeg, jend, nF, halves ? 2 * kBN : kBN, halves ? qt * kBN : 0, ok ? tiles : 0,
                              tq, dmax, p.cache.NBk, s_addr, tmem + lane_base + o_col,
                              sfull, bar(C::B_PFULL + kPParts * qt), sl2, tab, k_scales, v_scales, dF, ring, abort, lim};
            const float4 r = wide_softmax<D>(wa);
            finish(ok && r.w != 0.f, r.x, r.y * 128.f, ptx::ex2_approx(r.z - r.x));  // l * 2^kPShift, as sums of stored P
        } else {
            int done = 0;
            if (!__any_sync(0xffffffffu, qi < n_q)) {
                // All 32 rows of the warp lie past the class's end: it leaves their S as it is (rows of P and
                // O do not mix) and only keeps the barriers going.
                for (; ok && done < tiles; ++done) {
                    ok = __all_sync(0xffffffffu, ptx::mbar_wait(sfull, done & 1, abort, lim));
                    for (int h = 0; ok && h < kPParts; ++h) ptx::mbar_arrive(bar(C::B_PFULL + kPParts * qt + h));
                }
            }
            for (int j = done; ok && j < tiles; ++j) {
                // Every wait of a softmax warp is made uniform over the warp (a lane can see the abort
                // flag while another sees the phase complete): the tcgen05.ld/st below are
                // .sync.aligned and need all 32 lanes.
                const int j0 = jbeg + (halves ? 2 * j + qt : j) * kBN;
                const int f0 = dF.div(j0);
                const int border = (f0 + 1) * nF - j0;  // tile column where the next frame starts
                float off = !CACHE && cols ? 0.f : bias_of(f0), mul = sl2;  // scores are S * mul + off, in log2
                if (!__all_sync(0xffffffffu, ptx::mbar_wait(sfull, j & 1, abort, lim))) {
                    ok = false;
                    break;
                }
                ptx::tc_fence_after();
                // Whether a frame starts inside the tile, and with another bias (for some row of this warp; distances
                // that share a bucket are common): d = 64 and 32, 40 and 64 frames, 910 -> 859 and 682 -> 620 us. At
                // d = 128 the second question costs more than it saves (480p chunk 636 -> 698 us).
                bool mixed = border < kBN && (CACHE ? p.bias.table != nullptr : !cols);
                if (CACHE && D < 128 && mixed && border + nF >= kBN) mixed = __any_sync(0xffffffffu, bias_of(f0 + 1) != off);
                if (mixed) {
                    // S becomes S * scale + bias in place, some columns at a
                    // time, before the softmax below reads the row. (Biases per 32 columns carried through
                    // the softmax instead cost the tiles without a border 18 %.)
                    if (nF >= 32) {  // at most one border in 32 columns
                        int f = f0, next = border;  // column of this chunk where the next frame starts
#pragma unroll 1
                        for (int g = 0; g < 4; ++g) {
                            uint32_t sv[32];
                            ptx::tmem_ld32(s_addr + 32 * g, sv);
                            ptx::tmem_wait_ld();
                            if (next >= 32) {
#pragma unroll
                                for (int e = 0; e < 32; e += 2) {  // two columns per instruction
                                    const float2 y = __ffma2_rn(make_float2(__uint_as_float(sv[e]), __uint_as_float(sv[e + 1])),
                                                                make_float2(sl2, sl2), make_float2(off, off));
                                    sv[e] = __float_as_uint(y.x);
                                    sv[e + 1] = __float_as_uint(y.y);
                                }
                            } else {
                                const float o1 = bias_of(++f);
#pragma unroll
                                for (int e = 0; e < 32; ++e)
                                    sv[e] = __float_as_uint(fmaf(__uint_as_float(sv[e]), sl2, e < next ? off : o1));
                                off = o1;
                                next += nF;
                            }
                            next -= 32;
                            ptx::tmem_st16(s_addr + 32 * g, *reinterpret_cast<uint32_t(*)[16]>(&sv[0]));
                            ptx::tmem_st16(s_addr + 32 * g + 16, *reinterpret_cast<uint32_t(*)[16]>(&sv[16]));
                        }
                    } else {
                        // Frames of fewer tokens: a lookup per score (columns past the last frame are masked
                        // below). The width decides how the rest of this loop compiles: 16 columns make the
                        // bf16 form 6 % faster than 32 at 480p, 32 the cache form 7 % faster than 16 at 720p.
                        constexpr int WIDTH = CACHE ? 32 : 16;
#pragma unroll 1
                        for (int g = 0; g < kBN / WIDTH; ++g) {
                            const int jg = j0 + WIDTH * g;
                            uint32_t sv[WIDTH];
                            if constexpr (WIDTH == 32)
                                ptx::tmem_ld32(s_addr + WIDTH * g, sv);
                            else
                                ptx::tmem_ld16(s_addr + WIDTH * g, sv);
                            ptx::tmem_wait_ld();
#pragma unroll
                            for (int e = 0; e < WIDTH; ++e)
                                sv[e] = __float_as_uint(fmaf(__uint_as_float(sv[e]), sl2, bias_of(dF.div(jg + e))));
#pragma unroll
                            for (int w = 0; w < WIDTH; w += 16)
                                ptx::tmem_st16(s_addr + WIDTH * g + w, *reinterpret_cast<uint32_t(*)[16]>(&sv[w]));
                        }
                    }
                    ptx::tmem_wait_st();
                    off = 0.f;
                    mul = 1.f;
                }
                float sc[kBN];
                {
                    uint32_t sv[kBN];
#pragma unroll
                    for (int g = 0; g < 4; ++g)
                        ptx::tmem_ld32(s_addr + 32 * g, *reinterpret_cast<uint32_t(*)[32]>(&sv[32 * g]));
                    ptx::tmem_wait_ld();  // one wait for the whole 128-column row
#pragma unroll
                    for (int e = 0; e < kBN; ++e) sc[e] = __uint_as_float(sv[e]);
                }
                if (j0 + kBN > jend) {
                    const int valid = jend - j0;
#pragma unroll
                    for (int e = 0; e < kBN; ++e)
                        if (e >= valid) sc[e] = -INFINITY;
                }
                // row max with 3-input max instructions, four independent chains
                float mx0 = ptx::max3f(sc[0], sc[1], sc[2]), mx1 = ptx::max3f(sc[3], sc[4], sc[5]);
                float mx2 = ptx::max3f(sc[6], sc[7], sc[8]), mx3 = ptx::max3f(sc[9], sc[10], sc[11]);
#pragma unroll
                for (int e = 12; e + 8 <= kBN; e += 8) {
                    mx0 = ptx::max3f(mx0, sc[e], sc[e + 1]);
                    mx1 = ptx::max3f(mx1, sc[e + 2], sc[e + 3]);
                    mx2 = ptx::max3f(mx2, sc[e + 4], sc[e + 5]);
                    mx3 = ptx::max3f(mx3, sc[e + 6], sc[e + 7]);
                }
                static_assert((kBN - 12) % 8 == 4, "tail of the max chains");
                mx0 = ptx::max3f(mx0, sc[kBN - 4], sc[kBN - 3]);
                mx1 = ptx::max3f(mx1, sc[kBN - 2], sc[kBN - 1]);
                const float mx = fmaf(fmaxf(fmaxf(mx0, mx1), fmaxf(mx2, mx3)), mul, off);
                float alpha = 1.f;
                if (j == 0 || mx > m_run + kRescaleLog2) {  // m_run = -inf: O and l are zero, alpha 0 keeps them
                    alpha = (j == 0) ? 0.f : ptx::ex2_approx(m_run - mx);
                    m_run = mx;
                }
                // P = 2^(S*scale*log2(e) + bias - m), written as bf16 pairs over the first 64 columns of
                // S, in two halves released as they are stored. A row that has seen no key yet keeps
                // the reference 0, so that its -inf scores give 0.
                const float neg = off - (m_run < -BiasCols::FAR_LOG2 ? 0.f : m_run) + (CACHE ? kPShift : 0.f);
                float2 sum_a = make_float2(0.f, 0.f), sum_b = sum_a;  // four short addition chains
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                    uint32_t pk[16];
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        // two columns per instruction (packed f32x2)
                        const float2 x = __ffma2_rn(make_float2(sc[32 * g + 2 * e], sc[32 * g + 2 * e + 1]),
                                                    make_float2(mul, mul), make_float2(neg, neg));
                        const float p0 = ptx::ex2_approx(x.x);
                        const float p1 = ptx::ex2_approx(x.y);
                        if (CACHE) {  // packed sums: 3 % faster here, 1 % slower in the bf16 form
                            float2& sum = e & 1 ? sum_b : sum_a;
                            sum = __fadd2_rn(sum, make_float2(p0, p1));
                        } else if (e & 1) {
                            sum_b.x += p0;
                            sum_b.y += p1;
                        } else {
                            sum_a.x += p0;
                            sum_a.y += p1;
                        }
                        pk[e] = CACHE ? pack_f16x2(p0, p1) : ptx::pack_bf16x2(p0, p1);
                    }
                    ptx::tmem_st16(s_addr + 16 * g, pk);
                    if (g == 1 && j > 0 && __any_sync(0xffffffffu, alpha != 1.f)) {
                        // Rare: a row max grew by more than 2^8. This warp rescales its rows of O_qt
                        // before releasing the first half of P, i.e. before this tile's P*V
                        // accumulates into O_qt; O_qt was completed by the previous P*V (the commit
                        // behind this tile's S covers it).
#pragma unroll
                        for (int go = 0; go < D / 16; ++go) {
                            uint32_t ov[16];
                            const uint32_t o_addr = tmem + lane_base + o_col + 16 * go;
                            ptx::tmem_ld16(o_addr, ov);
                            ptx::tmem_wait_ld();
#pragma unroll
                            for (int e = 0; e < 16; ++e) ov[e] = __float_as_uint(__uint_as_float(ov[e]) * alpha);
                            ptx::tmem_st16(o_addr, ov);
                        }
                    }
                    if (g & 1) {
                        ptx::tmem_wait_st();
                        ptx::tc_fence_before();
                        ptx::mbar_arrive(bar(C::B_PFULL + kPParts * qt + (g >> 1)));
                    }
                }
                l_run = l_run * alpha + ((sum_a.x + sum_a.y) + (sum_b.x + sum_b.y));
            }
            finish(ok, m_run, l_run, CACHE && nkv > 0 ? exp2_int(refs[1] - 127) : 1.f);
        }
    }

    ptx::tc_fence_before();
    __syncthreads();
    if (warp == C::MMA_WARP) {
        ptx::tc_fence_after();
        ptx::tmem_dealloc(tmem, C::NCOLS);
    }
}

// Joins the partial results of a split call: out = sum_s w_s o_s / sum_s w_s with
// w_s = 2^(l_s - max l). One warp per query row.
template <int D>
__global__ void __launch_bounds__(256) skiparse_frames_join_kernel(const FramesFwdParams p) {
    const long long at = (static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x) >> 5;  // partial results' row
    const int lane = threadIdx.x & 31;
    if (at >= p.plan.part_rows) return;
    const int splits = p.plan.splits;
    long long row = at;
    int b;
    if (p.npairs == 0) {  // few-query form
        b = static_cast<int>(row / (static_cast<long long>(p.g.T) * p.g.H * p.g.W * p.g.heads));
    } else {
        const int per = p.halves ? kBM : 2 * kBM;
        const int item = static_cast<int>(p.plan.whole) + static_cast<int>(at / per);
        const int sh = p.dPairs.div(item), seq = p.dHeads.div(sh);
        const int qi = (p.npairs - 1 - (item - sh * p.npairs)) * per + static_cast<int>(at % per);
        ClassView cls;
        cls.init(p.g, seq);
        if (qi >= p.g.T * cls.nF) return;
        row = cls.rows(p.g, sh - seq * p.g.heads)(qi);
        b = cls.b;
    }
    const int start = p.cache.start[b];
    if (start < 0 || start > kMaxStart || !row_ok(row, p.nrows, p.status)) return;
    const float* l = p.part_l + at * splits;
    float m = -INFINITY;
    for (int s = lane; s < splits; s += 32) m = fmaxf(m, l[s]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    constexpr int PER = D / 32;
    float acc[PER] = {}, total = 0.f;
    m = m == -INFINITY ? 0.f : m;  // no key seen, or NaNs alone, which have to stay
    for (int s = 0; s < splits; ++s) {
        const float w = ptx::ex2_approx(l[s] - m);
        total += w;
        const float* o = p.part_o + (at * splits + s) * D + lane * PER;
#pragma unroll
        for (int e = 0; e < PER; ++e) acc[e] = fmaf(w, o[e], acc[e]);
    }
    const float inv = total == 0.f ? 0.f : 1.f / total;
#pragma unroll
    for (int e = 0; e < PER; ++e)
        p.out[row * D + lane * PER + e] = __bfloat16_as_ushort(__float2bfloat16_rn(acc[e] * inv));
    if (lane == 0 && p.lse) p.lse[row] = total == 0.f ? -INFINITY : (m + ptx::lg2_approx(total)) * 0.6931471805599453f;
}

int launch_frames_join(const FramesFwdParams& p, int d, cudaStream_t stream) {
    const unsigned blocks = static_cast<unsigned>((p.plan.part_rows + 7) / 8);
    switch (d) {
        case 32: skiparse_frames_join_kernel<32><<<blocks, 256, 0, stream>>>(p); break;
        case 64: skiparse_frames_join_kernel<64><<<blocks, 256, 0, stream>>>(p); break;
        default: skiparse_frames_join_kernel<128><<<blocks, 256, 0, stream>>>(p); break;
    }
    return static_cast<int>(cudaGetLastError());
}

template <int D, bool CACHE>
int launch_d(const FramesFwdParams& p, const Geometry& g, cudaStream_t stream) {
    using C = Cfg<D, CACHE>;
    // per device: the kernel's shared-memory attribute is set (host threads may race here;
    // setting it twice is harmless, the flag only has to be a race-free read)
    static std::atomic<int> attr_done_dev[64];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return static_cast<int>(e);
    if (dev < 0 || dev >= 64 || !attr_done_dev[dev].load(std::memory_order_acquire)) {
        e = cudaFuncSetAttribute(skiparse_attn_frames_kernel<D, CACHE>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 C::SMEM_BYTES);
        if (e != cudaSuccess) return static_cast<int>(e);
        if (CACHE) {  // the kernel's register split counts on what it was compiled with
            cudaFuncAttributes a;
            e = cudaFuncGetAttributes(&a, skiparse_attn_frames_kernel<D, CACHE>);
            if (e != cudaSuccess) return static_cast<int>(e);
            if (a.numRegs != 128) return static_cast<int>(cudaErrorInvalidConfiguration);
        }
        if (dev >= 0 && dev < 64) attr_done_dev[dev].store(1, std::memory_order_release);
    }
    const long long items = static_cast<long long>(p.npairs) * g.heads * g.B * g.Ph * g.Pw;
    const dim3 grid(static_cast<unsigned>(CACHE ? p.plan.whole + (items - p.plan.whole) * p.plan.splits : items));
    skiparse_attn_frames_kernel<D, CACHE><<<grid, C::THREADS, C::SMEM_BYTES, stream>>>(p);
    e = cudaGetLastError();
    if (e != cudaSuccess || !CACHE || p.plan.splits == 1) return static_cast<int>(e);
    return launch_frames_join(p, D, stream);
}

template <int D>
int launch_kind(const FramesFwdParams& p, const Geometry& g, cudaStream_t stream) {
    return p.cache.k ? launch_d<D, true>(p, g, stream) : launch_d<D, false>(p, g, stream);
}

}  // namespace

// Whether 128-query CTAs, whose two softmax groups share the keys, finish a call of n queries and
// `keys` keys a class earlier than 256-query CTAs: by waves of one CTA per SM (148) times key steps,
// with three steps' worth for a CTA's start and end. One query tile alone always goes that way.
// Larger calls keep to 256 queries unless it gains a tenth: there each key tile is loaded half as often.
bool frames_halves(const Geometry& g, long long n, long long keys) {
    if (n <= kBM) return true;
    const long long pairs = static_cast<long long>(g.heads) * g.B * g.Ph * g.Pw, steps = (keys + kBN - 1) / kBN;
    auto waves = [&](long long rows) { return ((n + rows - 1) / rows * pairs + 147) / 148; };
    // a step of two key tiles takes 1.5 times a step of one at d = 128, where the loads bound it
    return 10 * waves(kBM) * ((steps + 1) / 2 * (g.d == 128 ? 3 : 2) + 6) < 9 * waves(2 * kBM) * (2 * steps + 6);
}

// How a cache call is cut: the choice that ends first by waves of one CTA per SM (148) times key tiles
// (five steps' worth of them for a CTA's start and end), where the fp32 partial results cost a step per
// 5 MB, each part keeping at least four key tiles. Either every item is cut (96 items of 168 tiles took
// 0.46 ms, in three parts each 0.40), or those behind the last full wave (640 items of 151 tiles: 1.57 ms
// whole, 1.45 with the last 48 in three parts; 480 of 75: 0.73 and 0.65). The cache's capacity stands for its length, which only the device knows.
CachePlan cached_plan(const Geometry& g, int cap) {
    const long long n = static_cast<long long>(g.T) * max_class_tokens(g), keys = static_cast<long long>(cap) * max_class_tokens(g);
    const long long pairs = static_cast<long long>(g.heads) * g.B * g.Ph * g.Pw;
    if (cached_small(g)) return {0, cached_small_splits(g, cap), static_cast<long long>(g.B) * g.T * g.H * g.W * g.heads};
    const long long rows = frames_halves(g, n, keys) ? kBM : 2 * kBM, tiles = (keys + kBN - 1) / kBN;
    const long long items = (n + rows - 1) / rows * pairs, ends = rows == kBM ? 10 : 5;
    CachePlan best{items, 1, 0};
    long long least = -1;
    for (const long long whole : {items / 148 * 148, 0ll})
        for (long long s = 1; s <= 148 && (s == 1 || s * 4 <= tiles); ++s) {
            const long long cut = items - whole, part_rows = s > 1 ? cut * rows : 0;
            const long long cost = whole / 148 * (tiles + ends) + (cut * s + 147) / 148 * ((tiles + s - 1) / s + ends) +
                                   (s > 1 ? 2 + part_rows * s * g.d * 8 / 5000000 : 0);
            if (least >= 0 && cost >= least) continue;
            least = cost;
            best = {s > 1 ? whole : items, static_cast<int>(s), part_rows};
        }
    return best;
}

int launch_frames_fwd(FramesFwdParams p, const Geometry& g, void* stream) {
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    p.halves = frames_halves(g, static_cast<long long>(g.T) * max_class_tokens(g),
                             static_cast<long long>(p.cache.k ? p.cache.cap : g.T) * max_class_tokens(g));
    if (p.cache.k && cached_small(g)) {
        const int e = launch_cached_small(p, g, stream);
        return e || p.plan.splits == 1 ? e : launch_frames_join(p, g.d, st);
    }
    const long long n_max = static_cast<long long>(g.T) * max_class_tokens(g);
    const int rows = p.halves ? kBM : 2 * kBM;
    p.npairs = static_cast<int>((n_max + rows - 1) / rows);
    p.dPairs.init(p.npairs);
    p.dHeads.init(g.heads);
    p.dSplits.init(p.plan.splits);
    p.order.init(g.heads * g.B * g.Ph * g.Pw, p.npairs, g.heads);
    switch (g.d) {
        case 32: return launch_kind<32>(p, g, st);
        case 64: return launch_kind<64>(p, g, st);
        case 128: return launch_kind<128>(p, g, st);
        default: return static_cast<int>(cudaErrorInvalidValue);
    }
}

}  // namespace skiparse
