// frames_internal.cuh -- parameters and launchers of the frame-aware attention operators: class
// attention with a learned bias by frame distance (forward and backward), the 8-bit frame cache
// and attention over it. Geometry, class rule and row maps are those of skiparse_internal.cuh.
#pragma once

#include <cstdint>

#include "attn_common.cuh"
#include "skiparse_internal.cuh"

namespace skiparse {

// The bias of a pair of tokens depends on the distance of their frames, u = clamp(t_q - t_k,
// -D, D): table[buckets[u + D]][head], the pair being masked where the bucket lies outside
// [0, NB) or the entry is at or below -65504 (so -inf, the lowest values of fp16, bf16 and fp32 and the
// usual -1e9 mask). A row that sees such entries only would, if they counted, have scores and a
// log-sum-exp whose fp32 rounding is too coarse for the backward pass to find the weights again and for
// weights in f16 to keep in range: half a step, in log2, is 2^-8 at 65504 and 64 at 1e9.
constexpr int kMaxDist = 255;                     // largest D
constexpr int kMaxDistEntries = 2 * kMaxDist + 1;
constexpr float kBiasMasked = -65504.f;  // between bf16's -65280 and -65536

struct FrameBias {
    const uint16_t* table;  // bf16 (NB, heads); nullptr: no bias and no mask
    const int* buckets;     // (2D+1)
    int D, NB;
};

// The dimensions of a call, filled from Geometry, and the divisions that the kernels need: by the
// rows, columns, tokens per frame and 32-token chunks per frame of each class, and by the class counts. (Their constants take a
// thread a 64-bit division each; in small calls those were a good part of the kernel's time.)
struct FrameGeom {
    int T, H, W, heads, Ph, Pw, mode;
    int Rc[kMaxAxisClasses], Sc[kMaxAxisClasses];
    FastDiv dR[kMaxAxisClasses], dS[kMaxAxisClasses], dF[kMaxAxisClasses], dC[kMaxAxisClasses], dPh, dPw, dClasses;
};

// The e4m3 frame cache of one layer: codes (B*classes, heads, cap, F, d), F the padded tokens
// of a class in one frame, of which class c uses the first Rc*Sc; scales (e8m0 bytes)
// (B*classes, heads, cap, NBk), one for every kCacheBlock tokens. Frame t lies in slot t % cap.
constexpr int kCacheBlock = 64;
constexpr int kScaleLow = 17;      // scale byte of 2^-110, the smallest a writer stores
constexpr int kMaxStart = 1 << 30; // frame numbers beyond this skip a sequence, as negative ones do

struct CacheView {
    uint8_t* k;
    uint8_t* v;
    uint8_t* ks;
    uint8_t* vs;
    const int* start;  // (B): frame number of the call's first frame; < 0: sequence skipped
    int cap, F, NBk;
};

// The order in which CTAs take the tiles of a call's units (one class and head of one batch element each).
// Under a mask the tiles of a unit differ in work, the first by most. Units are taken one after another,
// which keeps what their tiles share in L2, but for the last, of about kLastTiles tiles: of those first
// every unit's first tile, then every second one, and so on, so that no long tile starts late and leaves
// the other SMs idle. 9 causal frames of 27 x 40, P = 3, d = 64, 54 units: forward 47 -> 42 us, dQ 52 -> 47, dK and
// dV 70 -> 63; 480p frame-causal, 48 units: forward 880 -> 841 us; without a mask no change at 480p, where
// all units in groups that fit L2 cost 3 %.
constexpr int kLastTiles = 2 * 148;  // two waves of one CTA per SM
struct TileOrder {
    int units, tiles, last;  // last: units of the second kind
    FastDiv dTiles, dLast, dHeads;
    void init(int units_, int tiles_, int heads) {
        units = units_;
        tiles = tiles_;
        last = (kLastTiles + tiles - 1) / tiles;
        last = last < units ? last : units;
        dTiles.init(tiles);
        dLast.init(last);
        dHeads.init(heads);
    }
    // The tile, class (seq) and head of CTA `at` of the units * tiles.
    __device__ __forceinline__ void get(int at, int heads, int& tile, int& seq, int& head) const {
        int unit = dTiles.div(at);
        tile = at - unit * tiles;
        if (unit >= units - last) {
            at -= (units - last) * tiles;
            tile = dLast.div(at);
            unit = units - last + at - tile * last;
        }
        seq = dHeads.div(unit);
        head = unit - seq * heads;
    }
};

// How a cache call is cut into CTAs. An item is a tile of queries of one class and head. The first
// `whole` items are a CTA each; of the others, the keys are cut into `splits` parts, a CTA each, whose
// results a second kernel joins.
struct CachePlan {
    long long whole;
    int splits;
    long long part_rows;  // rows with partial results: those of the items that are cut; every row of the call, in
                          // its order, in the few-query form (which has no whole items)
};

// Forward: bf16 keys and values (k, v), or the cache (cache.k != nullptr).
struct FramesFwdParams {
    const uint16_t* q;
    const uint16_t* k;
    const uint16_t* v;
    uint16_t* out;
    uint16_t* out_lo; // optional: out's rounding residual (bf16 keys only)
    float* lse;       // optional
    float* part_o;    // splits > 1: (part_rows, splits, d) fp32 normalised partial outputs
    float* part_l;    // splits > 1: (part_rows, splits) fp32 partial log2-sum-exp
    int* status;
    FrameGeom g;
    FrameBias bias;
    CacheView cache;
    CachePlan plan;   // cache only
    int halves;       // 128-query CTAs; chosen by launch_frames_fwd
    int npairs;       // query tiles of the longest class; this and what follows: set by launch_frames_fwd
    FastDiv dPairs, dHeads, dSplits;
    TileOrder order;  // bf16 keys
    float scale_log2;
    unsigned long long wait_limit_ns;
    int fault;
    long long nrows;  // (token, head) rows of q: the debug bound
};

struct FramesBwdParams {
    const uint16_t* q;
    const uint16_t* k;
    const uint16_t* v;
    const uint16_t* out;
    const uint16_t* out_lo;  // optional
    const uint16_t* dout;
    const float* lse;
    float* delta;      // workspace (rows): D = rowsum(dO o (O + O_lo)), corrected, by the dQ kernel
    float* nlse2;      // workspace (rows): -lse * log2(e), kNoKeys for a row without a visible key, by the dQ kernel
    float* part;       // workspace (heads, ND, seqs, tiles): sums of dS by frame distance
    uint16_t* dtable;  // bf16 (NB, heads)
    uint16_t* dq;
    uint16_t* dk;
    uint16_t* dv;
    int* status;
    FrameGeom g;
    FrameBias bias;
    int Dn, ND;        // distances that occur: [-Dn, Dn], Dn = min(D, T-1), ND = 2 Dn + 1
    int seqs, tiles;   // B * classes; 128-key tiles of the longest class
    TileOrder order;
    float scale_log2, scale;
    unsigned long long wait_limit_ns;
    long long nrows;
    int fault;
};
// What stands for the -lse of a row without a visible key, whose lse is -inf: its masked scores of -inf
// still give exp2(-inf) = 0.
constexpr float kNoKeys = 1e30f;

struct AppendParams {
    const uint16_t* k;
    const uint16_t* v;
    int* status;
    FrameGeom g;       // g.T: new frames
    CacheView cache;
    int nblk;          // blocks of kCacheBlock tokens of the largest class
    long long nrows;
};

// Launchers. They return the cudaError_t as int.
int launch_frames_fwd(FramesFwdParams p, const Geometry& g, void* stream);
int launch_frames_bwd(const FramesBwdParams& p, const Geometry& g, void* stream);
int launch_cache_append(const AppendParams& p, const Geometry& g, int d, void* stream);
// Attention of few queries over the cache: whether a call's classes are small enough for it, its
// splits, and its launch (without the joining of the splits).
bool cached_small(const Geometry& g);
int cached_small_splits(const Geometry& g, int cap);
int launch_cached_small(const FramesFwdParams& p, const Geometry& g, void* stream);
// The plan that launch_frames_fwd should be given for a cache call of these sizes (splits 1: no
// workspace is needed).
CachePlan cached_plan(const Geometry& g, int cap);

inline int max_class_tokens(const Geometry& g) {  // tokens of one frame in the largest class
    int r = 0, s = 0;
    for (int c = 0; c < kMaxAxisClasses; ++c) {
        r = g.Rc[c] > r ? g.Rc[c] : r;
        s = g.Sc[c] > s ? g.Sc[c] : s;
    }
    return r * s;
}

inline void fill_frame_geom(FrameGeom& f, const Geometry& g) {
    f.T = g.T; f.H = g.H; f.W = g.W; f.heads = g.heads; f.Ph = g.Ph; f.Pw = g.Pw; f.mode = g.mode;
    for (int c = 0; c < g.Ph; ++c) {
        f.Rc[c] = g.Rc[c];
        f.dR[c].init(g.Rc[c]);
    }
    for (int c = 0; c < g.Pw; ++c) {
        f.Sc[c] = g.Sc[c];
        f.dS[c].init(g.Sc[c]);
    }
    for (int c = 0; c < g.Ph * g.Pw; ++c) {
        const int nF = g.Rc[c / g.Pw] * g.Sc[c % g.Pw];
        f.dF[c].init(nF);
        f.dC[c].init((nF + 31) / 32);
    }
    f.dPh.init(g.Ph);
    f.dPw.init(g.Pw);
    f.dClasses.init(g.Ph * g.Pw);
}

// One (batch, class, head) of a call: its sizes and row map.
struct ClassView {
    int b, c, ci, cj, Rc, Sc, nF;  // nF: tokens per frame
    FastDiv dF;
    __device__ __forceinline__ void init(const FrameGeom& g, int seq) {
        b = g.dClasses.div(seq);
        c = seq - b * g.Ph * g.Pw;
        ci = g.dPw.div(c);
        cj = c - ci * g.Pw;
        Rc = g.Rc[ci];
        Sc = g.Sc[cj];
        nF = Rc * Sc;
        dF = g.dF[c];
    }
    __device__ __forceinline__ RowMap rows(const FrameGeom& g, int head) const {
        RowMap r;
        r.T = g.T; r.H = g.H; r.W = g.W; r.heads = g.heads; r.Ph = g.Ph; r.Pw = g.Pw; r.mode = g.mode;
        r.ci = ci; r.cj = cj; r.Rc = Rc; r.Sc = Sc; r.b = b; r.head = head;
        r.dSc = g.dS[cj]; r.dRc = g.dR[ci]; r.dPh = g.dPh; r.dPw = g.dPw;
        return r;
    }
};

}  // namespace skiparse
