// frames_api.cu -- entry points of the frame-aware operators (include/skiparse.h): class attention
// with a learned bias by frame distance, the e4m3 frame cache and attention over it. Checks the
// arguments, lays out the caller's workspace and launches.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <initializer_list>

#include "../../include/skiparse.h"
#include "api_internal.cuh"
#include "frames_internal.cuh"

namespace {

using skiparse::Geometry;
namespace api = skiparse::api;

bool aligned(const void* p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }

struct Span {
    const void* p;
    size_t bytes;
};

// Whether an output range meets an input range or another output range (null spans are absent).
bool any_overlap(std::initializer_list<Span> outs, std::initializer_list<Span> ins) {
    for (const Span* a = outs.begin(); a != outs.end(); ++a) {
        if (!a->p || !a->bytes) continue;
        for (const Span& b : ins)
            if (b.p && b.bytes && api::ranges_overlap(a->p, a->bytes, b.p, b.bytes)) return true;
        for (const Span* b = a + 1; b != outs.end(); ++b)
            if (b->p && b->bytes && api::ranges_overlap(a->p, a->bytes, b->p, b->bytes)) return true;
    }
    return false;
}

int check_bias(const void* table, const int* buckets, int num_buckets, int max_distance) {
    if (!table || !buckets || num_buckets < 1 || max_distance < 0) return SKIPARSE_ERR_INVALID_ARG;
    if (max_distance > skiparse::kMaxDist) return SKIPARSE_ERR_UNSUPPORTED;
    if (!aligned(table, 2) || !aligned(buckets, 4)) return SKIPARSE_ERR_MISALIGNED;
    return SKIPARSE_OK;
}

skiparse::FrameBias make_bias(const void* table, const int* buckets, int num_buckets, int max_distance) {
    return {static_cast<const uint16_t*>(table), buckets, table ? max_distance : 0, num_buckets};
}

size_t table_bytes(int num_buckets, int heads) { return static_cast<size_t>(num_buckets) * heads * 2; }
size_t map_bytes(int max_distance) { return (2 * static_cast<size_t>(max_distance) + 1) * 4; }

double log2e_over_sqrt(int d) { return 1.4426950408889634 / std::sqrt(static_cast<double>(d)); }

// ------------------------------------------------------------------------ biased attention

int relbias_fwd(int dims, const void* q, const void* k, const void* v, const void* table, const int* buckets,
                int num_buckets, int max_distance, void* out, void* out_lo, float* lse, int B, int T, int H, int W,
                int heads, int d, int P, int mode, skiparse_stream_t stream) {
    if (!q || !k || !v || !out) return SKIPARSE_ERR_INVALID_ARG;
    Geometry g;
    int st = api::geometry(dims, B, T, H, W, heads, d, P, mode, g);
    if (st == SKIPARSE_OK) st = check_bias(table, buckets, num_buckets, max_distance);
    if (st != SKIPARSE_OK) return st;
    for (const void* ptr : {q, k, v, static_cast<const void*>(out)})
        if (!aligned(ptr, 16)) return SKIPARSE_ERR_MISALIGNED;
    if ((lse && !aligned(lse, 4)) || (out_lo && !aligned(out_lo, 16))) return SKIPARSE_ERR_MISALIGNED;
    const long long rows = static_cast<long long>(B) * T * H * W * heads;
    const size_t tb = static_cast<size_t>(rows) * d * 2;
    if (any_overlap({{out, tb}, {out_lo, tb}, {lse, static_cast<size_t>(rows) * 4}},
                    {{q, tb}, {k, tb}, {v, tb}, {table, table_bytes(num_buckets, heads)}, {buckets, map_bytes(max_distance)}}))
        return SKIPARSE_ERR_INVALID_ARG;
    skiparse::FramesFwdParams p{};
    p.q = static_cast<const uint16_t*>(q);
    p.k = static_cast<const uint16_t*>(k);
    p.v = static_cast<const uint16_t*>(v);
    p.out = static_cast<uint16_t*>(out);
    p.out_lo = static_cast<uint16_t*>(out_lo);
    p.lse = lse;
    if (!(p.status = api::status_word())) return SKIPARSE_ERR_CUDA;
    skiparse::fill_frame_geom(p.g, g);
    p.bias = make_bias(table, buckets, num_buckets, max_distance);
    p.scale_log2 = static_cast<float>(log2e_over_sqrt(d));
    p.wait_limit_ns = api::wait_limit_ns();
    p.fault = api::pending_fault(1);
    p.nrows = api::debug_bound(rows);
    const int e = skiparse::launch_frames_fwd(p, g, stream);
    return e == 0 ? SKIPARSE_OK : api::cuda_fail(e);
}

// Workspace of the backward pass, in order (each part 256-byte aligned): D and lse * log2(e) of
// every row, the sums of dS by head, distance, subsequence and key tile.
struct BwdSpace {
    size_t lse2, part, bytes;
    int Dn, ND, tiles;
};

size_t pad256(size_t n) { return (n + 255) / 256 * 256; }

BwdSpace bwd_space(const Geometry& g, int max_distance) {
    BwdSpace w;
    w.Dn = max_distance < g.T - 1 ? max_distance : g.T - 1;
    w.ND = 2 * w.Dn + 1;
    const long long n = static_cast<long long>(g.T) * skiparse::max_class_tokens(g);
    w.tiles = static_cast<int>((n + 127) / 128);
    const size_t rows = static_cast<size_t>(g.B) * g.T * g.H * g.W * g.heads;
    w.lse2 = pad256(rows * 4);
    w.part = w.lse2 + pad256(rows * 4);
    w.bytes = w.part + pad256(static_cast<size_t>(g.heads) * g.B * g.Ph * g.Pw * w.tiles * w.ND * 4);
    return w;
}

long long relbias_bwd_workspace(int dims, int B, int T, int H, int W, int heads, int d, int P, int max_distance) {
    Geometry g;
    if (api::geometry(dims, B, T, H, W, heads, d, P, SKIPARSE_TOKEN_WISE, g) != SKIPARSE_OK) return -1;
    if (max_distance < 0 || max_distance > skiparse::kMaxDist) return -1;
    // the largest class is the same size in both modes up to the padded one: take the larger
    Geometry h;
    api::geometry(dims, B, T, H, W, heads, d, P, SKIPARSE_GROUP_WISE, h);
    const size_t a = bwd_space(g, max_distance).bytes, b = bwd_space(h, max_distance).bytes;
    return static_cast<long long>(a > b ? a : b);
}

int relbias_bwd(int dims, const void* q, const void* k, const void* v, const void* out, const void* out_lo,
                const void* dout, const float* lse, const void* table, const int* buckets, int num_buckets, int max_distance, void* dq,
                void* dk, void* dv, void* dtable, void* workspace, size_t workspace_bytes, int B, int T, int H, int W,
                int heads, int d, int P, int mode, skiparse_stream_t stream) {
    if (!q || !k || !v || !out || !dout || !lse || !dq || !dk || !dv || !dtable || !workspace)
        return SKIPARSE_ERR_INVALID_ARG;
    Geometry g;
    int st = api::geometry(dims, B, T, H, W, heads, d, P, mode, g);
    if (st == SKIPARSE_OK) st = check_bias(table, buckets, num_buckets, max_distance);
    if (st != SKIPARSE_OK) return st;
    for (const void* ptr : {q, k, v, out, dout, static_cast<const void*>(dq), static_cast<const void*>(dk),
                            static_cast<const void*>(dv)})
        if (!aligned(ptr, 16)) return SKIPARSE_ERR_MISALIGNED;
    if (!aligned(lse, 4) || !aligned(dtable, 2) || (out_lo && !aligned(out_lo, 16)) || !aligned(workspace, 256)) return SKIPARSE_ERR_MISALIGNED;
    const BwdSpace w = bwd_space(g, max_distance);
    if (workspace_bytes < w.bytes) return SKIPARSE_ERR_INVALID_ARG;
    const long long rows = static_cast<long long>(B) * T * H * W * heads;
    const size_t tb = static_cast<size_t>(rows) * d * 2, nt = table_bytes(num_buckets, heads);
    if (any_overlap({{dq, tb}, {dk, tb}, {dv, tb}, {dtable, nt}, {workspace, w.bytes}},
                    {{q, tb}, {k, tb}, {v, tb}, {out, tb}, {out_lo, tb}, {dout, tb}, {lse, static_cast<size_t>(rows) * 4}, {table, nt},
                     {buckets, map_bytes(max_distance)}}))
        return SKIPARSE_ERR_INVALID_ARG;
    char* ws = static_cast<char*>(workspace);
    skiparse::FramesBwdParams p{};
    p.q = static_cast<const uint16_t*>(q);
    p.k = static_cast<const uint16_t*>(k);
    p.v = static_cast<const uint16_t*>(v);
    p.out = static_cast<const uint16_t*>(out);
    p.out_lo = static_cast<const uint16_t*>(out_lo);
    p.dout = static_cast<const uint16_t*>(dout);
    p.lse = lse;
    p.delta = reinterpret_cast<float*>(ws);
    p.nlse2 = reinterpret_cast<float*>(ws + w.lse2);
    p.part = reinterpret_cast<float*>(ws + w.part);
    p.dtable = static_cast<uint16_t*>(dtable);
    p.dq = static_cast<uint16_t*>(dq);
    p.dk = static_cast<uint16_t*>(dk);
    p.dv = static_cast<uint16_t*>(dv);
    if (!(p.status = api::status_word())) return SKIPARSE_ERR_CUDA;
    skiparse::fill_frame_geom(p.g, g);
    p.bias = make_bias(table, buckets, num_buckets, max_distance);
    p.Dn = w.Dn;
    p.ND = w.ND;
    p.seqs = B * g.Ph * g.Pw;
    p.tiles = w.tiles;
    p.order.init(heads * p.seqs, p.tiles, heads);
    p.scale = static_cast<float>(1.0 / std::sqrt(static_cast<double>(d)));
    p.scale_log2 = static_cast<float>(log2e_over_sqrt(d));
    p.wait_limit_ns = api::wait_limit_ns();
    p.nrows = api::debug_bound(rows);
    p.fault = api::pending_fault(2);
    const int e = skiparse::launch_frames_bwd(p, g, stream);
    return e == 0 ? SKIPARSE_OK : api::cuda_fail(e);
}

// -------------------------------------------------------------------------------- the cache

long long frame_tokens(const Geometry& g) { return static_cast<long long>(g.R) * g.S; }

// Geometry of a cache call; capacity in frames.
int cache_geometry(int dims, int B, int T, int H, int W, int heads, int d, int P, int mode, int capacity, Geometry& g) {
    const int st = api::geometry(dims, B, T, H, W, heads, d, P, mode, g);
    if (st != SKIPARSE_OK) return st;
    if (capacity < T) return SKIPARSE_ERR_INVALID_ARG;  // a call's own frames have to fit
    if (capacity > (1 << 24) || capacity * frame_tokens(g) > (1ll << 30)) return SKIPARSE_ERR_UNSUPPORTED;
    return SKIPARSE_OK;
}

struct CacheBytes {
    size_t codes, scales;
};
CacheBytes cache_bytes(const Geometry& g, int capacity) {
    const size_t slots = static_cast<size_t>(g.B) * g.Ph * g.Pw * g.heads * capacity, F = static_cast<size_t>(frame_tokens(g));
    return {slots * F * g.d, slots * ((F + skiparse::kCacheBlock - 1) / skiparse::kCacheBlock)};
}

skiparse::CacheView cache_view(const Geometry& g, const void* k, const void* v, const void* ks, const void* vs,
                               const int* start, int capacity) {
    skiparse::CacheView c;
    c.k = static_cast<uint8_t*>(const_cast<void*>(k));
    c.v = static_cast<uint8_t*>(const_cast<void*>(v));
    c.ks = static_cast<uint8_t*>(const_cast<void*>(ks));
    c.vs = static_cast<uint8_t*>(const_cast<void*>(vs));
    c.start = start;
    c.cap = capacity;
    c.F = static_cast<int>(frame_tokens(g));
    c.NBk = (c.F + skiparse::kCacheBlock - 1) / skiparse::kCacheBlock;
    return c;
}

int cache_append(int dims, const void* k, const void* v, const int* start, void* k_cache, void* v_cache, void* k_scale,
                 void* v_scale, int B, int T, int H, int W, int heads, int d, int P, int mode, int capacity,
                 skiparse_stream_t stream) {
    if (!k || !v || !start || !k_cache || !v_cache || !k_scale || !v_scale) return SKIPARSE_ERR_INVALID_ARG;
    Geometry g;
    const int st = cache_geometry(dims, B, T, H, W, heads, d, P, mode, capacity, g);
    if (st != SKIPARSE_OK) return st;
    for (const void* ptr : {k, v, static_cast<const void*>(k_cache), static_cast<const void*>(v_cache)})
        if (!aligned(ptr, 16)) return SKIPARSE_ERR_MISALIGNED;
    if (!aligned(start, 4)) return SKIPARSE_ERR_MISALIGNED;
    const long long rows = static_cast<long long>(B) * T * H * W * heads;
    const size_t tb = static_cast<size_t>(rows) * d * 2;
    const CacheBytes cb = cache_bytes(g, capacity);
    if (any_overlap({{k_cache, cb.codes}, {v_cache, cb.codes}, {k_scale, cb.scales}, {v_scale, cb.scales}},
                    {{k, tb}, {v, tb}, {start, static_cast<size_t>(B) * 4}}))
        return SKIPARSE_ERR_INVALID_ARG;
    skiparse::AppendParams p{};
    p.k = static_cast<const uint16_t*>(k);
    p.v = static_cast<const uint16_t*>(v);
    if (!(p.status = api::status_word())) return SKIPARSE_ERR_CUDA;
    skiparse::fill_frame_geom(p.g, g);
    p.cache = cache_view(g, k_cache, v_cache, k_scale, v_scale, start, capacity);
    p.nblk = (skiparse::max_class_tokens(g) + skiparse::kCacheBlock - 1) / skiparse::kCacheBlock;
    p.nrows = api::debug_bound(rows);
    const int e = skiparse::launch_cache_append(p, g, d, stream);
    return e == 0 ? SKIPARSE_OK : api::cuda_fail(e);
}

// Workspace of a cache call: log-sum-exps, then outputs, of the parts of its split items.
size_t cached_part_l(const skiparse::CachePlan& c) { return pad256(static_cast<size_t>(c.part_rows) * c.splits * 4); }
size_t cached_space(const skiparse::CachePlan& c, int d) {
    return c.splits == 1 ? 0 : cached_part_l(c) + static_cast<size_t>(c.part_rows) * c.splits * d * 4;
}

long long cached_workspace(int dims, int B, int T, int H, int W, int heads, int d, int P, int capacity) {
    Geometry g, h;
    if (cache_geometry(dims, B, T, H, W, heads, d, P, SKIPARSE_TOKEN_WISE, capacity, g) != SKIPARSE_OK) return -1;
    cache_geometry(dims, B, T, H, W, heads, d, P, SKIPARSE_GROUP_WISE, capacity, h);
    const size_t a = cached_space(skiparse::cached_plan(g, capacity), d), b = cached_space(skiparse::cached_plan(h, capacity), d);
    return static_cast<long long>(a > b ? a : b);
}

int attn_cached(int dims, const void* q, const void* k_cache, const void* v_cache, const void* k_scale,
                const void* v_scale, const int* start, const void* table, const int* buckets, int num_buckets,
                int max_distance, void* out, float* lse, void* workspace, size_t workspace_bytes, int B, int T, int H,
                int W, int heads, int d, int P, int mode, int capacity, skiparse_stream_t stream) {
    if (!q || !k_cache || !v_cache || !k_scale || !v_scale || !start || !out) return SKIPARSE_ERR_INVALID_ARG;
    if (!table != !buckets) return SKIPARSE_ERR_INVALID_ARG;
    Geometry g;
    int st = cache_geometry(dims, B, T, H, W, heads, d, P, mode, capacity, g);
    if (st == SKIPARSE_OK && table) st = check_bias(table, buckets, num_buckets, max_distance);
    if (st != SKIPARSE_OK) return st;
    for (const void* ptr : {q, k_cache, v_cache, static_cast<const void*>(out)})
        if (!aligned(ptr, 16)) return SKIPARSE_ERR_MISALIGNED;
    if (!aligned(start, 4) || (lse && !aligned(lse, 4)) || (workspace && !aligned(workspace, 256)))
        return SKIPARSE_ERR_MISALIGNED;
    const skiparse::CachePlan plan = skiparse::cached_plan(g, capacity);
    const size_t need = cached_space(plan, d);
    if (need && (!workspace || workspace_bytes < need)) return SKIPARSE_ERR_INVALID_ARG;
    const long long rows = static_cast<long long>(B) * T * H * W * heads;
    const size_t tb = static_cast<size_t>(rows) * d * 2;
    const CacheBytes cb = cache_bytes(g, capacity);
    if (any_overlap({{out, tb}, {lse, static_cast<size_t>(rows) * 4}, {need ? workspace : nullptr, need}},
                    {{q, tb}, {k_cache, cb.codes}, {v_cache, cb.codes}, {k_scale, cb.scales}, {v_scale, cb.scales},
                     {start, static_cast<size_t>(B) * 4}, {table, table ? table_bytes(num_buckets, heads) : 0},
                     {buckets, table ? map_bytes(max_distance) : 0}}))
        return SKIPARSE_ERR_INVALID_ARG;
    skiparse::FramesFwdParams p{};
    p.q = static_cast<const uint16_t*>(q);
    p.out = static_cast<uint16_t*>(out);
    p.lse = lse;
    p.plan = plan;
    p.part_l = static_cast<float*>(workspace);
    p.part_o = reinterpret_cast<float*>(static_cast<char*>(workspace) + cached_part_l(plan));
    if (!(p.status = api::status_word())) return SKIPARSE_ERR_CUDA;
    skiparse::fill_frame_geom(p.g, g);
    p.bias = make_bias(table, buckets, num_buckets, max_distance);
    p.cache = cache_view(g, k_cache, v_cache, k_scale, v_scale, start, capacity);
    p.scale_log2 = static_cast<float>(log2e_over_sqrt(d));
    p.wait_limit_ns = api::wait_limit_ns();
    p.fault = skiparse::cached_small(g) ? 0 : api::pending_fault(1);  // the few-query kernel has no waits
    p.nrows = api::debug_bound(rows);
    const int e = skiparse::launch_frames_fwd(p, g, stream);
    return e == 0 ? SKIPARSE_OK : api::cuda_fail(e);
}

}  // namespace

extern "C" {

#define SKIPARSE_FRAMES_ENTRIES(N)                                                                                      \
    int skiparse##N##d_attn_relbias_fwd(const void* q, const void* k, const void* v, const void* table,                 \
                                        const int* buckets, int num_buckets, int max_distance, void* out, void* out_lo, \
                                        float* lse, int B, int T, int H, int W, int heads, int d, int P, int mode,      \
                                        skiparse_stream_t stream) {                                                     \
        return relbias_fwd(N, q, k, v, table, buckets, num_buckets, max_distance, out, out_lo, lse, B, T, H, W, heads,  \
                           d, P, mode, stream);                                                                         \
    }                                                                                                                   \
    int skiparse##N##d_attn_relbias_bwd(const void* q, const void* k, const void* v, const void* out,                   \
                                        const void* out_lo, const void* dout, const float* lse, const void* table,      \
                                        const int* buckets, int num_buckets, int max_distance, void* dq, void* dk,      \
                                        void* dv, void* dtable, void* workspace, size_t workspace_bytes, int B, int T,  \
                                        int H, int W, int heads, int d, int P, int mode, skiparse_stream_t stream) {    \
        return relbias_bwd(N, q, k, v, out, out_lo, dout, lse, table, buckets, num_buckets, max_distance, dq, dk, dv,   \
                           dtable, workspace, workspace_bytes, B, T, H, W, heads, d, P, mode, stream);                  \
    }                                                                                                                   \
    long long skiparse##N##d_attn_relbias_bwd_workspace_bytes(int B, int T, int H, int W, int heads, int d, int P,      \
                                                              int max_distance) {                                       \
        return relbias_bwd_workspace(N, B, T, H, W, heads, d, P, max_distance);                                         \
    }                                                                                                                   \
    long long skiparse##N##d_cache_frame_tokens(int H, int W, int P) {                                                  \
        Geometry g;                                                                                                     \
        if (api::geometry(N, 1, 1, H, W, 1, 32, P, SKIPARSE_TOKEN_WISE, g) != SKIPARSE_OK) return -1;                   \
        return frame_tokens(g);                                                                                         \
    }                                                                                                                   \
    int skiparse##N##d_cache_append(const void* k, const void* v, const int* start, void* k_cache, void* v_cache,       \
                                    void* k_scale, void* v_scale, int B, int T, int H, int W, int heads, int d, int P,  \
                                    int mode, int capacity, skiparse_stream_t stream) {                                 \
        return cache_append(N, k, v, start, k_cache, v_cache, k_scale, v_scale, B, T, H, W, heads, d, P, mode,          \
                            capacity, stream);                                                                          \
    }                                                                                                                   \
    long long skiparse##N##d_attn_cached_workspace_bytes(int B, int T, int H, int W, int heads, int d, int P,           \
                                                         int capacity) {                                                \
        return cached_workspace(N, B, T, H, W, heads, d, P, capacity);                                                  \
    }                                                                                                                   \
    int skiparse##N##d_attn_cached(const void* q, const void* k_cache, const void* v_cache, const void* k_scale,        \
                                   const void* v_scale, const int* start, const void* table, const int* buckets,        \
                                   int num_buckets, int max_distance, void* out, float* lse, void* workspace,           \
                                   size_t workspace_bytes, int B, int T, int H, int W, int heads, int d, int P,         \
                                   int mode, int capacity, skiparse_stream_t stream) {                                  \
        return attn_cached(N, q, k_cache, v_cache, k_scale, v_scale, start, table, buckets, num_buckets, max_distance,  \
                           out, lse, workspace, workspace_bytes, B, T, H, W, heads, d, P, mode, capacity, stream);      \
    }

SKIPARSE_FRAMES_ENTRIES(2)
SKIPARSE_FRAMES_ENTRIES(1)

}  // extern "C"
