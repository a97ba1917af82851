// pi_paged.hip -- host side of the C ABI declared in include/pi_paged_kv.h: argument checks, the
// choice of kernel and grid, launches.  As in pi_abi.hip nothing here allocates, frees, synchronizes
// or issues memset/memcpy nodes, and no C++ exception crosses the ABI.
#include "pi_paged.hpp"

#include <algorithm>
#include <cmath>

namespace {

using namespace pik;

constexpr int kMaxHeads = 1024;
// Key ranges are cut so that about as many workgroups share the work of all requests as the 256 CUs hold
// at once: 3, 2 or 1 each, by the registers of either kernel.
constexpr int split_target(int hd) { return hd == 64 ? 768 : hd == 128 ? 512 : 256; }
constexpr int kCus = 256;
constexpr int kJoinGroups = 1024;         // workgroups of k_kv_join, at most

inline bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// log2 of a page size, or -1.
int page_log(int32_t page) {
    switch (page) {
        case 16: return 4;
        case 32: return 5;
        case 64: return 6;
        case 128: return 7;
        case 256: return 8;
        default: return -1;
    }
}

int check_cache(const pi_kv_cache *c) {
    if (!c || !c->k_pages || !c->v_pages) return PI_ERR_NULL;
    if (c->dtype != PI_KV_F16 && c->dtype != PI_KV_BF16) return PI_ERR_DTYPE;
    if (page_log(c->page) < 0 || c->n_pages < 1 || c->n_kv < 1 || c->n_kv > kMaxHeads) return PI_ERR_SHAPE;
    if (c->head_dim != 64 && c->head_dim != 128 && c->head_dim != 256) return PI_ERR_SHAPE;
    if ((int64_t)c->n_pages * c->page > INT32_MAX) return PI_ERR_SHAPE;
    if (!aligned16(c->k_pages) || !aligned16(c->v_pages)) return PI_ERR_ALIGN;
    return PI_OK;
}

int check_batch(const pi_kv_batch *b) {
    if (!b || !b->block_table || !b->q_start || !b->kv_len) return PI_ERR_NULL;
    if (b->n_req < 1 || b->n_req > PI_KV_MAX_REQ || b->max_pages < 1 || b->max_pages > PI_KV_MAX_TABLE ||
        b->table_stride < b->max_pages || b->max_q < 1 || b->max_q > PI_KV_MAX_TOKENS || b->max_kv < 0)
        return PI_ERR_SHAPE;
    return PI_OK;
}

int check_rows(const pi_kv_cache *c, int32_t total_q, int32_t n_q) {
    if (total_q < 0 || total_q > PI_KV_MAX_TOKENS || n_q < 1 || n_q > kMaxHeads || n_q % c->n_kv != 0) return PI_ERR_SHAPE;
    return PI_OK;
}

// Rows of [n][heads][head_dim] with strides in elements: 16-byte rows.
int check_strides(const void *p, int64_t ts, int64_t hs) {
    if (ts < 0 || hs < 0) return PI_ERR_SHAPE;
    if (!aligned16(p) || ts % 8 != 0 || hs % 8 != 0) return PI_ERR_ALIGN;
    return PI_OK;
}

// Whether two of the rows [hd] at t * ts + h * hs, t < n, h < heads, share an element.
bool rows_overlap(int64_t ts, int64_t hs, int n, int heads, int hd) {
    if ((n > 1 && ts < hd) || (heads > 1 && hs < hd)) return true;
    if (n < 2 || heads < 2) return false;
    if (ts / hs >= heads) return false;              // whole tokens after one another
    for (int h = 1; h < heads; ++h) {                // a row h heads on, and the nearest ones t tokens on
        const __int128 x = (__int128)h * hs, t = x / ts;
        if ((t < n && x - t * ts < hd) || (t + 1 < n && (t + 1) * ts - x < hd)) return true;
    }
    return false;
}

// Rows per workgroup by the most query rows that a request can have per kv head: single tokens and
// drafts go to k_kv_rows, whose waves share out the keys; the rest, and whatever single tokens run
// beside it, to k_kv_tile.
struct AttnPlan {
    int TR;
    bool shorts;     // k_kv_rows with more waves per workgroup
    bool single;     // k_kv_rows in workgroups of one wave
    bool mixed;      // k_kv_tile with a path of its own for requests of few rows
    int tiles;       // row tiles per kv head, at most
    int items;       // items per kv head, at most
    int slots;       // split items per kv head, at most
    int target;      // split target, 0: no key range is cut
    size_t bytes;    // of the split items' partial sums
};

AttnPlan attn_plan(const pi_kv_cache *c, const pi_kv_batch *b, int total_q, int n_q) {
    AttnPlan p{};
    const int64_t group = n_q / c->n_kv, rows = std::min(b->max_q, total_q) * group, reqs = std::min(b->n_req, total_q);
    // Up to 128 rows fit one wide tile, but tiles of 16, whose waves share out the keys, are done sooner where the latency
    // of the blocks counts and reading the keys again, from L2, does not: up to 64 MB of that (2 x 3 tokens on 600 keys, 8
    // kv heads of 64 for 128: 17.0 us wide, 8.3 so; 1 x 8 on 8000: 20.0 wide, 26.1 so), and up to 512 MB for heads of 256,
    // whose wide tiles run one wave per SIMD (16 x 4 on 8000 keys: 69.6 wide, 59.5 so).
    const double again = 4.0 * reqs * ((rows + kKvRowTile - 1) / kKvRowTile) * c->n_kv * b->max_kv * c->head_dim;
    const bool narrow = rows <= kKvRowTile || (rows <= kKvWideTile && again <= (c->head_dim == 256 ? 512 << 20 : 64 << 20));
    p.TR = narrow ? kKvRowTile : kKvWideTile;
    // on average, requests of fewer than half of max_q tokens: some of them have few rows
    p.mixed = (int64_t)2 * total_q < (int64_t)b->max_q * b->n_req;
    p.tiles = (int)std::min(total_q * group / p.TR + reqs, reqs * ((rows + p.TR - 1) / p.TR));
    p.items = p.tiles;
    p.bytes = 16;
    // Nothing is cut where there are too few keys for two pieces, or row tiles to fill the chip many times.
    // With few tiles the pieces fill the chip just once (4 x 60k grouped: 84.8 us, and 88.6 with twice as many); with
    // about as many as it holds, finer ones even out their lengths (16 x 2k: 62.6 us, and 66.3 with half as many), unless
    // the tiles are wide: their partial sums cost more (2048 tokens on 8000 keys, 32 heads of 128: 349 us cut in two,
    // 259 not).
    int target = split_target(c->head_dim);
    const int64_t all = (int64_t)p.tiles * c->n_kv;
    // With a CU for each range, more waves in one workgroup read a short one sooner than its pieces are joined (1 x 513,
    // 16 heads of 64: 7.5 us, and 9.7 cut; 8 x 1000, 32 heads of 128: 27.8, and 34.4).  A CU alone reads at about 50
    // GB/s, so the longer ones of these are worth it only if most CUs have one.
    const int64_t range = (int64_t)b->max_kv * c->head_dim * 4;
    p.shorts = p.TR == kKvRowTile && c->head_dim != 256 && b->max_kv > kKvMinPiece && all <= kCus &&
               range <= (2 * all >= kCus ? 512 : 256) << 10;
    // More workgroups than the chip holds, of short ranges each: one wave each, so that it holds four times as many (49
    // requests of up to 18 keys, 56 heads of 128: 32.2 -> 18.5 us).
    p.single = p.TR == kKvRowTile && all > target && b->max_kv <= kKvMinPiece;
    if (narrow && 2 * all > target && all < 8 * target) target *= 2;
    // (the tiles of one request alone are all cut in target / all + 1/4: with less than 2 no join is launched)
    const bool whole = reqs == 1 && 4 * target < 7 * all;
    if (!p.shorts && !p.single && !whole && all < 8 * target && b->max_kv >= kv_min_cut(c->head_dim)) {
        p.target = target;
        p.items += target / c->n_kv + 2;             // 2: the device sums the work in fp32
        p.slots = std::min(p.items, 2 * target / c->n_kv + 4);
        p.bytes = (size_t)p.slots * c->n_kv * p.TR * (c->head_dim + 2) * sizeof(float);
    }
    return p;
}

template <class T, int HD, int TR>
int launch_join(const KvAttnArgs &a, const AttnPlan &p, hipStream_t st) {
    if (!p.target) return PI_OK;
    // at most every row of every tile, a few rows per workgroup; long lists are walked by a bounded grid
    const int64_t rows = std::min<int64_t>((int64_t)p.tiles * TR, (int64_t)a.total_q * a.group);
    const int64_t groups = (rows * (HD / 4) + 63) / 64 * a.n_kv;
    hipLaunchKernelGGL((k_kv_join<T, HD, TR>), dim3((uint32_t)std::min<int64_t>(groups, kJoinGroups)), dim3(256), 0, st, a);
    return hipGetLastError() == hipSuccess ? PI_OK : PI_ERR_HIP;
}

template <class T, int HD, bool MIXED>
void launch_tile(const KvAttnArgs &a, dim3 grid, hipStream_t st) {
    constexpr int kKeys = KvTile<HD, 16>::kKeys;
    if (a.page_log == 4)
        hipLaunchKernelGGL((k_kv_tile<T, HD, 16, MIXED>), grid, dim3(256), 0, st, a);
    else if (a.page_log == 5 || kKeys == 32)
        hipLaunchKernelGGL((k_kv_tile<T, HD, 32, MIXED>), grid, dim3(256), 0, st, a);
    else
        hipLaunchKernelGGL((k_kv_tile<T, HD, kKeys, MIXED>), grid, dim3(256), 0, st, a);
}

template <class T, int HD>
int launch_attn(const KvAttnArgs &a, const AttnPlan &p, hipStream_t st) {
    const dim3 grid((uint32_t)p.items * a.n_kv);
    constexpr int kShort = HD == 256 ? kKvRowWaves : kv_short_waves(HD);
    if (p.single)
        hipLaunchKernelGGL((k_kv_rows<T, HD, 1>), grid, dim3(64), 0, st, a);
    else if (HD != 256 && p.shorts)
        hipLaunchKernelGGL((k_kv_rows<T, HD, kShort>), grid, dim3(64 * kShort), 0, st, a);
    else if (p.TR == kKvRowTile)
        hipLaunchKernelGGL((k_kv_rows<T, HD, kKvRowWaves>), grid, dim3(64 * kKvRowWaves), 0, st, a);
    else if (p.mixed)
        launch_tile<T, HD, true>(a, grid, st);
    else
        launch_tile<T, HD, false>(a, grid, st);
    if (hipGetLastError() != hipSuccess) return PI_ERR_HIP;
    return p.TR == kKvRowTile ? launch_join<T, HD, kKvRowTile>(a, p, st) : launch_join<T, HD, kKvWideTile>(a, p, st);
}

template <class T>
int launch_attn_hd(int hd, const KvAttnArgs &a, const AttnPlan &g, hipStream_t st) {
    if (hd == 64) return launch_attn<T, 64>(a, g, st);
    if (hd == 128) return launch_attn<T, 128>(a, g, st);
    return launch_attn<T, 256>(a, g, st);
}

template <int TT>
int launch_append(const KvAppendArgs &a, hipStream_t st) {
    const size_t lds = (size_t)TT * (a.hd / 2 + 1) * sizeof(uint32_t);
    hipLaunchKernelGGL((k_kv_append<TT>), dim3(a.n_kv, (a.n_tokens + TT - 1) / TT), dim3(256), lds, st, a);
    return hipGetLastError() == hipSuccess ? PI_OK : PI_ERR_HIP;
}

}  // namespace

extern "C" int pi_kv_step(const pi_kv_tables *t, void *stream) {
    if (!t || !t->cached || !t->fresh || !t->free_ring || !t->pool || !t->block_table || !t->q_start || !t->kv_len ||
        !t->cached_next || !t->slots || !t->pool_next || !t->counts)
        return PI_ERR_NULL;
    if (t->n_req < 1 || t->n_req > PI_KV_MAX_REQ || page_log(t->page) < 0 || t->n_pages < 1 || t->max_pages < 1 ||
        t->max_pages > PI_KV_MAX_TABLE || t->max_tokens < 1 || t->max_tokens > PI_KV_MAX_TOKENS ||
        t->table_stride < t->max_pages || (int64_t)t->n_pages * t->page > INT32_MAX ||
        (int64_t)t->max_pages * t->page > INT32_MAX)
        return PI_ERR_SHAPE;
    KvTablesArgs a{t->n_req, page_log(t->page), t->n_pages, t->max_pages, t->max_tokens, t->table_stride, t->cached, t->fresh,
                   t->free_ring, t->pool, t->block_table, t->q_start, t->kv_len, t->cached_next, t->slots, t->pool_next, t->counts};
    // A step in place runs in one workgroup, which reads all of the old state before it writes.
    const bool in_place = t->cached_next == t->cached || t->pool_next == t->pool;
    const int groups = in_place ? 1 : std::min(64, std::max((t->max_tokens + 1023) / 1024, (t->n_req + 255) / 256));
    hipLaunchKernelGGL(k_kv_tables, dim3(groups), dim3(kKvTableThreads), 0, static_cast<hipStream_t>(stream), a);
    return hipGetLastError() == hipSuccess ? PI_OK : PI_ERR_HIP;
}

extern "C" int pi_kv_append(const pi_kv_cache *cache, const void *k, int64_t k_token_stride, int64_t k_head_stride, const void *v,
                            int64_t v_token_stride, int64_t v_head_stride, const int32_t *slots, int32_t n_tokens,
                            void *stream) {
    int rc = check_cache(cache);
    if (rc) return rc;
    if (n_tokens < 0 || n_tokens > PI_KV_MAX_TOKENS) return PI_ERR_SHAPE;
    if (n_tokens == 0) return PI_OK;                 // empty tensors have no address
    if (!k || !v || !slots) return PI_ERR_NULL;
    if ((rc = check_strides(k, k_token_stride, k_head_stride)) || (rc = check_strides(v, v_token_stride, v_head_stride))) return rc;
    KvAppendArgs a{n_tokens, cache->n_kv, cache->head_dim, page_log(cache->page), cache->n_pages * cache->page,
                   k_token_stride, k_head_stride, v_token_stride, v_head_stride, static_cast<const uint16_t *>(k),
                   static_cast<const uint16_t *>(v), slots, static_cast<uint16_t *>(cache->k_pages),
                   static_cast<uint16_t *>(cache->v_pages)};
    hipStream_t st = static_cast<hipStream_t>(stream);
    // Tiles of 64 tokens, or of 16 where those are fewer workgroups than two per CU (3000 tokens of 2 heads of 256:
    // 10.6 -> 7.0 us; 64 tokens of 32 heads of 128: 9.3 -> 5.5).
    return (int64_t)((n_tokens + 63) / 64) * cache->n_kv >= 2 * kCus ? launch_append<64>(a, st) : launch_append<16>(a, st);
}

extern "C" size_t pi_kv_attn_workspace_bytes(const pi_kv_cache *cache, const pi_kv_batch *batch, int32_t total_q, int32_t n_q) {
    if (check_cache(cache) || check_batch(batch) || check_rows(cache, total_q, n_q)) return 0;
    return attn_plan(cache, batch, total_q, n_q).bytes;
}

extern "C" int pi_kv_attn(const pi_kv_cache *cache, const pi_kv_batch *batch, const void *q, int64_t q_token_stride,
                          int64_t q_head_stride, void *out, int64_t out_token_stride, int64_t out_head_stride, int32_t total_q,
                          int32_t n_q, float scale, int32_t window, void *ws, size_t ws_bytes, void *stream) {
    int rc = check_cache(cache);
    if (rc || (rc = check_batch(batch))) return rc;
    if ((rc = check_rows(cache, total_q, n_q))) return rc;
    if (total_q == 0) return PI_OK;
    if (!q || !out) return PI_ERR_NULL;
    if (window < 0 || !(scale > 0.f) || !std::isfinite(scale)) return PI_ERR_SHAPE;
    if ((rc = check_strides(q, q_token_stride, q_head_stride)) || (rc = check_strides(out, out_token_stride, out_head_stride)))
        return rc;
    if (rows_overlap(out_token_stride, out_head_stride, total_q, n_q, cache->head_dim)) return PI_ERR_SHAPE;
    const AttnPlan g = attn_plan(cache, batch, total_q, n_q);
    if (!ws || ws_bytes < g.bytes) return PI_ERR_WORKSPACE;
    if (!aligned16(ws)) return PI_ERR_ALIGN;
    KvAttnArgs a{};
    a.n_pages = cache->n_pages, a.n_kv = cache->n_kv, a.page_log = page_log(cache->page);
    a.n_req = batch->n_req, a.max_pages = batch->max_pages, a.max_q = batch->max_q, a.max_kv = batch->max_kv;
    // positions stay below 2^31 - 2^19 - window: the lower ends of windows are computed in 32 bits
    a.total_q = total_q, a.n_q = n_q, a.group = n_q / cache->n_kv, a.window = std::min(window, INT32_MAX - PI_KV_MAX_TOKENS);
    a.split_target = g.target, a.slots = g.slots, a.items = g.items;
    a.scale_log2 = scale * 1.4426950408889634f;
    a.table_stride = batch->table_stride;
    a.q_ts = q_token_stride, a.q_hs = q_head_stride, a.o_ts = out_token_stride, a.o_hs = out_head_stride;
    a.k = static_cast<const uint16_t *>(cache->k_pages), a.v = static_cast<const uint16_t *>(cache->v_pages);
    a.q = static_cast<const uint16_t *>(q), a.out = static_cast<uint16_t *>(out);
    a.table = batch->block_table, a.q_start = batch->q_start, a.kv_len = batch->kv_len;
    a.part = static_cast<float *>(ws);
    hipStream_t st = static_cast<hipStream_t>(stream);
    return cache->dtype == PI_KV_F16 ? launch_attn_hd<KvF16>(cache->head_dim, a, g, st)
                                     : launch_attn_hd<KvBf16>(cache->head_dim, a, g, st);
}
