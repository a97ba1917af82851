// pi_paged_launch.hpp -- the choice of kernel and grid for attention over pages, and its launches; one unit each for the
// window alone (pi_paged.hip) and for the window and the first tokens (pi_paged_sinks.hip).
#pragma once

#include "pi_paged.hpp"
#include "pi_paged_host.hpp"

#include <algorithm>
#include <cmath>

namespace pik {

// Key ranges are cut so that about as many workgroups share the work of all requests as the 256 CUs hold
// at once: 3, 2 or 1 each, by the registers of either kernel.
constexpr int split_target(int hd) { return hd == 64 ? 768 : hd == 128 ? 512 : 256; }
constexpr int kJoinGroups = 1024;         // workgroups of k_kv_join, at most

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

// max_kv: keys of a request that the step may read, at most.  even: most requests read as many.
inline AttnPlan attn_plan(const pi_kv_cache *c, const pi_kv_batch *b, int total_q, int n_q, int max_kv,
                          bool even) {
    AttnPlan p{};
    const int64_t group = n_q / c->n_kv, rows = std::min(b->max_q, total_q) * group, reqs = std::min(b->n_req, total_q);
    // Up to 128 rows fit one wide tile, but tiles of 16, whose waves share out the keys, are done sooner where the latency
    // of the blocks counts and reading the keys again, from L2, does not: up to 64 MB of that (2 x 3 tokens on 600 keys, 8
    // kv heads of 64 for 128: 17.0 us wide, 8.3 so; 1 x 8 on 8000: 20.0 wide, 26.1 so), and up to 512 MB for heads of 256,
    // whose wide tiles run one wave per SIMD (16 x 4 on 8000 keys: 69.6 wide, 59.5 so).
    const double again = 4.0 * reqs * ((rows + kKvRowTile - 1) / kKvRowTile) * c->n_kv * max_kv * c->head_dim;
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
    const int64_t range = (int64_t)max_kv * c->head_dim * 4;
    p.shorts = p.TR == kKvRowTile && c->head_dim != 256 && max_kv > kKvMinPiece && all <= kCus &&
               range <= (2 * all >= kCus ? 512 : 256) << 10;
    // More workgroups than the chip holds, of short ranges each: one wave each, so that it holds four times as many (49
    // requests of up to 18 keys, 56 heads of 128: 32.2 -> 18.5 us).
    p.single = p.TR == kKvRowTile && all > target && max_kv <= kKvMinPiece;
    if (narrow && 2 * all > target && all < 8 * target) target *= 2;
    // (the tiles of one request alone are all cut in target / all + 1/4: with less than 2 no join is launched)
    const bool whole = reqs == 1 && 4 * target < 7 * all;
    // Ranges of one length need no evening out: with as many as the chip holds they are read whole, and no join follows (16 x
    // 4100 of 8 to 30 thousand keys, 32 heads of 128: 195 us in halves).
    const bool full = even && all >= split_target(c->head_dim);
    if (!p.shorts && !p.single && !whole && !full && all < 8 * target && max_kv >= kv_min_cut(c->head_dim)) {
        p.target = target;
        p.items += target / c->n_kv + 2;             // 2: the device sums the work in fp32
        p.slots = std::min(p.items, 2 * target / c->n_kv + 4);
        p.bytes = (size_t)p.slots * c->n_kv * p.TR * (c->head_dim + 2) * sizeof(float);
    }
    return p;
}

template <class T, int HD, int TR, bool SINKS>
int launch_join(const KvAttnArgs &a, const AttnPlan &p, hipStream_t st) {
    if (!p.target) return PI_OK;
    // at most every row of every tile, a few rows per workgroup; long lists are walked by a bounded grid
    const int64_t rows = std::min<int64_t>((int64_t)p.tiles * TR, (int64_t)a.total_q * a.group);
    const int64_t groups = (rows * (HD / 4) + 63) / 64 * a.n_kv;
    hipLaunchKernelGGL((k_kv_join<T, HD, TR, SINKS>), dim3((uint32_t)std::min<int64_t>(groups, kJoinGroups)), dim3(256), 0, st, a);
    return hipGetLastError() == hipSuccess ? PI_OK : PI_ERR_HIP;
}

template <class T, int HD, bool MIXED, bool SINKS>
void launch_tile(const KvAttnArgs &a, dim3 grid, hipStream_t st) {
    constexpr int kKeys = KvTile<HD, 16>::kKeys;
    if (a.page_log == 4)
        hipLaunchKernelGGL((k_kv_tile<T, HD, 16, MIXED, SINKS>), grid, dim3(256), 0, st, a);
    else if (a.page_log == 5 || kKeys == 32)
        hipLaunchKernelGGL((k_kv_tile<T, HD, 32, MIXED, SINKS>), grid, dim3(256), 0, st, a);
    else
        hipLaunchKernelGGL((k_kv_tile<T, HD, kKeys, MIXED, SINKS>), grid, dim3(256), 0, st, a);
}

template <class T, int HD, bool SINKS>
int launch_attn(const KvAttnArgs &a, const AttnPlan &p, hipStream_t st) {
    const dim3 grid((uint32_t)p.items * a.n_kv);
    constexpr int kShort = HD == 256 ? kKvRowWaves : kv_short_waves(HD);
    if (p.single)
        hipLaunchKernelGGL((k_kv_rows<T, HD, 1, SINKS>), grid, dim3(64), 0, st, a);
    else if (HD != 256 && p.shorts)
        hipLaunchKernelGGL((k_kv_rows<T, HD, kShort, SINKS>), grid, dim3(64 * kShort), 0, st, a);
    else if (p.TR == kKvRowTile)
        hipLaunchKernelGGL((k_kv_rows<T, HD, kKvRowWaves, SINKS>), grid, dim3(64 * kKvRowWaves), 0, st, a);
    else if (p.mixed)
        launch_tile<T, HD, true, SINKS>(a, grid, st);
    else
        launch_tile<T, HD, false, SINKS>(a, grid, st);
    if (hipGetLastError() != hipSuccess) return PI_ERR_HIP;
    return p.TR == kKvRowTile ? launch_join<T, HD, kKvRowTile, SINKS>(a, p, st) : launch_join<T, HD, kKvWideTile, SINKS>(a, p, st);
}

template <class T, bool SINKS>
int launch_attn_hd(int hd, const KvAttnArgs &a, const AttnPlan &g, hipStream_t st) {
    if (hd == 64) return launch_attn<T, 64, SINKS>(a, g, st);
    if (hd == 128) return launch_attn<T, 128, SINKS>(a, g, st);
    return launch_attn<T, 256, SINKS>(a, g, st);
}

// The call, with sinks = 0 for a window alone.  max_kv: as of attn_plan.
template <bool SINKS>
int run_attn(const pi_kv_cache *cache, const pi_kv_batch *batch, const void *q, int64_t q_token_stride, int64_t q_head_stride,
             void *out, int64_t out_token_stride, int64_t out_head_stride, int32_t total_q, int32_t n_q, float scale,
             int32_t window, int32_t sinks, int max_kv, bool even, void *ws, size_t ws_bytes, hipStream_t st) {
    int rc;
    if ((rc = check_strides(q, q_token_stride, q_head_stride)) || (rc = check_strides(out, out_token_stride, out_head_stride)))
        return rc;
    if (rows_overlap(out_token_stride, out_head_stride, total_q, n_q, cache->head_dim)) return PI_ERR_SHAPE;
    const AttnPlan g = attn_plan(cache, batch, total_q, n_q, max_kv, even);
    if (!ws || ws_bytes < g.bytes) return PI_ERR_WORKSPACE;
    if (!aligned16(ws)) return PI_ERR_ALIGN;
    KvAttnArgs a{};
    a.n_pages = cache->n_pages, a.n_kv = cache->n_kv, a.page_log = page_log(cache->page);
    a.n_req = batch->n_req, a.max_pages = batch->max_pages, a.max_q = batch->max_q, a.max_kv = batch->max_kv;
    // positions stay below 2^31 - 2^19 - window: the lower ends of windows are computed in 32 bits
    a.total_q = total_q, a.n_q = n_q, a.group = n_q / cache->n_kv, a.window = std::min(window, INT32_MAX - PI_KV_MAX_TOKENS);
    a.sinks = std::min(sinks, 1 << 30);              // (rounded up to blocks on the device)
    a.split_target = g.target, a.slots = g.slots, a.items = g.items;
    a.scale_log2 = scale * 1.4426950408889634f;
    a.table_stride = batch->table_stride;
    a.q_ts = q_token_stride, a.q_hs = q_head_stride, a.o_ts = out_token_stride, a.o_hs = out_head_stride;
    a.k = static_cast<const uint16_t *>(cache->k_pages), a.v = static_cast<const uint16_t *>(cache->v_pages);
    a.q = static_cast<const uint16_t *>(q), a.out = static_cast<uint16_t *>(out);
    a.table = batch->block_table, a.q_start = batch->q_start, a.kv_len = batch->kv_len;
    a.part = static_cast<float *>(ws);
    return cache->dtype == PI_KV_F16 ? launch_attn_hd<KvF16, SINKS>(cache->head_dim, a, g, st)
                                     : launch_attn_hd<KvBf16, SINKS>(cache->head_dim, a, g, st);
}

}  // namespace pik
