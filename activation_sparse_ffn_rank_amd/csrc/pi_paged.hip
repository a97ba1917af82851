// pi_paged.hip -- host side of the C ABI declared in include/pi_paged_kv.h: argument checks, the
// choice of kernel and grid, launches.  As in pi_abi.hip nothing here allocates, frees, synchronizes
// or issues memset/memcpy nodes, and no C++ exception crosses the ABI.
#include "pi_paged_launch.hpp"

#include <algorithm>

namespace {

using namespace pik;

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
    return attn_plan(cache, batch, total_q, n_q, batch->max_kv, false).bytes;
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
    return run_attn<false>(cache, batch, q, q_token_stride, q_head_stride, out, out_token_stride, out_head_stride, total_q, n_q,
                           scale, window, 0, batch->max_kv, false, ws, ws_bytes, static_cast<hipStream_t>(stream));
}
