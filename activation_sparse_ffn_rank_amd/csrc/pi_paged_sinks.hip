// pi_paged_sinks.hip -- host side of pi_kv_attn_sinks (include/pi_paged_kv.h): attention over a window and the first tokens.
#include "pi_paged_launch.hpp"

namespace {

using namespace pik;

// Keys that a request's axis has at most: the first ones in whole blocks of 64, the window of every new token, and the window's
// own rounding down to a block.  Kernel and pieces are chosen by these, not by the length of the request.
int most_keys(const pi_kv_batch *b, int32_t window, int32_t sinks) {
    const int64_t keys = ((int64_t)sinks + 63) / 64 * 64 + window + b->max_q - 1 + 63;
    return (int)std::min<int64_t>(keys, b->max_kv);
}

// Of requests of up to twice as many keys as they read or more, most read that many.
bool even_ranges(const pi_kv_batch *b, int32_t window, int32_t sinks) { return b->max_kv / 2 >= most_keys(b, window, sinks); }

int check_window(int32_t window, int32_t sinks) {
    return window < 0 || sinks < 0 || (window == 0 && sinks > 0) ? PI_ERR_SHAPE : PI_OK;
}

}  // namespace

extern "C" size_t pi_kv_attn_sinks_workspace_bytes(const pi_kv_cache *cache, const pi_kv_batch *batch, int32_t total_q, int32_t n_q,
                                                   int32_t window, int32_t sinks) {
    if (sinks == 0 && window >= 0) return pi_kv_attn_workspace_bytes(cache, batch, total_q, n_q);
    if (check_cache(cache) || check_batch(batch) || check_rows(cache, total_q, n_q) || check_window(window, sinks)) return 0;
    return attn_plan(cache, batch, total_q, n_q, most_keys(batch, window, sinks), even_ranges(batch, window, sinks)).bytes;
}

extern "C" int pi_kv_attn_sinks(const pi_kv_cache *cache, const pi_kv_batch *batch, const void *q, int64_t q_token_stride,
                                int64_t q_head_stride, void *out, int64_t out_token_stride, int64_t out_head_stride,
                                int32_t total_q, int32_t n_q, float scale, int32_t window, int32_t sinks, void *ws,
                                size_t ws_bytes, void *stream) {
    if (sinks == 0)
        return pi_kv_attn(cache, batch, q, q_token_stride, q_head_stride, out, out_token_stride, out_head_stride, total_q, n_q,
                          scale, window, ws, ws_bytes, stream);
    int rc = check_cache(cache);
    if (rc || (rc = check_batch(batch))) return rc;
    if ((rc = check_rows(cache, total_q, n_q)) || (rc = check_window(window, sinks))) return rc;
    if (total_q == 0) return PI_OK;
    if (!q || !out) return PI_ERR_NULL;
    if (!(scale > 0.f) || !std::isfinite(scale)) return PI_ERR_SHAPE;
    return run_attn<true>(cache, batch, q, q_token_stride, q_head_stride, out, out_token_stride, out_head_stride, total_q, n_q,
                          scale, window, sinks, most_keys(batch, window, sinks), even_ranges(batch, window, sinks), ws, ws_bytes,
                          static_cast<hipStream_t>(stream));
}
