// pi_paged_rope.hip -- host side of pi_kv_rope_append and pi_rope_frequencies (include/pi_paged_kv.h).
#include "pi_paged_host.hpp"
#include "pi_paged_rope.hpp"

#include <algorithm>
#include <cmath>

namespace {

using namespace pik;

int check_rope(const pi_kv_cache *c, const pi_kv_rope *r) {
    if (!r) return PI_ERR_NULL;
    if (r->rot_dim < 0 || r->rot_dim > c->head_dim || r->rot_dim % 16 != 0) return PI_ERR_SHAPE;
    if (r->layout != PI_ROPE_HALF && r->layout != PI_ROPE_PAIRS) return PI_ERR_DTYPE;
    if (r->rot_dim > 0 && !r->freq) return PI_ERR_NULL;
    if (!std::isfinite(r->scale) || !std::isfinite(r->eps) || r->eps < 0.f) return PI_ERR_SHAPE;
    if (!r->norm && (r->q_weight || r->k_weight)) return PI_ERR_DTYPE;
    if (reinterpret_cast<uintptr_t>(r->freq) % 8 != 0 || !aligned16(r->q_weight) || !aligned16(r->k_weight)) return PI_ERR_ALIGN;
    return PI_OK;
}

template <class T, int HD>
void launch(const KvRopeArgs &a, bool pairs, dim3 grid, hipStream_t st) {
    const size_t lds = std::max<size_t>(a.v_tile * (HD / 2 + 1), 4 * HD) * sizeof(uint32_t);
    if (pairs) hipLaunchKernelGGL((k_kv_rope<T, HD, true>), grid, dim3(256), lds, st, a);
    else hipLaunchKernelGGL((k_kv_rope<T, HD, false>), grid, dim3(256), lds, st, a);
}
template <class T>
void launch_hd(int hd, const KvRopeArgs &a, bool pairs, dim3 grid, hipStream_t st) {
    if (hd == 64) launch<T, 64>(a, pairs, grid, st);
    else if (hd == 128) launch<T, 128>(a, pairs, grid, st);
    else launch<T, 256>(a, pairs, grid, st);
}

}  // namespace

extern "C" int pi_rope_frequencies(int32_t rot_dim, double base, double factor, double trained, double low, double high,
                                   double *freq) {
    if (!freq) return PI_ERR_NULL;
    auto positive = [](double x) { return std::isfinite(x) && x > 0.0; };
    if (rot_dim < 2 || rot_dim > 256 || rot_dim % 2 != 0 || !positive(base) || !positive(factor) || !positive(trained) ||
        !std::isfinite(low) || !std::isfinite(high) || low < 0.0 || !(high > low || (low == 0.0 && high == 0.0)))
        return PI_ERR_SHAPE;
    for (int i = 0; i < rot_dim / 2; ++i) {
        const double b = std::pow(base, -2.0 * i / rot_dim), turns = trained * b / 6.283185307179586;
        const double keep = high > low ? std::min(std::max((turns - low) / (high - low), 0.0), 1.0) : 0.0;
        freq[i] = b * (keep + (1.0 - keep) / factor);
    }
    return PI_OK;
}

extern "C" int pi_kv_rope_append(const pi_kv_cache *cache, const pi_kv_batch *batch, const pi_kv_rope *rope, const void *q,
                                 int64_t q_token_stride, int64_t q_head_stride, const void *k, int64_t k_token_stride,
                                 int64_t k_head_stride, const void *v, int64_t v_token_stride, int64_t v_head_stride,
                                 const int32_t *slots, void *q_out, int64_t out_token_stride, int64_t out_head_stride,
                                 int32_t total_q, int32_t n_q, void *stream) {
    int rc = check_cache(cache);
    if (rc || (rc = check_batch(batch)) || (rc = check_rope(cache, rope))) return rc;
    if ((rc = check_rows(cache, total_q, n_q))) return rc;
    if (total_q == 0) return PI_OK;
    if (!q || !k || !v || !slots || !q_out) return PI_ERR_NULL;
    if ((rc = check_strides(q, q_token_stride, q_head_stride)) || (rc = check_strides(k, k_token_stride, k_head_stride)) ||
        (rc = check_strides(v, v_token_stride, v_head_stride)) || (rc = check_strides(q_out, out_token_stride, out_head_stride)))
        return rc;
    if (rows_overlap(out_token_stride, out_head_stride, total_q, n_q, cache->head_dim)) return PI_ERR_SHAPE;
    if (q_out == q && ((total_q > 1 && out_token_stride != q_token_stride) || (n_q > 1 && out_head_stride != q_head_stride)))
        return PI_ERR_SHAPE;
    KvRopeArgs a{};
    a.n_req = batch->n_req, a.total_q = total_q, a.n_q = n_q, a.n_kv = cache->n_kv, a.page_log = page_log(cache->page);
    a.n_slots = cache->n_pages * cache->page, a.rot = rope->rot_dim, a.norm = rope->norm != 0;
    a.scale = rope->scale, a.eps = rope->eps, a.freq = rope->freq;
    a.q_weight = static_cast<const uint16_t *>(rope->q_weight), a.k_weight = static_cast<const uint16_t *>(rope->k_weight);
    a.q_ts = q_token_stride, a.q_hs = q_head_stride, a.k_ts = k_token_stride, a.k_hs = k_head_stride;
    a.v_ts = v_token_stride, a.v_hs = v_head_stride, a.o_ts = out_token_stride, a.o_hs = out_head_stride;
    a.q = static_cast<const uint16_t *>(q), a.k = static_cast<const uint16_t *>(k), a.v = static_cast<const uint16_t *>(v);
    a.slots = slots, a.q_start = batch->q_start, a.kv_len = batch->kv_len;
    a.q_out = static_cast<uint16_t *>(q_out), a.k_pages = static_cast<uint16_t *>(cache->k_pages);
    a.v_pages = static_cast<uint16_t *>(cache->v_pages);
    // A wave per token and round of heads, until there are many: then up to four rounds one after another for the angles' sake
    // (4096 tokens of 24 rounds: 139 us with one, 124.7 two, 123.2 four, 128 eight).
    const int side = 64 / (cache->head_dim / 16), rounds = (n_q + a.n_kv + side - 1) / side;
    a.per_wave = 1;
    while (a.per_wave < 4 && (int64_t)total_q * rounds > (int64_t)a.per_wave * 8192) a.per_wave *= 2;
    a.parts = (rounds + a.per_wave - 1) / a.per_wave;
    // values: tiles as of pi_kv_append
    a.v_tile = (int64_t)((total_q + 63) / 64) * cache->n_kv >= 2 * kCus ? 64 : 16;
    a.v_groups = (total_q + a.v_tile - 1) / a.v_tile * a.n_kv;
    const int64_t waves = (int64_t)total_q * a.parts;
    const dim3 grid((uint32_t)(a.v_groups + (waves + 3) / 4));
    hipStream_t st = static_cast<hipStream_t>(stream);
    const bool pairs = rope->layout == PI_ROPE_PAIRS;
    if (cache->dtype == PI_KV_F16) launch_hd<KvF16>(cache->head_dim, a, pairs, grid, st);
    else launch_hd<KvBf16>(cache->head_dim, a, pairs, grid, st);
    return hipGetLastError() == hipSuccess ? PI_OK : PI_ERR_HIP;
}
