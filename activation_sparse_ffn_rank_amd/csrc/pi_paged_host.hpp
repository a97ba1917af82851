// pi_paged_host.hpp -- argument checks shared by the host sides of the paged-cache calls.
#pragma once

#include <stdint.h>

#include "pi_paged_kv.h"

namespace pik {

constexpr int kMaxHeads = 1024;
constexpr int kCus = 256;

inline bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// log2 of a page size, or -1.
inline int page_log(int32_t page) {
    switch (page) {
        case 16: return 4;
        case 32: return 5;
        case 64: return 6;
        case 128: return 7;
        case 256: return 8;
        default: return -1;
    }
}

inline int check_cache(const pi_kv_cache *c) {
    if (!c || !c->k_pages || !c->v_pages) return PI_ERR_NULL;
    if (c->dtype != PI_KV_F16 && c->dtype != PI_KV_BF16) return PI_ERR_DTYPE;
    if (page_log(c->page) < 0 || c->n_pages < 1 || c->n_kv < 1 || c->n_kv > kMaxHeads) return PI_ERR_SHAPE;
    if (c->head_dim != 64 && c->head_dim != 128 && c->head_dim != 256) return PI_ERR_SHAPE;
    if ((int64_t)c->n_pages * c->page > INT32_MAX) return PI_ERR_SHAPE;
    if (!aligned16(c->k_pages) || !aligned16(c->v_pages)) return PI_ERR_ALIGN;
    return PI_OK;
}

inline int check_batch(const pi_kv_batch *b) {
    if (!b || !b->block_table || !b->q_start || !b->kv_len) return PI_ERR_NULL;
    if (b->n_req < 1 || b->n_req > PI_KV_MAX_REQ || b->max_pages < 1 || b->max_pages > PI_KV_MAX_TABLE ||
        b->table_stride < b->max_pages || b->max_q < 1 || b->max_q > PI_KV_MAX_TOKENS || b->max_kv < 0)
        return PI_ERR_SHAPE;
    return PI_OK;
}

inline int check_rows(const pi_kv_cache *c, int32_t total_q, int32_t n_q) {
    if (total_q < 0 || total_q > PI_KV_MAX_TOKENS || n_q < 1 || n_q > kMaxHeads || n_q % c->n_kv != 0) return PI_ERR_SHAPE;
    return PI_OK;
}

// Rows of [n][heads][head_dim] with strides in elements: 16-byte rows.
inline int check_strides(const void *p, int64_t ts, int64_t hs) {
    if (ts < 0 || hs < 0) return PI_ERR_SHAPE;
    if (!aligned16(p) || ts % 8 != 0 || hs % 8 != 0) return PI_ERR_ALIGN;
    return PI_OK;
}

// Whether two of the rows [hd] at t * ts + h * hs, t < n, h < heads, share an element.
inline bool rows_overlap(int64_t ts, int64_t hs, int n, int heads, int hd) {
    if ((n > 1 && ts < hd) || (heads > 1 && hs < hd)) return true;
    if (n < 2 || heads < 2) return false;
    if (ts / hs >= heads) return false;              // whole tokens after one another
    for (int h = 1; h < heads; ++h) {                // a row h heads on, and the nearest ones t tokens on
        const __int128 x = (__int128)h * hs, t = x / ts;
        if ((t < n && x - t * ts < hd) || (t + 1 < n && (t + 1) * ts - x < hd)) return true;
    }
    return false;
}

}  // namespace pik
