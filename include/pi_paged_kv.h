/*
 * pi_paged_kv.h -- C ABI of the paged key/value cache and the attention that reads it, for MI355X
 * (gfx950): the attention side of a decode or prefill step whose FFN side is pi_sparse_ffn.h.
 *
 * Keys and values of all running requests live in one pool of pages of `page` token positions each:
 *   k_pages [n_pages][n_kv][page][head_dim]      v_pages [n_pages][n_kv][head_dim][page]
 * (V is held transposed inside a page, so that both products of attention read their operands along
 * the contraction).  block_table [n_req][max_pages] names, per request, the page of positions
 * [c*page, (c+1)*page).  A slot is page_id*page + offset.  A step is
 *   pi_kv_step    lengths -> block tables, slot map, packed row starts, key counts
 *   pi_kv_append  the step's new keys and values into their slots
 *   pi_kv_attn    attention of the step's new tokens over the pages
 *
 * Attention of one request with n new tokens and m = kv_len keys (the new ones included): its token
 * i (0 <= i < n) stands at position p = m - n + i and sees the keys j with
 *   j <= p,   and   j > p - window when window > 0.
 * Query head h reads kv head h / (n_q / n_kv).  With s_j = scale * q . k_j over the keys seen,
 *   out = sum_j exp(s_j - max s) v_j / sum_j exp(s_j - max s),
 * and zero for a token that sees no key (m = 0, or p < 0), or whose scores are all -infinity.  What
 * keys and values that a token does not see hold (infinities and NaN included) has no effect on its
 * output.
 *
 * Conventions are those of pi_sparse_ffn.h: device memory owned by the caller, work only enqueued on
 * `stream`, arguments checked on the host before any HIP call, nothing enqueued on a nonzero return
 * except PI_ERR_HIP, no memset nodes (the calls may be captured into a HIP graph; lengths, tables
 * and slots are read on the device at replay).  The contents of the integer arrays are checked on
 * the device: an entry out of range never makes a kernel read or write outside the arrays, and what
 * it means instead is said at each call.
 */
#ifndef PI_PAGED_KV_H
#define PI_PAGED_KV_H

#include "pi_sparse_ffn.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum { PI_KV_F16 = 1, PI_KV_BF16 = 2 } pi_kv_dtype;

#define PI_KV_MAX_REQ 4096
#define PI_KV_MAX_TABLE (1 << 17)    /* pages of one request */
#define PI_KV_MAX_TOKENS (1 << 19)   /* packed tokens of a step */

/* The pool of pages.  head_dim: 64, 128 or 256; page: 16, 32, 64, 128 or 256 positions; n_pages *
 * page < 2^31 slots.  Both arrays contiguous and 16-byte aligned. */
typedef struct pi_kv_cache {
    int32_t n_pages, n_kv, page, head_dim;
    int32_t dtype;               /* pi_kv_dtype of keys, values, queries and outputs */
    void *k_pages;               /* [n_pages][n_kv][page][head_dim] */
    void *v_pages;               /* [n_pages][n_kv][head_dim][page] */
} pi_kv_cache;

/* The requests of one step.  Rows q_start[r] .. q_start[r+1]-1 of the packed queries are request r's
 * new tokens.  max_q and max_kv bound the lengths on the host (they choose kernels and grids): a
 * request's new tokens past max_q and keys past max_kv are not read, nor keys past max_pages*page.
 * A table entry outside [0, n_pages) is a page without keys.  A request whose q_start range is
 * negative, decreasing or past the packed rows is left out, and of ranges that overlap some may be, or some
 * of their rows. */
typedef struct pi_kv_batch {
    int32_t n_req, max_pages, max_q, max_kv;
    int64_t table_stride;          /* entries from one request's table row to the next, >= max_pages */
    const int32_t *block_table;    /* [n_req][max_pages] */
    const int32_t *q_start;        /* [n_req + 1] */
    const int32_t *kv_len;         /* [n_req] keys of the request, its new tokens included */
} pi_kv_batch;

/* One step of the block tables.  In: cached [n_req] positions held, fresh [n_req] new tokens of this
 * step (0: none; -1 or less: the request has ended), the free pages as a ring (pool[1] of them from
 * free_ring[pool[0] % n_pages] on).  In and out: block_table, free_ring.  Out: the rest.  Requests
 * are served in order:
 *  - an ended one gives its ceil(cached / page) pages back behind the free ones (they are handed out
 *    from the next step on), with kv_len = cached_next = 0 and no tokens;
 *  - the others take rows q_start[r] .. q_start[r+1]-1 (row starts are clamped to max_tokens) and,
 *    for positions cached .. cached + fresh - 1, pages from the front of the ring as needed; their
 *    kv_len and cached_next are cached + fresh, and slots holds each row's slot.  One that does not
 *    fit its table row, the max_tokens rows or the free pages is refused: it keeps its rows with
 *    slot -1, its pages and cached_next = cached, and kv_len = 0 (attention gives its rows zeros).
 *    The pages that it asked for count against later requests of the step too.
 *  - rows past the last request's have slot -1.
 * pool_next = {head, count} of the ring after the step; counts = {rows, pages taken, pages given
 * back, requests refused}.  cached outside [0, max_pages*page] is refused, and gives nothing back.
 * cached_next may be cached and pool_next may be pool, itself in both cases (the step then advances
 * its own state, as a replayed graph does); no other arrays may overlap. */
typedef struct pi_kv_tables {
    int32_t n_req, page, n_pages, max_pages, max_tokens;
    int64_t table_stride;
    const int32_t *cached, *fresh;   /* [n_req] */
    int32_t *free_ring;              /* [n_pages] */
    const int32_t *pool;             /* [2] */
    int32_t *block_table;            /* [n_req][max_pages] */
    int32_t *q_start;                /* [n_req + 1] */
    int32_t *kv_len, *cached_next;   /* [n_req] */
    int32_t *slots;                  /* [max_tokens] */
    int32_t *pool_next;              /* [2] */
    int32_t *counts;                 /* [4] */
} pi_kv_tables;

int pi_kv_step(const pi_kv_tables *t, void *stream);

/* k, v: [n_tokens][n_kv][head_dim] with strides in elements between tokens and between heads
 * (multiples of 8; rows 16-byte aligned), so slices of a fused projection's output are taken as they
 * are.  Row t goes to slots[t]; a slot outside [0, n_pages*page) is skipped.  Valid slots must be
 * distinct.  n_tokens = 0 does nothing. */
int pi_kv_append(const pi_kv_cache *cache, const void *k, int64_t k_token_stride, int64_t k_head_stride,
                 const void *v, int64_t v_token_stride, int64_t v_head_stride, const int32_t *slots,
                 int32_t n_tokens, void *stream);

/* q, out: [total_q][n_q][head_dim], strides in elements (multiples of 8, rows 16-byte aligned); n_q a
 * multiple of n_kv; window 0 = all keys; scale finite and above zero.  Rows of q may overlap, rows of
 * out may not, nor out an input.  Rows that belong to no request are not written.  The
 * workspace (16-byte aligned, no zero fill) holds the partial sums of long key ranges; the size call
 * returns 0 on invalid arguments.  Results do not depend on timing (fixed summation orders). */
size_t pi_kv_attn_workspace_bytes(const pi_kv_cache *cache, const pi_kv_batch *batch, int32_t total_q, int32_t n_q);
int pi_kv_attn(const pi_kv_cache *cache, const pi_kv_batch *batch, const void *q, int64_t q_token_stride,
               int64_t q_head_stride, void *out, int64_t out_token_stride, int64_t out_head_stride,
               int32_t total_q, int32_t n_q, float scale, int32_t window, void *ws, size_t ws_bytes, void *stream);

#ifdef __cplusplus
}
#endif
#endif /* PI_PAGED_KV_H */
