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
 * Around it: pi_kv_rope_append (the append with rotary positions and head norms), pi_kv_attn_sinks (attention over a window
 * and the first tokens), pi_kv_verify (which drafted tokens stay), pi_kv_release, pi_kv_fork and pi_kv_copy (pages given back,
 * shared and copied).
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

/* ---- rotary positions and head norms with the append ----
 *
 * Frequencies of rotary positions, in radians per position: freq[i] = f_i, i < rot_dim / 2, with
 *   b_i = base^(-2 i / rot_dim),   t_i = trained * b_i / (2 pi)   (turns over the trained positions),
 *   g_i = min(max((t_i - low) / (high - low), 0), 1),             f_i = b_i (g_i + (1 - g_i) / factor).
 * factor 1 gives b_i; low = high = 0 divides all of them by factor (positions interpolated evenly); otherwise those of
 * fewer than `low` turns are divided and those of more than `high` kept.  rot_dim: even, 2 to 256; base, factor, trained
 * finite and above zero, 0 <= low < high (or both 0).  freq is HOST memory; synchronous. */
int pi_rope_frequencies(int32_t rot_dim, double base, double factor, double trained, double low, double high, double *freq);

/* Which elements of a head form pairs: i and i + rot_dim/2, or 2i and 2i + 1. */
typedef enum { PI_ROPE_HALF = 0, PI_ROPE_PAIRS = 1 } pi_rope_layout;

/* What is done to a head x of q and k.  With norm != 0 first x <- x / sqrt(mean(x^2) + eps) * weight over all of its
 * head_dim elements (a weight of NULL: ones; weights in the cache's element type, 16-byte aligned).  Then the pairs (a, b) of its
 * first rot_dim elements (a multiple of 16, at most head_dim; 0: none) become scale * (a cos - b sin, a sin + b cos) of the
 * angle position * freq[i]; the other elements stay.  All in fp32 (angles reduced in fp64), rounded once.  eps >= 0 and
 * scale are finite. */
typedef struct pi_kv_rope {
    int32_t rot_dim, layout, norm;
    float scale, eps;
    const double *freq;              /* [rot_dim / 2] radians per position, device memory */
    const void *q_weight, *k_weight; /* [head_dim] each, or NULL */
} pi_kv_rope;

/* pi_kv_append of new keys turned as `rope` says and of new values, and the step's queries turned the same way to q_out, in
 * one pass.  Row q_start[r] + i of the packed rows stands at position kv_len[r] - n + i (of batch, max_q and max_kv bound
 * nothing here and the table is not read).  Rows that belong to no request are left alone: not appended, q_out not written.
 * q_start must not decrease (rows of ranges that do may be left out, query, key and value together).  Slots, strides and
 * pointers are as in pi_kv_append and pi_kv_attn; q_out may be q itself with the same strides, and overlaps no other argument.
 * total_q = 0 does nothing. */
int pi_kv_rope_append(const pi_kv_cache *cache, const pi_kv_batch *batch, const pi_kv_rope *rope, const void *q,
                      int64_t q_token_stride, int64_t q_head_stride, const void *k, int64_t k_token_stride,
                      int64_t k_head_stride, const void *v, int64_t v_token_stride, int64_t v_head_stride,
                      const int32_t *slots, void *q_out, int64_t out_token_stride, int64_t out_head_stride, int32_t total_q,
                      int32_t n_q, void *stream);

/* ---- attention over a window and the first tokens ----
 *
 * pi_kv_attn in which the first `sinks` keys of a request stay visible: the token at position p sees the keys j with
 *   j <= p  and  (j > p - window  or  j < sinks).
 * sinks >= 0 (0: pi_kv_attn with this window), window > 0 with sinks.  Pages between the first tokens and the windows of a step's tokens
 * are not read: their table entries may be out of range (pi_kv_release).  All else, the workspace included, is as in
 * pi_kv_attn; its size depends on window and sinks.  Keys are taken as they were appended: positions that pi_kv_rope_append
 * gave the first tokens stay theirs, and the distance to them grows with the request. */
size_t pi_kv_attn_sinks_workspace_bytes(const pi_kv_cache *cache, const pi_kv_batch *batch, int32_t total_q, int32_t n_q,
                                        int32_t window, int32_t sinks);
int pi_kv_attn_sinks(const pi_kv_cache *cache, const pi_kv_batch *batch, const void *q, int64_t q_token_stride,
                     int64_t q_head_stride, void *out, int64_t out_token_stride, int64_t out_head_stride, int32_t total_q,
                     int32_t n_q, float scale, int32_t window, int32_t sinks, void *ws, size_t ws_bytes, void *stream);

/* ---- drafted tokens ----
 *
 * A step whose requests carry their last token and then their drafts (rows q_start[r] .. q_start[r+1]-1 of the packed
 * tokens) gives the target's probabilities of what follows each row.  The draft in row t + 1, x = tokens[t + 1], is accepted if
 *   u_accept[t] * q[t][x] < p[t][x]
 * and all drafts before it are; q is the distribution that it was drawn from (NULL: all of it on x).  With a the number
 * accepted of n - 1 drafts and t = q_start[r] + a the row after them, the next token is drawn from the weights
 *   w_j = max(p[t][j] - q[t][j], 0)  if a draft was rejected,   w_j = max(p[t][j], 0)  if none was (or the former are all 0)
 * as the first j with w_0 + .. + w_j > u_next[r] * (w_0 + w_1 + ..) -- which leaves every token with the target's
 * probability.  Products, differences and sums are in 64 bits; a NaN counts as a weight of 0 and rejects; where no j passes (u_next
 * at or above 1) it is the last one with a weight above 0.  tokens outside [0, vocab) are rejected, and have no part of w.
 * accepted [n_req] = a; next [n_req], -1 if all weights are 0 or the request has no rows (q_start negative,
 * decreasing or past `rows` included); keep [n_req], with kv_len the keys of the step's attention, = kv_len - (n - 1 - a), the
 * positions that stay (pi_kv_release's drop_from).
 * A request that pi_kv_step refused (kv_len 0, or fewer keys than rows) holds none of its rows, and attention gave them zeros:
 * a = 0, next = its own last token tokens[q_start[r]], so that the next step asks for the same again (-1 if it has no rows), and
 * keep = INT32_MAX, which as drop_from drops nothing; it is no length (those behind the step are pi_kv_release's
 * cached_next).  Without kv_len such a request is taken for one that was served.
 * kv_len and keep: both or neither NULL, and keep may be kv_len. */
#define PI_KV_MAX_VOCAB (1 << 22)
typedef struct pi_kv_drafts {
    int32_t n_req, rows, vocab;
    const int32_t *q_start;          /* [n_req + 1] */
    const int32_t *tokens;           /* [rows] */
    const float *target;             /* [rows][vocab] p, row stride in elements, 4-byte aligned */
    int64_t target_stride;
    const float *draft;              /* [rows][vocab] q or NULL; the last row of a request is not read */
    int64_t draft_stride;
    const float *u_accept;           /* [rows], in [0, 1); the last one of a request is not read */
    const float *u_next;             /* [n_req], in [0, 1) */
} pi_kv_drafts;

/* The workspace is 16-byte aligned and zero-filled before the first call that uses it; each call leaves it ready for the next
 * one, of any size (never clear or share it while a call is in flight).  Results do not depend on timing. */
size_t pi_kv_verify_workspace_bytes(const pi_kv_drafts *drafts);
int pi_kv_verify(const pi_kv_drafts *drafts, const int32_t *kv_len, int32_t *accepted, int32_t *next, int32_t *keep, void *ws,
                 size_t ws_bytes, void *stream);

/* ---- pages given back, shared and copied ----
 *
 * Requests may share pages: shares[p] counts the owners of page p beyond the first (0 for a page that pi_kv_step hands out,
 * which knows nothing of shares).  Only full pages are shared, so appends never touch one.  A request that
 * shares pages, or has given pages back from its middle, ends by pi_kv_release (drop_from 0), not by fresh < 0 of pi_kv_step.
 *
 * The state is pi_kv_step's: pages of positions below cached[r] in block_table, the free ones in the ring.  Both calls judge
 * it as it stands before them.  cached_next may be cached and pool_next may be pool, itself in both cases; no other arrays may
 * overlap. */
typedef struct pi_kv_pages {
    int32_t n_req, page, n_pages, max_pages;
    int64_t table_stride;
    const int32_t *cached;           /* [n_req] */
    int32_t *free_ring;              /* [n_pages] */
    const int32_t *pool;             /* [2] */
    int32_t *block_table;            /* [n_req][max_pages] */
    int32_t *shares;                 /* [n_pages] */
    int32_t *cached_next;            /* [n_req] */
    int32_t *pool_next;              /* [2] */
    int32_t *counts;                 /* [4] */
    void *ws;                        /* pi_kv_pages_workspace_bytes, 16-byte aligned, no zero fill (pi_kv_release) */
    size_t ws_bytes;
} pi_kv_pages;

/* Bytes of workspace for this state (0: invalid).  It must not be shared by calls in flight at the same time. */
size_t pi_kv_pages_workspace_bytes(const pi_kv_pages *pages);

/* Gives up the positions drop_from[r] .. drop_to[r]-1 of every request (drop_to NULL: to the end; a negative drop_from is 0;
 * none where drop_from >= cached): the pages all of whose held positions lie among them.
 *  - drop_to >= cached cuts the request: cached_next = drop_from (what its table holds past that is void).  If that lies inside
 *    a page with further owners, the request gives up that page too and takes a free one in its place: copies[r] = {old, new}
 *    (pi_kv_copy makes the copy, before the next append), else {-1, -1}.  Such a request is refused, and nothing of it
 *    changes, if the free pages do not suffice; requests are served in order.
 *  - drop_to < cached drops from the middle: cached_next = cached, the dropped entries become -1 (pages without keys).
 *    What a window has passed goes this way: drop_from = the first tokens that stay, drop_to = min(c - window + 1, c - 1) of a
 *    request of c positions whose next token stands at position c, so that it ends below c with a window of one token too.
 *    The columns stay used, so a request holds at most max_pages * page positions, dropped ones included; tokens appended to
 *    a dropped page (after a cut back into it) have no slot.
 * A page given up once more than it has further owners goes behind the free ones, in the order of first mention (requests in order,
 * a page given up for a copy before the later ones); entries outside [0, n_pages) are skipped.  cached outside [0, max_pages * page]
 * is refused.  counts = {entries given up, pages gone back, pages taken, requests refused}. */
int pi_kv_release(const pi_kv_pages *pages, const int32_t *drop_from, const int32_t *drop_to, int32_t *copies, void *stream);

/* Makes request dst[i], which must hold nothing (cached 0), a copy of request src[i], i < n_fork: its full pages are shared, of
 * a partly filled last one a copy is due: copies[i] = {old, new}, else {-1, -1}.  Refused, with nothing changed: src or dst out
 * of range or equal, dst holding something or named by an earlier fork, cached[src] out of range, free pages that do not suffice
 * (forks are served in order).  cached_next = cached but for the forks.  counts = {forks made, entries shared
 * (missing pages among them), pages taken, forks refused}.  0 <= n_fork <= PI_KV_MAX_REQ. */
int pi_kv_fork(const pi_kv_pages *pages, const int32_t *src, const int32_t *dst, int32_t n_fork, int32_t *copies, void *stream);

/* Copies keys and values of page copies[i][0] to page copies[i][1], i < n.  Pairs with an entry out of range are skipped; no
 * destination may be named twice or be a source. */
int pi_kv_copy(const pi_kv_cache *cache, const int32_t *copies, int32_t n, void *stream);

#ifdef __cplusplus
}
#endif
#endif /* PI_PAGED_KV_H */
