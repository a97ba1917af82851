// pi_paged.hpp -- gfx950 kernels of the paged key/value cache: block tables (k_kv_tables), cache
// append (k_kv_append) and attention over the pages (k_kv_rows for few query rows, k_kv_tile for many,
// k_kv_join), with the first tokens of a request in sight or not (SINKS).
//
// Both products of attention run on MFMA with the keys along the rows of the first one,
//   S^T = K Q^T   (A = K: 16 keys x 32 head dims, B = Q^T: 32 head dims x 16 query rows)
//   O^T = V^T P^T (A = V^T: 16 head dims x 32 keys, B = P^T: 32 keys x 16 query rows),
// so a lane holds scores and outputs of one query row only (row = lane % 16): the running maximum
// and sum of the softmax, and every rescaling, are per-lane numbers.  The result of the first product
// is the operand of the second one as it stands when the 32 keys of a block go to the two 16-key
// tiles in this order: tile u, tile row 4a + b holds key 8a + 4u + b.  Lane group g = lane / 16 then
// holds keys 8g .. 8g+7 of its row, which is the B operand's order, and V^T, held transposed in the
// pages, is read 16 bytes (8 keys) per lane.  No value crosses lanes through LDS.
#pragma once

#include "pi_kernels.hpp"
#include "pi_paged_kv.h"

namespace pik {

// ------------------------------------------------------------------------------ element types

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

struct KvF16 {
    typedef f16 e;
    typedef f16 v2 __attribute__((ext_vector_type(2)));
    typedef f16 v8 __attribute__((ext_vector_type(8)));
    static constexpr uint32_t kExpMask = 0x7c007c00u;   // exponent bits: all ones = infinity or NaN
    // Weights are held as exp2(s - max + 8): fp16 keeps 8 more binary orders below the largest
    // weight before it rounds to subnormals; the factor is in the row's sum too and divides out.
    static constexpr float kShift = 8.f;
    // The reference may lag the true maximum by this many powers of two (weights stay <= 2^14 < 65504).
    static constexpr float kLag = 6.f;
    static constexpr float kHead = 1.f - 0x1p-7f;       // of kv_weights
    static __device__ __forceinline__ f32x4 mfma16(uint4 a, uint4 b, f32x4 c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(v8, a), __builtin_bit_cast(v8, b), c, 0, 0, 0);
    }
    static __device__ __forceinline__ f32x16 mfma32(uint4 a, uint4 b, f32x16 c) {
        return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(v8, a), __builtin_bit_cast(v8, b), c, 0, 0, 0);
    }
};

struct KvBf16 {
    typedef __bf16 e;
    typedef __bf16 v2 __attribute__((ext_vector_type(2)));
    typedef __bf16 v8 __attribute__((ext_vector_type(8)));
    static constexpr uint32_t kExpMask = 0x7f807f80u;
    static constexpr float kShift = 0.f;                // bf16 has fp32's exponents
    static constexpr float kLag = 6.f;
    static constexpr float kHead = 1.f - 0x1p-6f;
    static __device__ __forceinline__ f32x4 mfma16(uint4 a, uint4 b, f32x4 c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8, a), __builtin_bit_cast(v8, b), c, 0, 0, 0);
    }
    static __device__ __forceinline__ f32x16 mfma32(uint4 a, uint4 b, f32x16 c) {
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(v8, a), __builtin_bit_cast(v8, b), c, 0, 0, 0);
    }
};

// Two values rounded to the element type (to nearest even), first one in the low half.
template <class T>
__device__ __forceinline__ uint32_t kv_pack(float a, float b) {
    const f32x2 x = {a, b};
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(x, typename T::v2));
}

// Eight weights as the sum of two operands of the element type: most of each, rounded, and the rest, rounded.  The
// rest of a weight above zero is above zero too, down to the type's smallest numbers (the head is short of it by more
// than it was rounded), so that an infinite value times either has its sign.  At most 2^-17 (fp16) or 2^-13 (bf16) of a
// weight is lost, where the type alone loses up to 2^-11 or 2^-8.
template <class T>
__device__ __forceinline__ void kv_weights(const float (&p)[8], uint4 &head, uint4 &rest) {
    uint32_t h[4], r[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float a = p[2 * i], b = p[2 * i + 1];
        h[i] = kv_pack<T>(a * T::kHead, b * T::kHead);
        const typename T::v2 x = __builtin_bit_cast(typename T::v2, h[i]);
        r[i] = kv_pack<T>(a - (float)x[0], b - (float)x[1]);
    }
    head = make_uint4(h[0], h[1], h[2], h[3]);
    rest = make_uint4(r[0], r[1], r[2], r[3]);
}

// ------------------------------------------------------------------------------ block tables

struct KvTablesArgs {
    int n_req, page_log, n_pages, max_pages, max_tokens;
    int64_t table_stride;
    const int *cached, *fresh;
    int *ring;
    const int *pool;
    int *table, *q_start, *kv_len, *cached_next, *slots, *pool_next, *counts;
};

constexpr uint32_t kKvRefused = 0x80000000u, kKvEnded = 0x40000000u, kKvNeed = 0x3fffffffu;
constexpr int kKvTableThreads = 1024;
constexpr int kKvReqPerThread = PI_KV_MAX_REQ / kKvTableThreads;

// Exclusive block scan of v (unsigned, mod 2^32); *total receives the sum.  part: one word per wave.
__device__ __forceinline__ uint32_t kv_block_scan(uint32_t v, uint32_t *part, uint32_t *total) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, waves = blockDim.x >> 6;
    const uint32_t incl = (uint32_t)wave_incl_scan((int)v);
    __syncthreads();                       // part may still be read by the scan before
    if (lane == 63) part[wave] = incl;
    __syncthreads();
    uint32_t before = 0, all = 0;
    for (int w = 0; w < waves; ++w) {
        before += w < wave ? part[w] : 0u;
        all += part[w];
    }
    *total = all;
    return before + incl - v;
}

// The step of the block tables.  Two scans over the requests (rows; then pages taken and pages given
// back) that every workgroup makes for itself from the lengths (at most 32 KB from L2), after which
// the workgroups share out the pages and the rows: nothing waits on another workgroup.  With one
// workgroup all inputs are read before the first output is written, so a step may run in place.
// The row sums stay below 2^32: at most 4096 requests of at most 2^19 + 1 counted rows.  Bound by the
// latency of its few dependent loads: a pass over 64 requests 6.4 us, 1500 with 66 thousand new tokens 9.2 us.  In place
// the one workgroup finds all the slots: the same two take 9 and 119 us, with events around a call alone, and 9 and 12
// with separate outputs.
static __global__ __launch_bounds__(kKvTableThreads) void k_kv_tables(KvTablesArgs a) {
    __shared__ uint32_t s_row[PI_KV_MAX_REQ + 1];   // first row
    __shared__ uint32_t s_need[PI_KV_MAX_REQ];      // pages asked for (ended: given back) by the requests before | flags
    __shared__ uint32_t s_held[PI_KV_MAX_REQ];      // cached
    __shared__ uint32_t s_part[kKvTableThreads / 64];
    __shared__ uint32_t s_taken, s_denied;
    const int tid = threadIdx.x, n = a.n_req;
    const int per = (n + (int)blockDim.x - 1) / (int)blockDim.x;
    const int page = 1 << a.page_log;
    const int64_t room = (int64_t)a.max_pages << a.page_log;
    int head = a.pool[0] % a.n_pages;
    if (head < 0) head += a.n_pages;
    const int count = min(max(a.pool[1], 0), a.n_pages);
    if (tid == 0) s_taken = s_denied = 0;

    int c[kKvReqPerThread], f[kKvReqPerThread];
    uint32_t rows = 0;
#pragma unroll
    for (int k = 0; k < kKvReqPerThread; ++k) {
        const int r = tid * per + k;
        const bool in = k < per && r < n;
        c[k] = in ? a.cached[r] : 0;
        f[k] = in ? a.fresh[r] : 0;
        rows += (uint32_t)min(max(f[k], 0), a.max_tokens + 1);
    }
    uint32_t total_rows, total_need, total_back;
    uint32_t row = kv_block_scan(rows, s_part, &total_rows);
    uint32_t need[kKvReqPerThread], back[kKvReqPerThread], need_sum = 0, back_sum = 0;
    bool fits[kKvReqPerThread];
#pragma unroll
    for (int k = 0; k < kKvReqPerThread; ++k) {
        const int r = tid * per + k;
        const bool in = k < per && r < n;
        if (in) s_row[r] = row;
        row += (uint32_t)min(max(f[k], 0), a.max_tokens + 1);
        const bool bad = c[k] < 0 || c[k] > room;
        const int64_t end = (int64_t)c[k] + f[k];
        const int have = bad ? 0 : (c[k] + page - 1) >> a.page_log;
        fits[k] = in && f[k] >= 0 && !bad && end <= room && row <= (uint32_t)a.max_tokens;
        need[k] = fits[k] ? (uint32_t)(((int)end + page - 1) >> a.page_log) - have : 0u;
        back[k] = in && f[k] < 0 ? (uint32_t)have : 0u;
        need_sum += need[k];
        back_sum += back[k];
    }
    uint32_t nd = kv_block_scan(need_sum, s_part, &total_need);
    uint32_t bk = kv_block_scan(back_sum, s_part, &total_back);
    uint32_t taken = 0, denied = 0;
#pragma unroll
    for (int k = 0; k < kKvReqPerThread; ++k) {
        const int r = tid * per + k;
        if (k >= per || r >= n) continue;
        const bool ended = f[k] < 0;
        const bool ok = fits[k] && (need[k] == 0 || nd + need[k] <= (uint32_t)count);
        s_need[r] = (ended ? bk | kKvEnded : nd) | (ok || back[k] ? 0u : kKvRefused);
        s_held[r] = (uint32_t)c[k];
        if (ok && need[k]) taken = max(taken, nd + need[k]);
        denied += !ended && !ok;
        nd += need[k];
        bk += back[k];
        if (blockIdx.x == 0) {
            a.q_start[r + 1] = (int)min(s_row[r] + (uint32_t)min(max(f[k], 0), a.max_tokens + 1), (uint32_t)a.max_tokens);
            a.kv_len[r] = ok ? c[k] + f[k] : 0;
            a.cached_next[r] = ended ? 0 : ok ? c[k] + f[k] : c[k];
        }
    }
    if (taken) atomicMax(&s_taken, taken);          // whole numbers: any order gives the same result
    if (denied) atomicAdd(&s_denied, denied);
    if (tid == 0) s_row[n] = total_rows;
    __syncthreads();
    if (blockIdx.x == 0 && tid == 0) {
        a.q_start[0] = 0;
        a.pool_next[0] = (int)(((int64_t)head + s_taken) % a.n_pages);
        a.pool_next[1] = (int)min((int64_t)count - s_taken + total_back, (int64_t)a.n_pages);
        a.counts[0] = (int)min(total_rows, (uint32_t)a.max_tokens);
        a.counts[1] = (int)s_taken;
        a.counts[2] = (int)total_back;
        a.counts[3] = (int)s_denied;
    }

    // pages: a wave per request
    const int lane = tid & 63;
    for (int r = blockIdx.x * (blockDim.x >> 6) + (tid >> 6); r < n; r += gridDim.x * (blockDim.x >> 6)) {
        const uint32_t w = s_need[r];
        if (w & kKvRefused) continue;
        int *const row_tab = a.table + (int64_t)r * a.table_stride;
        if (w & kKvEnded) {
            const uint32_t first = w & kKvNeed;
            const int have = ((int)s_held[r] + page - 1) >> a.page_log;
            for (int j = lane; j < have; j += 64)
                a.ring[((int64_t)head + count + first + j) % a.n_pages] = row_tab[j];
            continue;
        }
        const int have = ((int)s_held[r] + page - 1) >> a.page_log;
        const int m = (((int)s_held[r] + (int)(s_row[r + 1] - s_row[r]) + page - 1) >> a.page_log) - have;
        for (int j = lane; j < m; j += 64)
            row_tab[have + j] = a.ring[((int64_t)head + (w & kKvNeed) + j) % a.n_pages];
    }

    // slots: a row per thread, its request by bisection over the first rows
    for (int t = blockIdx.x * blockDim.x + tid; t < a.max_tokens; t += gridDim.x * blockDim.x) {
        int slot = -1;
        if ((uint32_t)t < total_rows) {
            int lo = 0, hi = n;                      // s_row[lo] <= t < s_row[hi]
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (s_row[mid] <= (uint32_t)t) lo = mid;
                else hi = mid;
            }
            const uint32_t w = s_need[lo];
            if (!(w & kKvRefused)) {
                const int pos = (int)s_held[lo] + (int)((uint32_t)t - s_row[lo]);
                const int have = ((int)s_held[lo] + page - 1) >> a.page_log, col = pos >> a.page_log;
                const int id = col < have ? a.table[(int64_t)lo * a.table_stride + col]
                                          : a.ring[((int64_t)head + (w & kKvNeed) + (col - have)) % a.n_pages];
                if (id >= 0 && id < a.n_pages) slot = (id << a.page_log) + (pos & (page - 1));
            }
        }
        a.slots[t] = slot;
    }
}

// ------------------------------------------------------------------------------ cache append

struct KvAppendArgs {
    int n_tokens, n_kv, hd, page_log, n_slots;
    int64_t k_ts, k_hs, v_ts, v_hs;
    const uint16_t *k, *v;
    const int *slots;
    uint16_t *k_pages, *v_pages;
};

// TT tokens of one kv head per workgroup, heads fastest, so that workgroups near one another read whole rows of a
// fused projection and fill whole pages (5000 tokens of 56 heads of 128: 96 us with token tiles fastest, 74
// so).  Keys: 16-byte copies.  Values go through LDS so that a lane stands for a token on the way out: tokens in
// neighbouring slots of a page then store neighbouring 2-byte elements of one V^T row.  (Runs of 8 slots stored as
// 16 bytes were no faster.)  Bound by memory traffic: 4096 tokens of 96 heads of 128, 403 MB, 92 us.
template <int TT>
__global__ __launch_bounds__(256) void k_kv_append(KvAppendArgs a) {
    extern __shared__ uint32_t s_v[];                // [TT][hd/2 + 1]
    const int t0 = blockIdx.y * TT, h = blockIdx.x, tid = threadIdx.x;
    const int nt = min(TT, a.n_tokens - t0);
    const int per = a.hd >> 3, lds_row = (a.hd >> 1) + 1;
    for (int i = tid; i < nt * per; i += 256) {
        const int t = i / per, ch = i - t * per;
        const uint32_t slot = (uint32_t)a.slots[t0 + t];
        if (slot >= (uint32_t)a.n_slots) continue;
        const uint4 kx = ld16(a.k + (t0 + t) * a.k_ts + h * a.k_hs + ch * 8);
        const uint4 vx = ld16(a.v + (t0 + t) * a.v_ts + h * a.v_hs + ch * 8);
        const int64_t pg = slot >> a.page_log, off = slot & ((1u << a.page_log) - 1);
        *reinterpret_cast<uint4 *>(a.k_pages + ((((pg * a.n_kv + h) << a.page_log) + off) * a.hd + ch * 8)) = kx;
        uint32_t *const d = s_v + t * lds_row + ch * 4;
        d[0] = vx.x, d[1] = vx.y, d[2] = vx.z, d[3] = vx.w;
    }
    __syncthreads();
    const int t = tid & (TT - 1);
    if (t >= nt) return;
    const uint32_t slot = (uint32_t)a.slots[t0 + t];
    if (slot >= (uint32_t)a.n_slots) return;
    const int64_t pg = slot >> a.page_log, off = slot & ((1u << a.page_log) - 1);
    uint16_t *const vp = a.v_pages + (((pg * a.n_kv + h) * a.hd) << a.page_log) + off;
    for (int d = tid / TT; d < (a.hd >> 1); d += 256 / TT) {
        const uint32_t w = s_v[t * lds_row + d];
        vp[(int64_t)(2 * d) << a.page_log] = (uint16_t)w;
        vp[(int64_t)(2 * d + 1) << a.page_log] = (uint16_t)(w >> 16);
    }
}

// ------------------------------------------------------------------------------ attention

struct KvAttnArgs {
    int n_pages, n_kv, page_log;
    int n_req, max_pages, max_q, max_kv, total_q, n_q, group, window;
    int sinks;                        // first keys that stay visible (kernels with SINKS; window > 0)
    int split_target;                 // 0: key ranges are not cut
    int slots;                        // split items per kv head that the workspace holds
    int items;                        // items per kv head that the grid has
    float scale_log2;                 // scale / ln 2, > 0: weights are powers of two
    int64_t table_stride, q_ts, q_hs, o_ts, o_hs;
    const uint16_t *k, *v, *q;
    const int *table, *q_start, *kv_len;
    uint16_t *out;
    float *part;                      // per split item of TR rows: weighted sums [TR][HD], reference [TR], sum of weights [TR]
};

// Rows and keys of request r: the rows of one kv head are (token, query head of the group), token
// major; new tokens past max_q and keys past the bounds are left out.
struct KvReq {
    int q0, n, m;          // first packed row, new tokens, keys
    int rows;              // query rows per kv head
    int lo, hi;            // keys that any of its rows may see
    int first;             // SINKS: and the keys [0, first) before lo, whole blocks; 0: lo is 0 or there are none
    __device__ __forceinline__ int keys() const { return first + hi - lo; }
};

// SINKS: the first a.sinks keys stay visible behind the window.  A request's keys are then an axis of two pieces, [0, first)
// and [lo, hi), which is what is cut and shared out; kernels walk it in blocks and step from one piece to the other, so that
// nothing between them is read and no block holds keys of both.  Single tokens of 16 requests, 4 first keys and a window of 4096,
// 32 heads of 128, 1.07 GB: 185 us (5.8 TB/s); a chunk of 4096 tokens, 64 and 2048, the same heads: 178 to 185 us, 780 TFLOP/s of
// products that count, at 36 blocks a tile of which five are masked.
// Blocks of the first keys: 32 for kernels of 16-row tiles (4 first keys and a window of 500: one request of 16 heads of 64 8.3 us
// with 64 and 7.8 with 32, 64 requests of 32 heads of 128 111.6 and 110.7), 64 for wide ones.
constexpr int kKvRowTile = 16;          // query rows of a k_kv_rows workgroup
constexpr int kKvWideTile = 128;        // ... and of a k_kv_tile workgroup
template <int TR>
__device__ __forceinline__ int kv_first_blocks(const KvAttnArgs &a, int hi) {
    constexpr int kBlock = TR == kKvRowTile ? 32 : 64;
    return (min(a.sinks, hi) + kBlock - 1) & ~(kBlock - 1);
}

template <int TR, bool SINKS>
__device__ __forceinline__ KvReq kv_req(const KvAttnArgs &a, int r) {
    KvReq x;
    const int q0 = a.q_start[r], q1 = a.q_start[r + 1];
    x.q0 = q0;
    const bool ok = q0 >= 0 && q1 >= q0 && q1 <= a.total_q;
    x.n = ok ? q1 - q0 : 0;
    x.m = max(a.kv_len[r], 0);
    x.rows = min(x.n, a.max_q) * a.group;
    x.hi = (int)min((int64_t)min(x.m, a.max_kv), (int64_t)a.max_pages << a.page_log);
    x.lo = a.window ? min(max(x.m - x.n - a.window + 1, 0), x.hi) & ~63 : 0;
    x.first = 0;
    if constexpr (SINKS) {
        x.first = kv_first_blocks<TR>(a, x.hi);
        if (x.first >= x.lo) x.lo = x.first = 0;
    }
    return x;
}

// Keys of a row tile in blocks of KT: [a0, a1), then [lo, hi), without those that lie outside the item's piece of the request's
// axis.  tile_lo, tile_hi: the window's keys that some row of the tile sees.  a1 < 0 without SINKS or where the first keys
// run on into the window.
struct KvSpan {
    int a0, a1, lo, hi;
    __device__ __forceinline__ int after(int kb, int step) const { return kb + step == a1 ? lo : kb + step; }
};
template <int TR, bool SINKS, int KT>
__device__ __forceinline__ KvSpan kv_span(const KvAttnArgs &a, const KvReq &q, int tile_lo, int tile_hi, int splits, int split,
                                          int piece) {
    KvSpan x;
    x.a0 = x.a1 = -1;
    x.lo = max(tile_lo & ~(KT - 1), q.lo), x.hi = tile_hi;
    if constexpr (SINKS) {
        const int past = q.lo - q.first, first = kv_first_blocks<TR>(a, q.hi);    // key = place on the axis + past, in [lo, hi)
        const bool apart = x.lo - past > first && tile_hi > 0;
        if (apart) x.a0 = 0, x.a1 = first;
        else x.lo = q.first ? q.lo : 0;
        // (not apart: either the tile's window begins at the request's, which follows the first keys on the axis, or all of it
        // is one piece from key 0)
        if (!apart && q.first && tile_hi > 0) x.a0 = 0, x.a1 = q.first;
        if (splits > 1) {
            const int from = split * piece, to = from + piece;
            if (x.a1 >= 0) x.a0 = max(x.a0, from), x.a1 = min(x.a1, to);
            x.lo = max(x.lo, from + past), x.hi = min(x.hi, to + past);
            if (x.a1 >= 0 && x.a0 >= x.a1) x.a0 = x.a1 = -1;
        }
        if (x.a1 >= 0 && x.hi <= x.lo) x.lo = x.a0, x.hi = x.a1, x.a0 = x.a1 = -1;
    } else if (splits > 1) {
        const int from = q.lo + split * piece;
        x.lo = max(x.lo, from);
        x.hi = min(x.hi, from + piece);
    }
    return x;
}

constexpr int kKvMinPiece = 256;        // keys of a piece, about, at least
// Ranges of fewer keys (256 KB of keys and values) are not cut: one workgroup reads them at about 50 GB/s, and a
// join costs 5 to 7 us (16 x 100..500 keys, 32 heads of 128: 29.3 us cut from 512 on in pieces of 256, 20.5 uncut).
constexpr int kv_min_cut(int hd) { return (1 << 16) / hd; }
constexpr int kKvRowWaves = 4;          // waves that share the keys of 16 query rows
constexpr int kv_short_waves(int hd) { return hd == 64 ? 16 : 8; }      // ... of a short range

// How key ranges are cut: into pieces of about sum / split_target keys, the sum taken over all requests of row
// tiles (of TR rows) x keys, so that the pieces fill the chip once; but each piece more writes and reads the
// partial sums of all their rows once more, so no further than that costs what it saves: a range of m keys in n pieces
// takes a m / n + b n, least at n = sqrt(m a / b), with a = 20 ns a key (heads of 256: 60) and b = 8 bytes an
// element at 5 TB/s (300 new tokens on 1000 keys, 96 heads of 128: 85 us cut in four, 41 uncut by this rule).  Tiles of 16
// rows never reach that.
struct KvCut {
    float rate;          // pieces per key; 0: none is cut
    float most2;         // square of pieces, at most, per key
};
template <int HD, int TR, bool SINKS>
__device__ __forceinline__ KvCut kv_cut(const KvAttnArgs &a, int lane) {
    if (!a.split_target) return {0.f, 0.f};
    float sum = 0.f, rows = 0.f;
    for (int r0 = 0; r0 < a.n_req; r0 += 64) {
        float x = 0.f, y = 0.f;
        if (r0 + lane < a.n_req) {
            const KvReq q = kv_req<TR, SINKS>(a, r0 + lane);
            x = (float)((q.rows + TR - 1) / TR) * (float)q.keys();
            y = q.keys() >= kv_min_cut(HD) ? (float)q.rows : 0.f;
        }
        sum += wave_sum(x);
        if (TR != kKvRowTile) rows += wave_sum(y);
    }
    if (!(sum > 0.f)) return {0.f, 0.f};
    return {(float)a.split_target / (sum * (float)a.n_kv),
            (HD == 256 ? 0.06f : 0.02f) * 5e6f / (8.f * (HD + 2) * fmaxf(rows, 1.f) * (float)a.n_kv)};
}

// Keys per piece of a request of `keys` keys.  A range is cut in c only from c - 1/4 times the aim on: a little
// more than the chip holds at once costs a second round.  Hence the pieces of all cut ranges number at most
// (2 / 1.75) * split_target.
template <int HD, int TR>
__device__ __forceinline__ int kv_piece(int keys, KvCut cut) {
    if (keys < kv_min_cut(HD)) return max(keys, 1);
    float aim = (float)keys * cut.rate + 0.25f;
    if (TR != kKvRowTile) aim = fminf(aim, __builtin_amdgcn_sqrtf((float)keys * cut.most2));
    const int n = min((int)fminf(aim, 65536.f), (keys + kKvMinPiece / 2) / kKvMinPiece);
    return n > 1 ? ((keys + n - 1) / n + 63) & ~63 : max(keys, 1);
}

// Item `want` of one kv head: requests in order, row tiles, pieces.  Items of requests whose key range is
// cut are numbered apart (slot), so that the workspace does not grow with the row tiles.
struct KvItem {
    int r, tile, split, splits;     // r < 0: there is no such item
    int slot;                       // of the tile's first piece, if splits > 1
    int piece;                      // keys of a piece
    KvReq q;
};
// ROWS > 0 counts groups of ROWS rows of the cut requests instead (for the join; split is then the group), of those whose
// items all had a workgroup.
template <int HD, int TR, int ROWS, bool SINKS>
__device__ __forceinline__ KvItem kv_item(const KvAttnArgs &a, int want, KvCut aim, int lane) {
    KvItem it;
    it.r = -1;
    int base = 0, base_slot = 0, base_item = 0;
    for (int r0 = 0; r0 < a.n_req; r0 += 64) {
        KvReq q{};
        int tiles = 0, splits = 1, piece = 1;
        if (r0 + lane < a.n_req) {
            q = kv_req<TR, SINKS>(a, r0 + lane);
            tiles = (q.rows + TR - 1) / TR;
            piece = kv_piece<HD, TR>(q.keys(), aim);
            splits = max((q.keys() + piece - 1) / piece, 1);
        }
        const int cut = splits > 1 ? tiles * splits : 0;
        const int mine = ROWS == 0 ? tiles * splits : splits > 1 ? (q.rows + ROWS - 1) / (ROWS == 0 ? 1 : ROWS) : 0;
        const int incl = wave_incl_scan(mine), total = __builtin_amdgcn_readlane(incl, 63);
        const int incl_slot = a.split_target ? wave_incl_scan(cut) : 0;
        const int incl_item = ROWS != 0 ? wave_incl_scan(tiles * splits) : 0;
        if (want < base + total) {
            const uint64_t past = __ballot(incl > want - base);
            const int l = __builtin_ctzll(past);
            const int at = want - base - (bcast(incl, l) - bcast(mine, l));
            it.r = r0 + l;
            it.splits = bcast(splits, l);
            it.piece = bcast(piece, l);
            it.q.q0 = bcast(q.q0, l), it.q.n = bcast(q.n, l), it.q.m = bcast(q.m, l);
            it.q.rows = bcast(q.rows, l), it.q.lo = bcast(q.lo, l), it.q.hi = bcast(q.hi, l);
            it.q.first = SINKS ? bcast(q.first, l) : 0;
            if (ROWS == 0) {
                it.tile = at / it.splits;
                it.split = at - it.tile * it.splits;
                // wide tiles: later rows see more keys and go first
                if (TR != kKvRowTile) it.tile = bcast(tiles, l) - 1 - it.tile;
            } else {
                it.tile = at * ROWS / TR;
                it.split = at;
            }
            it.slot = base_slot + bcast(incl_slot, l) - bcast(cut, l) + it.tile * it.splits;
            // (row ranges that overlap can ask for more than the workspace holds, or the grid; those are left out)
            if (it.splits > 1 && it.slot + it.splits > a.slots) it.r = -2;
            if (ROWS != 0 && base_item + bcast(incl_item, l) > a.items) it.r = -2;
            return it;
        }
        base += total;
        base_slot += __builtin_amdgcn_readlane(incl_slot, 63);
        if (ROWS != 0) base_item = min(base_item + __builtin_amdgcn_readlane(incl_item, 63), 1 << 30);
    }
    return it;
}

// Running state of 16 query rows in one wave: O^T tiles, the reference of the exponents (log2 units)
// and this lane's share of the row's sum.
template <int HD>
struct KvRowState {
    f32x4 o[HD / 16];
    float ref, sum;
};

// The largest of the four lane groups' values, per row.
__device__ __forceinline__ float kv_row_max(float x) {
    x = fmaxf(x, __shfl_xor(x, 16));
    return fmaxf(x, __shfl_xor(x, 32));
}
__device__ __forceinline__ float kv_row_sum(float x) {
    x += __shfl_xor(x, 16);
    return x + __shfl_xor(x, 32);
}

// What the waves of a workgroup hand over to each other at the end of an item of 16 rows.
template <int HD, int WAVES>
struct KvRowsLds {
    f32x4 o[WAVES > 1 ? WAVES / 2 : 1][HD / 16][64];
    float ref[WAVES][16], sum[WAVES > 1 ? WAVES / 2 : 1][64];
};

// One workgroup: one item (16 query rows of one kv head, one key range) of one request; its waves
// take a part of the range each, 32 keys at a time, straight from the pages into registers: nothing of K or V
// is read twice by one tile, so LDS would only add a step.  The next block's keys are loaded during the softmax and its values after
// the second product, 16 KB in flight per wave for heads of 128.  A score more than `lag` powers of two
// above the running reference moves it; smaller ones do not, so most blocks rescale nothing.  Scores, sums, references
// and outputs are fp32; a weight enters the second product as two numbers of the element type (kv_weights), as MFMA
// waits for memory here: 16 x 2k keys 61.1 us with one and 61.0 with both, 4 x 60k grouped 84.6 and 85.0 (1 x 513, all
// latency, 7.4 and 7.5), and the outputs are then as near to 64-bit ones as their type allows (16 x 2k: 3.2e-5 off in the
// mean square's root, now 2.4e-5, which is the rounding of the output alone).  Bound by HBM: 16 requests of 2k keys, 32
// heads of 128, 275 MB in 54.7 us, and 58.7 a pass with the join; 96 heads of 3k, 1.8 GB in 315 us (5.7 TB/s).  TR:
// rows of a split item in the workspace.
template <class T, int HD, int TR, int WAVES, bool SINKS>
__device__ __forceinline__ void kv_rows_item(const KvAttnArgs &a, const KvItem &it, int h, KvRowsLds<HD, WAVES> &sh) {
    constexpr int kSteps = HD / 32, kTiles = HD / 16, kWaves = WAVES;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int col = lane & 15, g = lane >> 4;
    const KvReq &rq = it.q;

    // this lane's query row
    const int row = it.tile * kKvRowTile + col, row_c = min(row, rq.rows - 1);
    const int tok = row_c / a.group, head = h * a.group + (row_c - tok * a.group);
    const int pos = rq.m - rq.n + tok;
    const int see_hi = min(pos + 1, rq.hi), see_lo = a.window ? max(pos - a.window + 1, 0) : 0;
    uint4 qf[kSteps];
    {
        const uint16_t *qp = a.q + (int64_t)(rq.q0 + tok) * a.q_ts + (int64_t)head * a.q_hs + 8 * g;
#pragma unroll
        for (int t = 0; t < kSteps; ++t) qf[t] = ld16(qp + 32 * t);
    }
    // keys that some row of the tile sees (first and last token), within the item's chunk
    const int tok_a = it.tile * kKvRowTile / a.group, tok_b = (min(it.tile * kKvRowTile + kKvRowTile, rq.rows) - 1) / a.group;
    const int pos_a = rq.m - rq.n + tok_a, pos_b = rq.m - rq.n + tok_b;
    const int tile_hi = min(pos_b + 1, rq.hi), tile_lo = a.window ? max(pos_a - a.window + 1, 0) : 0;
    // every row of the tile sees keys in [all_lo, all_hi)
    const int all_hi = min(pos_a + 1, rq.hi), all_lo = a.window ? max(pos_b - a.window + 1, 0) : 0;
    const KvSpan sp = kv_span<TR, SINKS, 32>(a, rq, tile_lo, tile_hi, it.splits, it.split, it.piece);
    // this wave's part
    const int before = SINKS && sp.a1 >= 0 ? sp.a1 - sp.a0 : 0, all = before + sp.hi - sp.lo;
    const int part = max((((all + kWaves - 1) / kWaves) + 31) & ~31, 32);
    int k_lo = sp.lo + wave * part, k_hi = min(k_lo + part, sp.hi);
    if constexpr (SINKS) {               // (whole blocks are before)
        const int from = wave * part, to = min(from + part, all);
        k_lo = from < before ? sp.a0 + from : sp.lo + from - before;
        k_hi = to <= before ? sp.a0 + to : sp.lo + to - before;
        if (from >= to) k_hi = k_lo;
    }
    const int sinks = SINKS ? a.sinks : 0;

    KvRowState<HD> st;
#pragma unroll
    for (int t = 0; t < kTiles; ++t) st.o[t] = f32x4{0.f, 0.f, 0.f, 0.f};
    st.ref = -INFINITY;
    st.sum = 0.f;

    const int *const tab = a.table + (int64_t)it.r * a.table_stride;
    const int page = 1 << a.page_log, held = (rq.hi + page - 1) >> a.page_log;
    const int64_t page_elems = ((int64_t)a.n_kv << a.page_log) * HD;
    const uint16_t *const k_head = a.k + ((int64_t)h * HD << a.page_log), *const v_head = a.v + ((int64_t)h * HD << a.page_log);
    int tab0 = 0, ids = 0;
    bool none = true;                    // no table entries at hand yet
    // Where the 32 keys of a block lie: elements of the pages of keys kb..+15 and kb+16..+31 (the same one unless
    // pages hold 16 positions), and whether there are such pages.
    struct Block {
        int64_t b0, b1;
        int in0, in1;
        bool dead0, dead1;
    };
    auto find = [&](int kb) -> Block {
        Block x;
        const int p0 = kb >> a.page_log, p1 = (kb + 16) >> a.page_log;
        if (none || p1 - tab0 >= 64) {                  // the next 64 table entries, one per lane
            tab0 = p0;
            ids = tab0 + lane < held ? tab[tab0 + lane] : -1;
            none = false;
        }
        const int id0 = bcast(ids, p0 - tab0), id1 = bcast(ids, p1 - tab0);
        x.dead0 = (uint32_t)id0 >= (uint32_t)a.n_pages, x.dead1 = (uint32_t)id1 >= (uint32_t)a.n_pages;
        // without a page something in bounds is read; its keys are masked
        x.b0 = (x.dead0 ? 0 : id0) * page_elems, x.b1 = (x.dead1 ? 0 : id1) * page_elems;
        x.in0 = kb & (page - 1), x.in1 = (kb + 16) & (page - 1);
        return x;
    };
    uint4 kf[2][kSteps], vf[kTiles];
    // keys: tile u, row 4a + b is key 8a + 4u + b
    const int krow = 8 * ((col >> 2) & 1) + (col & 3);
    auto load_k = [&](const Block &x) {
        const uint16_t *kp = k_head + (col & 8 ? x.b1 + (int64_t)x.in1 * HD : x.b0 + (int64_t)x.in0 * HD) + krow * HD + 8 * g;
#pragma unroll
        for (int t = 0; t < kSteps; ++t)
#pragma unroll
            for (int u = 0; u < 2; ++u) kf[u][t] = ld16(kp + 4 * u * HD + 32 * t);
    };
    auto load_v = [&](const Block &x) {
        const uint16_t *vp = v_head + (g & 2 ? x.b1 + x.in1 : x.b0 + x.in0) + 8 * (g & 1) + (col << a.page_log);
#pragma unroll
        for (int t = 0; t < kTiles; ++t) vf[t] = ld16(vp + ((16 * t) << a.page_log));
    };
    Block at{}, next{};
    if (k_lo < k_hi) {
        next = find(k_lo);
        load_k(next);
        load_v(next);
    }
    for (int kb = k_lo, kn; kb < k_hi; kb = kn) {
        at = next;
        const bool dead0 = at.dead0, dead1 = at.dead1, more = kb + 32 < k_hi;
        kn = SINKS && more ? sp.after(kb, 32) : kb + 32;
        if (more) next = find(kn);
        float s[8];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            f32x4 acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int t = 0; t < kSteps; ++t) acc = T::mfma16(kf[u][t], qf[t], acc);
#pragma unroll
            for (int i = 0; i < 4; ++i) s[4 * u + i] = acc[i] * a.scale_log2;
        }

        if (more) load_k(next);          // in flight during the softmax and the second product

        uint32_t odd_keys = 0;                           // keys of the block with an infinite or NaN value somewhere
        if ((kb < all_lo && (!SINKS || kb + 32 > sinks)) || kb + 32 > all_hi || dead0 || dead1) {
            const bool dead = g & 2 ? dead1 : dead0;
            // As bits of the lane's eight keys.  (Not a branch around each score: with the condition of SINKS hipcc 7.2 made one per
            // score for heads of 64, and the block that masks the eighth came out empty -- s_and_saveexec, s_or of exec -- so that
            // this score stayed.  No kernel built here has such an empty block.)
            const int j0 = kb + 8 * g;
            auto below = [&](int end) { return (1u << min(max(end - j0, 0), 8)) - 1u; };
            const uint32_t first = SINKS ? below(sinks) : 0u, live = dead ? 0u : 0xffu;
            const uint32_t seen = live & below(see_hi) & (~below(see_lo) | first);
            const uint32_t kept = live & below(tile_hi) & (~below(tile_lo) | first);     // values that some row of the tile sees
#pragma unroll
            for (int e = 0; e < 8; ++e) s[e] = seen >> e & 1 ? s[e] : -INFINITY;
            // Values that no row of the tile sees are cleared (0 x infinity would be NaN); those
            // that some rows see and others do not, and that are not finite, are added row by row.
            uint32_t odd = 0;
#pragma unroll
            for (int e2 = 0; e2 < 4; ++e2) {
                const uint32_t keep = (kept >> (2 * e2) & 1 ? 0xffffu : 0u) | (kept >> (2 * e2) & 2 ? 0xffff0000u : 0u);
#pragma unroll
                for (int t = 0; t < kTiles; ++t) {
                    uint32_t &w = e2 == 0 ? vf[t].x : e2 == 1 ? vf[t].y : e2 == 2 ? vf[t].z : vf[t].w;
                    w &= keep;
                    if ((w & T::kExpMask & 0xffffu) == (T::kExpMask & 0xffffu)) odd |= 1u << (2 * e2);
                    if ((w & T::kExpMask & 0xffff0000u) == (T::kExpMask & 0xffff0000u)) odd |= 2u << (2 * e2);
                }
            }
            if (pos_a != pos_b && __any(odd != 0)) {
#pragma unroll
                for (int x = 1; x < 16; x <<= 1) odd |= __shfl_xor(odd, x);
                odd_keys = (uint32_t)bcast((int)odd, 0) | (uint32_t)bcast((int)odd, 16) << 8 |
                           (uint32_t)bcast((int)odd, 32) << 16 | (uint32_t)bcast((int)odd, 48) << 24;
#pragma unroll
                for (int e2 = 0; e2 < 4; ++e2) {
                    const uint32_t keep = (odd >> (2 * e2) & 1 ? 0u : 0xffffu) | (odd >> (2 * e2) & 2 ? 0u : 0xffff0000u);
#pragma unroll
                    for (int t = 0; t < kTiles; ++t) (e2 == 0 ? vf[t].x : e2 == 1 ? vf[t].y : e2 == 2 ? vf[t].z : vf[t].w) &= keep;
                }
            }
        }

        float top = s[0];
#pragma unroll
        for (int e = 1; e < 8; ++e) top = fmaxf(top, s[e]);
        // The reference moves only when some score of the wave passes it by more than the lag.
        if (__any(top - T::kShift > st.ref + T::kLag)) {
            const float ref = fmaxf(kv_row_max(top) - T::kShift, st.ref);
            const float f = st.ref == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(st.ref - ref);
            st.sum *= f;
#pragma unroll
            for (int t = 0; t < kTiles; ++t) st.o[t] *= f;
            st.ref = ref;
        }
        const float ref = st.ref == -INFINITY ? 0.f : st.ref;
        float p[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            p[e] = __builtin_amdgcn_exp2f(s[e] - ref);
            st.sum += p[e];
        }
        uint4 head, rest;
        kv_weights<T>(p, head, rest);
#pragma unroll
        for (int t = 0; t < kTiles; ++t) st.o[t] = T::mfma16(vf[t], head, st.o[t]);
#pragma unroll
        for (int t = 0; t < kTiles; ++t) st.o[t] = T::mfma16(vf[t], rest, st.o[t]);

        if (more) load_v(next);

        while (odd_keys) {
            const int j = __builtin_ctz(odd_keys);
            odd_keys &= odd_keys - 1;
            float mine = p[0];
#pragma unroll
            for (int e = 1; e < 8; ++e) mine = (j & 7) == e ? p[e] : mine;
            const float w = __shfl(mine, (j >> 3) * 16 + col);
            if ((kb + j < see_lo && (!SINKS || kb + j >= sinks)) || kb + j >= see_hi) continue;
            int d0 = 4 * g;
            asm volatile("" : "+v"(d0));                // its addresses are not worth registers outside this loop
            const uint16_t *x = v_head + (j & 16 ? at.b1 + at.in1 + (j & 15) : at.b0 + at.in0 + j);
#pragma unroll
            for (int t = 0; t < kTiles; ++t)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    st.o[t][i] += w * (float)__builtin_bit_cast(typename T::e, x[(d0 + 16 * t + i) << a.page_log]);
        }
    }

    // the waves' parts: a common reference per row, then sums in a fixed order
    float ref = st.ref;
    if constexpr (kWaves > 1) {
        if (lane < 16) sh.ref[wave][lane] = st.ref;
        __syncthreads();
        ref = sh.ref[0][col];
#pragma unroll
        for (int w = 1; w < kWaves; ++w) ref = fmaxf(ref, sh.ref[w][col]);
        const float f = st.ref == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(st.ref - ref);
        st.sum *= f;
#pragma unroll
        for (int t = 0; t < kTiles; ++t) st.o[t] *= f;
#pragma unroll
        for (int half = kWaves / 2; half >= 1; half >>= 1) {
            if (wave >= half && wave < 2 * half) {
#pragma unroll
                for (int t = 0; t < kTiles; ++t) sh.o[wave - half][t][lane] = st.o[t];
                sh.sum[wave - half][lane] = st.sum;
            }
            __syncthreads();
            if (wave < half) {
#pragma unroll
                for (int t = 0; t < kTiles; ++t) st.o[t] += sh.o[wave][t][lane];
                st.sum += sh.sum[wave][lane];
            }
            __syncthreads();
        }
    }
    if (wave != 0) return;
    const float sum = kv_row_sum(st.sum);
    if (it.splits == 1) {
        if (row >= rq.rows) return;
        const float inv = sum == 0.f ? 0.f : 1.f / sum;
        uint16_t *op = a.out + (int64_t)(rq.q0 + tok) * a.o_ts + (int64_t)head * a.o_hs + 4 * g;
#pragma unroll
        for (int t = 0; t < kTiles; ++t)
            *reinterpret_cast<uint2 *>(op + 16 * t) = make_uint2(kv_pack<T>(st.o[t][0] * inv, st.o[t][1] * inv),
                                                                 kv_pack<T>(st.o[t][2] * inv, st.o[t][3] * inv));
        return;
    }
    float *const pt = a.part + ((int64_t)(it.slot + it.split) * a.n_kv + h) * (TR * (HD + 2));
    if (row < rq.rows) {
#pragma unroll
        for (int t = 0; t < kTiles; ++t) *reinterpret_cast<f32x4 *>(pt + col * HD + 16 * t + 4 * g) = st.o[t];
        if (g == 0) {
            pt[TR * HD + col] = ref;
            pt[TR * (HD + 1) + col] = sum;
        }
    }
}

// Calls in which no request has many query rows per kv head.  WAVES: 4; more for few short ranges, 1 for
// many short ones, neither of which are cut, so that no join follows.
template <class T, int HD, int WAVES, bool SINKS>
__global__ __launch_bounds__(64 * WAVES) void k_kv_rows(KvAttnArgs a) {
    __shared__ KvRowsLds<HD, WAVES> sh;
    const int lane = threadIdx.x & 63;
    const int h = blockIdx.x % a.n_kv, want = blockIdx.x / a.n_kv;
    const KvItem it = kv_item<HD, kKvRowTile, 0, SINKS>(a, want, kv_cut<HD, kKvRowTile, SINKS>(a, lane), lane);
    if (it.r < 0) return;
    kv_rows_item<T, HD, kKvRowTile, WAVES, SINKS>(a, it, h, sh);
}

// One workgroup: one item of 128 query rows of one kv head, 32 of them per wave, over one key
// range, KT keys at a time.  K and V of a block go from the pages to LDS without passing registers
// (16 bytes per lane), the next block's while this one is computed; the waves read them from there
// as MFMA operands.  Inside a row of either tile the 16-byte units are permuted by the row's number, on
// the way in, so that the 16 lanes that read the same unit of 16 rows find them in 16 bank groups.
// The products are those of k_kv_rows on 32x32x16 MFMA: tile row 16s + 8u + 4h + v is key 16s + 8h + 4u
// + v, so that lane half h holds keys 16s + 8h .. +7 of its query row in accumulators 8s .. 8s+7.  The weights are rounded
// to the element type for the second product, and their sums are of the unrounded ones: in two numbers each, as
// k_kv_rows has them, a 4096-token chunk on 12204 cached keys takes 1330 us and not 963, drafts of 5 tokens 30.6 and not 28.7.
// The outputs of that chunk are 6.1e-5 off 64-bit ones in the mean square's root, 4.3e-5 of it by their own rounding.
// Bound by MFMA and softmax together at the clock that the card holds: a 4096-token chunk on 12204 cached
// keys, 32 heads of 128, 936 us in a run of passes = 1022 TFLOP/s (a library product of 8192^3 reaches 1270), 1014 in the
// median of 24 passes under a trace; MFMA is busy half of the time, the vector units most of the other half, LDS a
// quarter.  More buffers in flight, other orders of the first product, wave priorities, and sums of the weights by dot
// products measured no faster.
// P: positions that a page gives to a block, the page's or all of the block's.  K lies in LDS as [key][HD], V as in the
// pages, [page][HD][P], so that every load reads 1 KB of one page from a scalar address (with V gathered as [HD][key],
// pages of 16 took 16% longer than pages of 64: 2048 tokens on 8000 keys, 32 heads of 128; now 277 and 270 us).
template <int HD, int P>
struct KvTile {
    static constexpr int kKeys = HD == 256 ? 32 : 64;      // 64 KB of LDS for both buffers at most
    static constexpr int kUnitsK = HD / 8, kUnitsV = P / 8;      // 16-byte units of a row
    static constexpr int kLoads = kKeys * HD * 2 / 1024 / 4;     // 1 KB loads per wave and operand
    static constexpr int kBytes = kKeys * HD * 2;                // of one operand's tile
    static __device__ __forceinline__ int swz_k(int key) { return kUnitsK >= 16 ? key & 15 : (key >> 1) & 7; }
    static __device__ __forceinline__ int swz_v(int d) { return kUnitsV == 8 ? (d >> 1) & 7 : kUnitsV == 4 ? (d >> 2) & 3 : (d >> 3) & 1; }
    // Where values 8u .. 8u+7 of row d of V^T lie.
    static __device__ __forceinline__ int at_v(int d, int u) {
        return (u / kUnitsV) * (HD * P) + d * P + ((u % kUnitsV) ^ swz_v(d)) * 8;
    }
};

// Eight values with those cleared whose bits are set in m.
__device__ __forceinline__ uint4 kv_clear(uint4 x, uint32_t m) {
    auto keep = [&](int b) { return (m >> b & 1 ? 0u : 0xffffu) | (m >> b & 2 ? 0u : 0xffff0000u); };
    x.x &= keep(0), x.y &= keep(2), x.z &= keep(4), x.w &= keep(6);
    return x;
}

// 64 lanes x 16 bytes from base + off (per lane) to 1 KB of LDS at byte address `lds`.  The compiler
// does not see the load in flight: kv_lds_wait before the barrier after which the bytes are read.  (m0 is an
// operand, so that the compiler writes it: as a reserved register it may not be clobbered by the statement.)
__device__ __forceinline__ void kv_lds_load(const uint16_t *base, uint32_t off, uint32_t lds) {
    asm volatile("s_nop 0\n\tglobal_load_lds_dwordx4 %0, %1" ::"v"(off), "s"(base), "{m0}"(lds) : "memory");
}
__device__ __forceinline__ void kv_lds_wait() { asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); }

// Bits 0 .. n-1 (n <= 64), and the bits of the 16-key groups named by a mask of at most 4 bits.
__device__ __forceinline__ uint64_t kv_bits(uint32_t n) { return n >= 64 ? ~0ull : (1ull << n) - 1; }
__device__ __forceinline__ uint64_t kv_dead_bits(uint32_t m) {
    // each bit to the foot of its group, then over the group
    const uint64_t f = (uint64_t)(m & 1) | (uint64_t)(m & 2) << 15 | (uint64_t)(m & 4) << 30 | (uint64_t)(m & 8) << 45;
    return f * 0xffffull;
}

// P: as in KvTile.  MIXED: requests of few rows, single tokens beside
// prompt chunks among them, are taken too, by kv_rows_item: they wait for memory, not for MFMA.  (14 single tokens
// beside two chunks of 777, 56 heads of 128: 165 us without this path, 156 with it, 147 a pass now, the join
// included.  Without such requests it stays out of the kernel, whose registers then serve the one loop: a 4096-token
// chunk 1009 -> 953.)
template <class T, int HD, int P, bool MIXED, bool SINKS>
__global__ __launch_bounds__(256, HD == 256 ? 1 : HD == 128 ? 2 : 3) void k_kv_tile(KvAttnArgs a) {
    typedef KvTile<HD, P> L;
    constexpr int KT = L::kKeys, kSub = KT / 32, kSteps = HD / 16, kTiles = HD / 32;
    // [buffer][K, V]
    __shared__ __align__(16) union {
        uint16_t kv[2][2][L::kBytes / 2];
        KvRowsLds<HD, kKvRowWaves> rows;     // of kv_rows_item
    } s_mem;
    uint16_t (&s_kv)[2][2][L::kBytes / 2] = s_mem.kv;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int col = lane & 31, half = lane >> 5;
    const int h = blockIdx.x % a.n_kv, want = blockIdx.x / a.n_kv;
    const KvItem it = kv_item<HD, kKvWideTile, 0, SINKS>(a, want, kv_cut<HD, kKvWideTile, SINKS>(a, lane), lane);
    if (it.r < 0) return;
    const KvReq &rq = it.q;
    if constexpr (MIXED) {
        if (rq.rows <= kKvRowTile) {
            kv_rows_item<T, HD, kKvWideTile, kKvRowWaves, SINKS>(a, it, h, s_mem.rows);
            return;
        }
    }
    const int tile = it.tile, past = rq.m - rq.n;

    // this lane's query row
    const int row = tile * kKvWideTile + wave * 32 + col, row_c = min(row, rq.rows - 1);
    const int tok = row_c / a.group, head = h * a.group + (row_c - tok * a.group);
    const int pos = past + tok;
    const int see_hi = min(pos + 1, rq.hi), see_lo = a.window ? max(pos - a.window + 1, 0) : 0;
    uint4 qf[kSteps];
    {
        const uint16_t *qp = a.q + (int64_t)(rq.q0 + tok) * a.q_ts + (int64_t)head * a.q_hs + 8 * half;
#pragma unroll
        for (int t = 0; t < kSteps; ++t) qf[t] = ld16(qp + 16 * t);
    }
    // keys that some row of the workgroup sees, within the item's chunk
    const int pos_first = past + tile * kKvWideTile / a.group;
    const int pos_last = past + (min((tile + 1) * kKvWideTile, rq.rows) - 1) / a.group;
    const KvSpan sp = kv_span<kKvWideTile, SINKS, KT>(a, rq, a.window ? max(pos_first - a.window + 1, 0) : 0,
                                                      min(pos_last + 1, rq.hi), it.splits, it.split, it.piece);
    const int lo = SINKS && sp.a1 >= 0 ? sp.a0 : sp.lo, hi = sp.hi, sinks = SINKS ? a.sinks : 0;
    // keys that some row of this wave sees, and those that all of them see
    const int wrow = tile * kKvWideTile + wave * 32;
    const int pos_a = past + min(wrow, rq.rows - 1) / a.group, pos_b = past + (min(wrow + 32, rq.rows) - 1) / a.group;
    const bool idle = wrow >= rq.rows;
    const int wave_hi = idle ? 0 : min(pos_b + 1, rq.hi), wave_lo = a.window ? max(pos_a - a.window + 1, 0) : 0;
    const int all_hi = min(pos_a + 1, rq.hi), all_lo = a.window ? max(pos_b - a.window + 1, 0) : 0;

    // where this lane's 16 bytes of each load come from, inside a page
    const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint16_t *)&s_kv[0][0][0];
    uint32_t off_k[L::kLoads], off_v[L::kLoads];
#pragma unroll
    for (int i = 0; i < L::kLoads; ++i) {
        const int u = (wave * L::kLoads + i) * 64 + lane;
        const int key = u / L::kUnitsK, d = u / L::kUnitsV % HD;
        const int first = (wave * L::kLoads + i) * 64 / L::kUnitsK;
        off_k[i] = (uint32_t)(((key - first) * HD + 8 * ((u % L::kUnitsK) ^ L::swz_k(key))) * 2);
        off_v[i] = (uint32_t)((d << a.page_log) + 8 * ((u % L::kUnitsV) ^ L::swz_v(d))) * 2;
    }

    const int *const tab = a.table + (int64_t)it.r * a.table_stride;
    const int page = 1 << a.page_log, held = (rq.hi + page - 1) >> a.page_log;
    const int64_t page_elems = ((int64_t)a.n_kv << a.page_log) * HD, head_elems = (int64_t)h * HD << a.page_log;
    int tab0 = 0, ids = 0;
    bool none = true;                    // no table entries at hand yet
    // The loads of block kb into buffer buf; returns which of its 16-key groups have no page.
    auto load = [&](int kb, int buf) -> uint32_t {
        const int p0 = kb >> a.page_log, p1 = (kb + KT - 1) >> a.page_log;
        // (a second pass goes back in the table; tested here, as a reset before it cost the loop 5%, heads of 256 40%)
        if (none || p1 - tab0 >= 64 || p0 < tab0) {
            tab0 = p0;
            ids = tab0 + lane < held ? tab[tab0 + lane] : -1;
            none = false;
        }
        uint32_t dead = 0;
        const bool bad = (uint32_t)ids >= (uint32_t)a.n_pages;
        const int id_safe = bad ? 0 : ids;               // something in bounds; its keys are masked
        const uint64_t bads = __ballot(bad);
        const uint32_t dst = lds0 + buf * 2 * L::kBytes + wave * L::kLoads * 1024;
        if constexpr (P == KT) {                         // one page
            const int64_t id = bcast(id_safe, p0 - tab0);
            if (bads >> (p0 - tab0) & 1) dead = 15u;
            const uint16_t *const kp = a.k + id * page_elems + head_elems + (int64_t)(kb & (page - 1)) * HD;
            const uint16_t *const vp = a.v + id * page_elems + head_elems + (kb & (page - 1));
#pragma unroll
            for (int i = 0; i < L::kLoads; ++i)
                kv_lds_load(kp + (wave * L::kLoads + i) * 512, off_k[i], dst + i * 1024);
#pragma unroll
            for (int i = 0; i < L::kLoads; ++i) kv_lds_load(vp, off_v[i], dst + L::kBytes + i * 1024);
        } else {
#pragma unroll
            for (int j = 0; j < KT / P; ++j)
                if (bads >> (p0 - tab0 + j) & 1) dead |= ((1u << (P / 16)) - 1) << (j * (P / 16));
#pragma unroll
            for (int i = 0; i < L::kLoads; ++i) {
                const int k0 = (wave * L::kLoads + i) * 64 / L::kUnitsK;
                const int64_t id = bcast(id_safe, p0 - tab0 + k0 / P);
                kv_lds_load(a.k + id * page_elems + head_elems + (k0 % P) * HD, off_k[i], dst + i * 1024);
            }
#pragma unroll
            for (int i = 0; i < L::kLoads; ++i) {
                const int64_t id = bcast(id_safe, p0 - tab0 + (wave * L::kLoads + i) * 64 / (HD * L::kUnitsV));
                kv_lds_load(a.v + id * page_elems + head_elems, off_v[i], dst + L::kBytes + i * 1024);
            }
        }
        return dead;
    };

    f32x16 o[kTiles];
    float ref, sum;
    const int krow = (col & ~12) | (col & 8) >> 1 | (col & 4) << 1;
    // An infinity or NaN among the values of keys that some rows of a tile see and others do not reaches
    // the others too (0 x infinity).  Such values are looked for only if a result is not finite: the
    // workgroup then computes its item once more and handles them apart (careful).
    for (bool careful = false;; careful = true) {
#pragma unroll
    for (int t = 0; t < kTiles; ++t)
#pragma unroll
        for (int i = 0; i < 16; ++i) o[t][i] = 0.f;
    ref = -INFINITY, sum = 0.f;
    uint32_t dead_next = 0;
    int buf = 0;
    if (lo < hi) dead_next = load(lo, 0);
    for (int kb = lo, kn; kb < hi; kb = kn, buf ^= 1) {
        kn = SINKS ? sp.after(kb, KT) : kb + KT;
        const uint32_t dead = dead_next;
        kv_lds_wait();
        __syncthreads();                 // block kb is in LDS, and every wave is done with the buffer before it
        if (kn < hi) dead_next = load(kn, buf ^ 1);
        uint16_t *const sk = s_kv[buf][0], *const sv = s_kv[buf][1];
        // Values past the request's keys and of missing pages may hold anything and are cleared (0 x infinity would be
        // NaN), in LDS, by all waves.
        if (kb + KT > rq.hi || dead != 0) {
            const uint64_t none = ~kv_bits((uint32_t)min(rq.hi - kb, KT)) | kv_dead_bits(dead);
            for (int i = threadIdx.x; i < HD * (KT / 8); i += 256) {
                const int d = i / (KT / 8), unit = i % (KT / 8);
                uint4 &x = *reinterpret_cast<uint4 *>(sv + L::at_v(d, unit));
                x = kv_clear(x, (uint32_t)(none >> (8 * unit)));
            }
            __syncthreads();
        }
        if (kb >= wave_hi || (kb + KT <= wave_lo && (!SINKS || kb >= sinks))) continue;

        f32x16 s[kSub];
#pragma unroll
        for (int u = 0; u < kSub; ++u) {
#pragma unroll
            for (int i = 0; i < 16; ++i) s[u][i] = 0.f;
            const int key = 32 * u + krow;
#pragma unroll
            for (int t = 0; t < kSteps; ++t) {
                const int unit = (2 * t + half) ^ L::swz_k(key);
                s[u] = T::mfma32(*reinterpret_cast<const uint4 *>(sk + key * HD + unit * 8), qf[t], s[u]);
            }
        }
        const bool edge = (kb < all_lo && (!SINKS || kb + KT > sinks)) || kb + KT > all_hi || dead != 0;
        const uint64_t kept = SINKS ? kv_bits((uint32_t)min(max(sinks - kb, 0), KT)) : 0;    // first keys of the block
        if (edge) {
            // the keys that this lane's row sees, a bit each; its half holds every other 8 of them
            const uint32_t n_all = KT == 64 ? 64 : 32;
            const uint32_t from = (uint32_t)min(max(see_lo - kb, 0), (int)n_all), to = (uint32_t)min(max(see_hi - kb, 0), (int)n_all);
            uint64_t see = kv_bits(to) & (~kv_bits(from) | kept) & ~kv_dead_bits(dead);
            see >>= 8 * half;
#pragma unroll
            for (int u = 0; u < kSub; ++u)
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const int e = 32 * u + 16 * (i >> 3) + (i & 7);
                    if (!((e < 32 ? (uint32_t)see : (uint32_t)(see >> 32)) >> (e & 31) & 1)) s[u][i] = -INFINITY;
                }
        }
        float top = s[0][0];
#pragma unroll
        for (int u = 0; u < kSub; ++u)
#pragma unroll
            for (int i = 0; i < 16; ++i) top = fmaxf(top, s[u][i]);
        top = top * a.scale_log2 - T::kShift;
        // The reference moves only when some score of the wave passes it by more than the lag.
        if (__any(top > ref + T::kLag)) {
            const float to = fmaxf(fmaxf(top, __shfl_xor(top, 32)), ref);
            const float f = ref == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(ref - to);
            sum *= f;
#pragma unroll
            for (int t = 0; t < kTiles; ++t) o[t] *= f;
            ref = to;
        }
        const float r = ref == -INFINITY ? 0.f : ref;
        float part = 0.f;
#pragma unroll
        for (int u = 0; u < kSub; ++u)
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                s[u][i] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[u][i], a.scale_log2, -r));
                part += s[u][i];
            }
        sum += part;
        // With `careful`, values of keys that no row of the wave sees are taken as zero, and so are those that some
        // rows see and others do not, and that are not finite: those are added row by row.
        uint64_t drop = 0;
        auto v_frag = [&](int t, int j) -> uint4 {
            return *reinterpret_cast<const uint4 *>(sv + L::at_v(32 * t + col, 2 * j + half));
        };
        auto clear = [&](uint4 x, int j) -> uint4 { return kv_clear(x, (uint32_t)(drop >> (16 * j + 8 * half))); };
        if (careful && edge) {
            drop = ~kv_bits((uint32_t)min(wave_hi - kb, KT)) | (kv_bits((uint32_t)min(max(wave_lo - kb, 0), KT)) & ~kept);
            uint64_t odd_keys = 0;
#pragma unroll 1
            for (int j = 0; j < 2 * kSub; ++j) {
                uint32_t odd = 0;
#pragma unroll 1
                for (int t = 0; t < kTiles; ++t) {
                    const uint4 x = clear(v_frag(t, j), j);
                    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                    for (int b = 0; b < 4; ++b) {
                        if ((w[b] & T::kExpMask & 0xffffu) == (T::kExpMask & 0xffffu)) odd |= 1u << (2 * b);
                        if ((w[b] & T::kExpMask & 0xffff0000u) == (T::kExpMask & 0xffff0000u)) odd |= 2u << (2 * b);
                    }
                }
                if (__any(odd != 0)) {
                    for (int x = 1; x < 32; x <<= 1) odd |= __shfl_xor(odd, x);
                    odd_keys |= ((uint64_t)(uint32_t)bcast((int)odd, 0) | (uint64_t)(uint32_t)bcast((int)odd, 32) << 8) << (16 * j);
                }
            }
            drop |= odd_keys;
            while (odd_keys) {
                const int j = __builtin_ctzll(odd_keys);
                odd_keys &= odd_keys - 1;
                float mine = 0.f;
#pragma unroll
                for (int u = 0; u < kSub; ++u)
#pragma unroll
                    for (int i = 0; i < 16; ++i) mine = (32 * u + 16 * (i >> 3) + (i & 7)) == (j & ~8) ? s[u][i] : mine;
                const float w = __shfl(mine, (j & 8 ? 32 : 0) + col);
                if ((kb + j < see_lo && (!SINKS || kb + j >= sinks)) || kb + j >= see_hi) continue;
                int d0 = 4 * half;
                asm volatile("" : "+v"(d0));        // its addresses are not worth registers outside this loop
#pragma unroll
                for (int t = 0; t < kTiles; ++t)
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const int d = 32 * t + 8 * (i >> 2) + d0 + (i & 3);
                        o[t][i] += w * (float)__builtin_bit_cast(typename T::e, sv[L::at_v(d, j >> 3) + (j & 7)]);
                    }
            }
        }
        auto weights = [&](int j) -> uint4 {
            const f32x16 &x = s[j >> 1];
            const int b = 8 * (j & 1);
            return make_uint4(kv_pack<T>(x[b], x[b + 1]), kv_pack<T>(x[b + 2], x[b + 3]), kv_pack<T>(x[b + 4], x[b + 5]),
                              kv_pack<T>(x[b + 6], x[b + 7]));
        };
        // (one branch around all of the product, so that its loads run ahead of its MFMAs)
        if (careful && edge) {
#pragma unroll
            for (int j = 0; j < 2 * kSub; ++j) {
                const uint4 pf = weights(j);
#pragma unroll
                for (int t = 0; t < kTiles; ++t) {
                    o[t] = T::mfma32(clear(v_frag(t, j), j), pf, o[t]);
                    __builtin_amdgcn_sched_barrier(0);       // (registers)
                }
            }
        } else {
#pragma unroll
            for (int j = 0; j < 2 * kSub; ++j) {
                const uint4 pf = weights(j);
#pragma unroll
                for (int t = 0; t < kTiles; ++t) o[t] = T::mfma32(v_frag(t, j), pf, o[t]);
            }
        }
    }
    if (careful) break;
    float probe = 0.f;                   // 0 if every sum is finite, NaN otherwise
#pragma unroll
    for (int t = 0; t < kTiles; ++t)
#pragma unroll
        for (int i = 0; i < 16; ++i) probe += 0.f * o[t][i];
    // (the buffers are free: a word of them carries the waves' vote, so that LDS stays at 64 KB)
    volatile int *const again = reinterpret_cast<volatile int *>(&s_kv[0][0][0]);
    __syncthreads();
    if (threadIdx.x == 0) *again = 0;
    __syncthreads();
    if (probe != 0.f) *again = 1;
    __syncthreads();
    const int vote = *again;
    __syncthreads();
    if (!vote) break;
    }

    if (row >= rq.rows) return;
    sum += __shfl_xor(sum, 32);
    if (it.splits == 1) {
        const float inv = sum == 0.f ? 0.f : 1.f / sum;
        uint16_t *op = a.out + (int64_t)(rq.q0 + tok) * a.o_ts + (int64_t)head * a.o_hs + 4 * half;
#pragma unroll
        for (int t = 0; t < kTiles; ++t)
#pragma unroll
            for (int i = 0; i < 16; i += 4)
                *reinterpret_cast<uint2 *>(op + 32 * t + 2 * i) = make_uint2(kv_pack<T>(o[t][i] * inv, o[t][i + 1] * inv),
                                                                             kv_pack<T>(o[t][i + 2] * inv, o[t][i + 3] * inv));
        return;
    }
    const int prow = wave * 32 + col;
    float *const pt = a.part + ((int64_t)(it.slot + it.split) * a.n_kv + h) * (kKvWideTile * (HD + 2));
#pragma unroll
    for (int t = 0; t < kTiles; ++t)
#pragma unroll
        for (int i = 0; i < 16; i += 4)
            *reinterpret_cast<f32x4 *>(pt + prow * HD + 32 * t + 2 * i + 4 * half) = f32x4{o[t][i], o[t][i + 1], o[t][i + 2], o[t][i + 3]};
    if (half == 0) {
        pt[kKvWideTile * HD + prow] = ref;
        pt[kKvWideTile * (HD + 1) + prow] = sum;
    }
}

// Joins the split items, each scaled to the largest reference, and divides by the row's sum: a workgroup takes a
// few rows of one kv head at a time (a row per HD / 4 lanes, 16 bytes each), its four waves a quarter of the pieces
// each, kDeep of them in flight; the quarters are added in order.  The grid does not depend on how many requests are
// cut: with none it ends at once.  Bound by latency, 5 to 8 us, of which 4 to 5 to find that there is nothing to do.
template <class T, int HD, int TR, bool SINKS>
__global__ __launch_bounds__(256) void k_kv_join(KvAttnArgs a) {
    constexpr int kLanes = HD / 4, kRows = 64 / kLanes, kDeep = 8, kWaves = 4;
    __shared__ f32x4 s_o[kWaves][64];
    __shared__ float s_ref[kWaves][64], s_sum[kWaves][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const KvCut cut = kv_cut<HD, TR, SINKS>(a, lane);
    const int64_t stride = (int64_t)a.n_kv * (TR * (HD + 2));
    const int d = (lane % kLanes) * 4;
    for (int u = blockIdx.x;; u += gridDim.x) {
        const int h = u % a.n_kv, want = u / a.n_kv;
        const KvItem it = kv_item<HD, TR, kRows, SINKS>(a, want, cut, lane);
        if (it.r == -1) return;
        if (it.r < 0) continue;
        const int row = it.split * kRows + lane / kLanes, row_c = min(row, it.q.rows - 1), prow = row_c - it.tile * TR;
        const float *const pt = a.part + ((int64_t)it.slot * a.n_kv + h) * (TR * (HD + 2));
        const int quarter = (it.splits + kWaves - 1) / kWaves, from = wave * quarter, to = min(from + quarter, it.splits);
        float ref = -INFINITY, sum = 0.f;
        f32x4 o = {0.f, 0.f, 0.f, 0.f};
        for (int s0 = from; s0 < to; s0 += kDeep) {
            float r[kDeep], w[kDeep];
            f32x4 x[kDeep];
#pragma unroll
            for (int i = 0; i < kDeep; ++i) {
                const float *const ps = pt + min(s0 + i, to - 1) * stride;
                r[i] = ps[TR * HD + prow];
                w[i] = ps[TR * (HD + 1) + prow];
                x[i] = *reinterpret_cast<const f32x4 *>(ps + prow * HD + d);
            }
            float top = ref;
#pragma unroll
            for (int i = 0; i < kDeep; ++i) top = fmaxf(top, r[i]);
            const float f0 = ref == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(ref - top);
            sum *= f0;
            o *= f0;
            ref = top;
#pragma unroll
            for (int i = 0; i < kDeep; ++i) {
                if (s0 + i >= to) break;
                const float f = r[i] == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(r[i] - ref);
                sum += f * w[i];
                o += f * x[i];
            }
        }
        s_o[wave][lane] = o;
        s_ref[wave][lane] = ref;
        s_sum[wave][lane] = sum;
        __syncthreads();
        if (wave == 0) {
            float top = s_ref[0][lane];
#pragma unroll
            for (int w = 1; w < kWaves; ++w) top = fmaxf(top, s_ref[w][lane]);
            sum = 0.f;
            o = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int w = 0; w < kWaves; ++w) {
                const float r = s_ref[w][lane], f = r == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(r - top);
                sum += f * s_sum[w][lane];
                o += f * s_o[w][lane];
            }
            if (row < it.q.rows) {
                const float inv = sum == 0.f ? 0.f : 1.f / sum;
                const int tok = row / a.group, head = h * a.group + (row - tok * a.group);
                *reinterpret_cast<uint2 *>(a.out + (int64_t)(it.q.q0 + tok) * a.o_ts + (int64_t)head * a.o_hs + d) =
                    make_uint2(kv_pack<T>(o[0] * inv, o[1] * inv), kv_pack<T>(o[2] * inv, o[3] * inv));
            }
        }
        __syncthreads();
    }
}

}  // namespace pik
