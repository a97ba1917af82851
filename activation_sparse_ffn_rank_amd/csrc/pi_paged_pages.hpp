// pi_paged_pages.hpp -- gfx950 kernels that give pages back (k_kv_release), share them (k_kv_fork) and copy them (k_kv_copy).
#pragma once

#include "pi_paged.hpp"

namespace pik {

struct KvPagesArgs {
    int n_req, page_log, n_pages, max_pages;
    int64_t table_stride;
    const int *cached;
    int *ring;
    const int *pool;
    int *table, *shares, *cached_next, *pool_next, *counts;
};
struct KvReleaseArgs {
    KvPagesArgs p;
    const int *from, *to;
    int *copies;
};
struct KvForkArgs {
    KvPagesArgs p;
    const int *src, *dst;
    int n_fork;
    int *copies;
};

__device__ __forceinline__ int kv_load(const int *p) { return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT); }

// The request (or fork) of entry e: the last r with first[r] <= e.
__device__ __forceinline__ int kv_owner_of(const uint32_t *first, int n, uint32_t e) {
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (first[mid] <= e) lo = mid;
        else hi = mid;
    }
    return lo;
}

constexpr int kKvMiddle = INT32_MIN;       // flag: the entries become -1

// One workgroup: ranges of entries per request by scans, then the entries, four per thread and round, three times over:
//  1. one owner less for each (whole numbers: any order gives the same),
//  2. of the pages that have run out of owners the first entry that names it, by a minimum over INT32_MIN + entry,
//  3. those entries' pages behind the free ones, by a scan.
// Nothing is kept in scratch memory: a page's count of further owners below zero says that it is free, and serves as the place of
// the minimum.  At most 4096 * 2^17 = 2^29 entries.
static __global__ __launch_bounds__(kKvTableThreads) void k_kv_release(KvReleaseArgs x) {
    const KvPagesArgs &a = x.p;
    __shared__ uint32_t s_first[PI_KV_MAX_REQ + 1];
    __shared__ int s_col[PI_KV_MAX_REQ];              // first column, | kKvMiddle
    __shared__ uint32_t s_part[kKvTableThreads / 64];
    __shared__ uint32_t s_given;
    const int tid = threadIdx.x, n = a.n_req, per = (n + kKvTableThreads - 1) / kKvTableThreads, page = 1 << a.page_log;
    const int64_t room = (int64_t)a.max_pages << a.page_log;
    int head = a.pool[0] % a.n_pages;
    if (head < 0) head += a.n_pages;
    const int count = min(max(a.pool[1], 0), a.n_pages);
    if (tid == 0) s_given = 0;

    int c[kKvReqPerThread], f[kKvReqPerThread], old[kKvReqPerThread];
    bool bad[kKvReqPerThread], tail[kKvReqPerThread], split[kKvReqPerThread];
    int end[kKvReqPerThread];
    uint32_t asks = 0;
#pragma unroll
    for (int k = 0; k < kKvReqPerThread; ++k) {
        const int r = tid * per + k;
        const bool in = k < per && r < n;
        c[k] = in ? a.cached[r] : 0;
        f[k] = in ? max(x.from[r], 0) : 0;
        const int t = in && x.to ? x.to[r] : INT32_MAX;
        bad[k] = c[k] < 0 || c[k] > room;
        tail[k] = in && !bad[k] && t >= c[k] && f[k] < c[k];
        end[k] = !in || bad[k] || f[k] >= c[k] ? 0 : tail[k] ? (c[k] + page - 1) >> a.page_log : max(t, 0) >> a.page_log;
        old[k] = -1;
        split[k] = false;
        if (tail[k] && (f[k] & (page - 1))) {
            old[k] = a.table[(int64_t)r * a.table_stride + (f[k] >> a.page_log)];
            split[k] = (uint32_t)old[k] < (uint32_t)a.n_pages && a.shares[old[k]] > 0;
        }
        asks += split[k];
    }
    uint32_t total_asks, total;
    uint32_t rank = kv_block_scan(asks, s_part, &total_asks);
    uint32_t entries = 0, denied = 0, mine[kKvReqPerThread];
    int fresh[kKvReqPerThread];
#pragma unroll
    for (int k = 0; k < kKvReqPerThread; ++k) {
        const int r = tid * per + k;
        mine[k] = 0;
        fresh[k] = -1;
        if (k >= per || r >= n) continue;
        bool refused = bad[k];
        if (split[k]) {
            refused = rank >= (uint32_t)count;
            if (!refused) fresh[k] = a.ring[((int64_t)head + rank) % a.n_pages];
            ++rank;
        }
        denied += refused;
        const int first = split[k] ? f[k] >> a.page_log : (int)(((int64_t)f[k] + page - 1) >> a.page_log);
        if (!refused) mine[k] = (uint32_t)max(end[k] - first, 0);
        split[k] = split[k] && !refused;
        tail[k] = tail[k] && !refused;
        s_col[r] = first | (tail[k] ? 0 : kKvMiddle);
        entries += mine[k];
        x.copies[2 * r] = split[k] ? old[k] : -1;
        x.copies[2 * r + 1] = split[k] ? fresh[k] : -1;
        a.cached_next[r] = tail[k] ? f[k] : c[k];
    }
    uint32_t at = kv_block_scan(entries, s_part, &total);
#pragma unroll
    for (int k = 0; k < kKvReqPerThread; ++k) {
        const int r = tid * per + k;
        if (k < per && r < n) s_first[r] = at;
        at += mine[k];
    }
    uint32_t total_denied;
    kv_block_scan(denied, s_part, &total_denied);       // (its barriers order s_first and the reads of the ring, too)

    // entry e .. e+3 of this thread: f(place in the table, page, whether it becomes -1), pages out of range left out
    constexpr int kEach = 4;
    auto walk = [&](uint32_t e0, auto &&each) {
        if (e0 >= total) return;
        int r = kv_owner_of(s_first, n, e0);
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
            const uint32_t e = e0 + i;
            if (e >= total) return;
            while (r + 1 < n && s_first[r + 1] <= e) ++r;
            int *const at = a.table + (int64_t)r * a.table_stride + (s_col[r] & INT32_MAX) + (e - s_first[r]);
            const int p = *at;
            if ((uint32_t)p < (uint32_t)a.n_pages) each(i, e, at, p, s_col[r] < 0);
        }
    };
    uint32_t given = 0;
    for (uint32_t e = tid * kEach; e < total; e += kKvTableThreads * kEach)
        walk(e, [&](int, uint32_t, int *, int p, bool) {
            atomicSub(a.shares + p, 1);
            ++given;
        });
    if (given) atomicAdd(&s_given, given);
    __threadfence();
    __syncthreads();
    for (uint32_t e = tid * kEach; e < total; e += kKvTableThreads * kEach)
        walk(e, [&](int, uint32_t e, int *, int p, bool) {
            if (kv_load(a.shares + p) < 0) atomicMin(a.shares + p, INT32_MIN + (int)e);
        });
    __threadfence();
    __syncthreads();
    uint32_t back = 0;
    for (uint32_t base = 0; base < total; base += kKvTableThreads * kEach) {
        int won[kEach];
        uint32_t wins = 0;
#pragma unroll
        for (int i = 0; i < kEach; ++i) won[i] = -1;
        walk(base + tid * kEach, [&](int i, uint32_t e, int *at, int p, bool middle) {
            if (kv_load(a.shares + p) == INT32_MIN + (int)e) won[i] = p, ++wins;
            if (middle) *at = -1;
        });
        uint32_t all;
        uint32_t to = kv_block_scan(wins, s_part, &all) + back;
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
            if (won[i] < 0) continue;
            a.ring[((int64_t)head + count + to++) % a.n_pages] = won[i];
            __hip_atomic_store(a.shares + won[i], 0, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        }
        back += all;
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kKvReqPerThread; ++k)
        if (split[k]) a.table[(int64_t)(tid * per + k) * a.table_stride + (f[k] >> a.page_log)] = fresh[k];
    if (tid == 0) {
        const uint32_t taken = min(total_asks, (uint32_t)count);
        a.pool_next[0] = (int)(((int64_t)head + taken) % a.n_pages);
        a.pool_next[1] = (int)min((int64_t)count - taken + back, (int64_t)a.n_pages);
        a.counts[0] = (int)s_given;
        a.counts[1] = (int)back;
        a.counts[2] = (int)taken;
        a.counts[3] = (int)total_denied;
    }
}

// One workgroup: which forks are made, by scans; then the shared entries, four per thread and round.
static __global__ __launch_bounds__(kKvTableThreads) void k_kv_fork(KvForkArgs x) {
    const KvPagesArgs &a = x.p;
    __shared__ uint32_t s_first[PI_KV_MAX_REQ + 1];
    __shared__ uint32_t s_pair[PI_KV_MAX_REQ];        // source | destination << 16
    __shared__ int s_claim[PI_KV_MAX_REQ];            // first fork to name a destination
    __shared__ uint32_t s_part[kKvTableThreads / 64];
    __shared__ uint32_t s_shared;
    const int tid = threadIdx.x, n = x.n_fork, per = (n + kKvTableThreads - 1) / kKvTableThreads, page = 1 << a.page_log;
    const int64_t room = (int64_t)a.max_pages << a.page_log;
    int head = a.pool[0] % a.n_pages;
    if (head < 0) head += a.n_pages;
    const int count = min(max(a.pool[1], 0), a.n_pages);
    if (tid == 0) s_shared = 0;
    int keep[kKvReqPerThread];                        // cached of all requests
#pragma unroll
    for (int r = tid, k = 0; k < kKvReqPerThread; r += kKvTableThreads, ++k) {
        keep[k] = r < a.n_req ? a.cached[r] : 0;
        if (r < a.n_req) s_claim[r] = INT32_MAX;
    }
    __syncthreads();
    int s[kKvReqPerThread], d[kKvReqPerThread];
#pragma unroll
    for (int k = 0; k < kKvReqPerThread; ++k) {
        const int i = tid * per + k;
        const bool in = k < per && i < n;
        s[k] = in ? x.src[i] : -1;
        d[k] = in ? x.dst[i] : -1;
        if ((uint32_t)d[k] < (uint32_t)a.n_req) atomicMin(&s_claim[d[k]], i);
    }
    __syncthreads();
    int len[kKvReqPerThread], old[kKvReqPerThread], fresh[kKvReqPerThread];
    bool ok[kKvReqPerThread], part[kKvReqPerThread];
    uint32_t asks = 0;
#pragma unroll
    for (int k = 0; k < kKvReqPerThread; ++k) {
        const int i = tid * per + k;
        ok[k] = (uint32_t)s[k] < (uint32_t)a.n_req && (uint32_t)d[k] < (uint32_t)a.n_req && s[k] != d[k];
        len[k] = ok[k] ? a.cached[s[k]] : 0;
        ok[k] = ok[k] && len[k] >= 0 && len[k] <= room && a.cached[d[k]] == 0 && s_claim[d[k]] == i;
        part[k] = ok[k] && (len[k] & (page - 1));
        old[k] = part[k] ? a.table[(int64_t)s[k] * a.table_stride + (len[k] >> a.page_log)] : -1;
        if ((uint32_t)old[k] >= (uint32_t)a.n_pages) old[k] = -1;
        asks += old[k] >= 0;
    }
    uint32_t total_asks, total, total_denied, total_done;
    uint32_t rank = kv_block_scan(asks, s_part, &total_asks);
    uint32_t entries = 0, denied = 0, done = 0, mine[kKvReqPerThread];
#pragma unroll
    for (int k = 0; k < kKvReqPerThread; ++k) {
        const int i = tid * per + k;
        mine[k] = 0;
        fresh[k] = -1;
        if (k >= per || i >= n) continue;
        if (old[k] >= 0) {
            if (rank >= (uint32_t)count) ok[k] = false, old[k] = -1;
            else fresh[k] = a.ring[((int64_t)head + rank) % a.n_pages];
            ++rank;
        }
        if (ok[k]) mine[k] = (uint32_t)(len[k] >> a.page_log), ++done;
        else ++denied;
        entries += mine[k];
        s_pair[i] = ok[k] ? (uint32_t)s[k] | (uint32_t)d[k] << 16 : 0u;
        x.copies[2 * i] = old[k];
        x.copies[2 * i + 1] = fresh[k];
    }
    uint32_t at = kv_block_scan(entries, s_part, &total);
#pragma unroll
    for (int k = 0; k < kKvReqPerThread; ++k) {
        const int i = tid * per + k;
        if (k < per && i < n) s_first[i] = at;
        at += mine[k];
    }
    kv_block_scan(denied, s_part, &total_denied);
    kv_block_scan(done, s_part, &total_done);         // (their barriers order the arrays above and the reads of cached, too)
    if (a.cached_next != a.cached)
#pragma unroll
        for (int r = tid, k = 0; k < kKvReqPerThread; r += kKvTableThreads, ++k)
            if (r < a.n_req) a.cached_next[r] = keep[k];
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kKvReqPerThread; ++k) {
        if (!ok[k] || k >= per || tid * per + k >= n) continue;
        a.cached_next[d[k]] = len[k];
        if (part[k]) a.table[(int64_t)d[k] * a.table_stride + (len[k] >> a.page_log)] = fresh[k];
    }
    constexpr int kEach = 4;
    uint32_t shared = 0;
    for (uint32_t e0 = tid * kEach; e0 < total; e0 += kKvTableThreads * kEach) {
        int i = kv_owner_of(s_first, n, e0);
#pragma unroll
        for (int j = 0; j < kEach; ++j) {
            const uint32_t e = e0 + j;
            if (e >= total) break;
            while (i + 1 < n && s_first[i + 1] <= e) ++i;
            const uint32_t pair = s_pair[i], col = e - s_first[i];
            const int p = a.table[(int64_t)(pair & 0xffff) * a.table_stride + col];
            a.table[(int64_t)(pair >> 16) * a.table_stride + col] = p;
            if ((uint32_t)p < (uint32_t)a.n_pages) {
                atomicAdd(a.shares + p, 1);
                ++shared;
            }
        }
    }
    if (shared) atomicAdd(&s_shared, shared);
    __syncthreads();
    if (tid == 0) {
        const uint32_t taken = min(total_asks, (uint32_t)count);
        a.pool_next[0] = (int)(((int64_t)head + taken) % a.n_pages);
        a.pool_next[1] = (int)((int64_t)count - taken);
        a.counts[0] = (int)total_done;
        a.counts[1] = (int)s_shared;
        a.counts[2] = (int)taken;
        a.counts[3] = (int)total_denied;
    }
}

struct KvCopyArgs {
    const int *copies;
    int n_pages;
    int64_t units;            // of 16 bytes, of one page's keys (as many of values)
    uint4 *k, *v;
};

// Workgroup (pair and operand, part): 16 KB at a time, every gridDim.y-th.
static __global__ __launch_bounds__(256) void k_kv_copy(KvCopyArgs a) {
    const int i = blockIdx.x >> 1;
    const int from = a.copies[2 * i], to = a.copies[2 * i + 1];
    if ((uint32_t)from >= (uint32_t)a.n_pages || (uint32_t)to >= (uint32_t)a.n_pages || from == to) return;
    uint4 *const base = blockIdx.x & 1 ? a.v : a.k;
    const uint4 *const src = base + from * a.units;
    uint4 *const dst = base + to * a.units;
    constexpr int kDeep = 4;
    for (int64_t u0 = (int64_t)blockIdx.y * (256 * kDeep) + threadIdx.x; u0 < a.units; u0 += (int64_t)gridDim.y * (256 * kDeep)) {
        uint4 x[kDeep];
#pragma unroll
        for (int j = 0; j < kDeep; ++j)
            if (u0 + j * 256 < a.units) x[j] = src[u0 + j * 256];
#pragma unroll
        for (int j = 0; j < kDeep; ++j)
            if (u0 + j * 256 < a.units) dst[u0 + j * 256] = x[j];
    }
}

}  // namespace pik
