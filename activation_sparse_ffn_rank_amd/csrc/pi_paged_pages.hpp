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
    int *ws;               // KvReleaseWs, or null: one workgroup does it all
};
struct KvForkArgs {
    KvPagesArgs p;
    const int *src, *dst;
    int n_fork;
    int *copies;
};

// Shares are changed and read by atomics of one workgroup, which its XCD's L2 serves, or of many (MANY), which are coherent over
// the whole device.
template <bool MANY>
struct KvShares {
    static constexpr int kScope = MANY ? __HIP_MEMORY_SCOPE_AGENT : __HIP_MEMORY_SCOPE_WORKGROUP;
    static __device__ __forceinline__ int load(const int *p) { return __hip_atomic_load(p, __ATOMIC_RELAXED, kScope); }
    static __device__ __forceinline__ void store(int *p, int v) { __hip_atomic_store(p, v, __ATOMIC_RELAXED, kScope); }
    static __device__ __forceinline__ int less(int *p) { return __hip_atomic_fetch_add(p, -1, __ATOMIC_RELAXED, kScope); }
    static __device__ __forceinline__ void lower(int *p, int v) { __hip_atomic_fetch_min(p, v, __ATOMIC_RELAXED, kScope); }
};

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

constexpr int kKvMiddle = INT32_MIN;       // flag of a first column: the entries become -1
constexpr int kKvEach = 4;                 // entries per thread and round
constexpr int kKvReleaseGroups = 256;      // workgroups of a long list

// What the first launch leaves for the ones behind it: ints at these places.
struct KvReleaseWs {
    static constexpr int kTotal = 0, kHead = 1, kCount = 2, kTaken = 3, kDenied = 4, kGiven = 5, kWins = 8;
    static constexpr int kFirst = kWins + kKvReleaseGroups;                // [n_req + 1] first entry of each request
    static constexpr int kCol = kFirst + PI_KV_MAX_REQ + 1;                // [n_req] its first column, | kKvMiddle
    static constexpr int kFresh = kCol + PI_KV_MAX_REQ;                    // [n_req] page for its first column, -1: none
    static constexpr int kInts = kFresh + PI_KV_MAX_REQ;
};

// Entries of a thread: their places in the table, pages (-1: none, or out of range), and whether they become -1.
template <int N>
struct KvEntries {
    int *at[N], p[N];
    bool middle[N];
};
// Those numbered e0 .. e0 + kKvEach - 1.
__device__ __forceinline__ KvEntries<kKvEach> kv_entries(const KvPagesArgs &a, const uint32_t *first, const int *col,
                                                         uint32_t total, uint32_t e0) {
    KvEntries<kKvEach> x;
#pragma unroll
    for (int i = 0; i < kKvEach; ++i) x.p[i] = -1, x.middle[i] = false, x.at[i] = a.table;
    if (e0 >= total) return x;
    int r = kv_owner_of(first, a.n_req, e0);
#pragma unroll
    for (int i = 0; i < kKvEach; ++i) {
        const uint32_t e = e0 + i;
        if (e < total) {
            while (r + 1 < a.n_req && first[r + 1] <= e) ++r;
            x.at[i] = a.table + (int64_t)r * a.table_stride + (col[r] & INT32_MAX) + (e - first[r]);
            x.middle[i] = col[r] < 0;
            x.p[i] = *x.at[i];
        }
    }
#pragma unroll
    for (int i = 0; i < kKvEach; ++i)
        if ((uint32_t)x.p[i] >= (uint32_t)a.n_pages) x.p[i] = -1;
    return x;
}
// each(i, e, place in the table, page, whether it becomes -1) for those with a page.
template <class F>
__device__ __forceinline__ void kv_walk(const KvPagesArgs &a, const uint32_t *first, const int *col, uint32_t total, uint32_t e0,
                                        F &&each) {
    const KvEntries<kKvEach> x = kv_entries(a, first, col, total, e0);
#pragma unroll
    for (int i = 0; i < kKvEach; ++i)
        if (x.p[i] >= 0) each(i, e0 + i, x.at[i], x.p[i], x.middle[i]);
}

// The three passes over the entries, for a range [from, to) of them in rounds of a workgroup:
//  1. one owner less for each (whole numbers: any order gives the same); returns this thread's number of valid ones, and, in one
//     workgroup, clears `plain` if a page had further owners or was named before: if its count was not 0 (over many workgroups
//     the counts' way back and a word for all cost 3 us, as much as the pass that they save),
template <bool MANY>
__device__ __forceinline__ uint32_t kv_give(const KvPagesArgs &a, const uint32_t *first, const int *col, uint32_t from, uint32_t to,
                                            bool &plain) {
    uint32_t given = 0;
    for (uint32_t e = from + threadIdx.x * kKvEach; e < to; e += blockDim.x * kKvEach) {
        int before[kKvEach] = {};
        kv_walk(a, first, col, to, e, [&](int i, uint32_t, int *, int p, bool) {
            before[i] = KvShares<MANY>::less(a.shares + p);
            ++given;
        });
        if constexpr (!MANY) {
#pragma unroll
            for (int i = 0; i < kKvEach; ++i) plain = plain && before[i] == 0;
        }
    }
    return given;
}
//  2. of the pages that have run out of owners the first entry that names it, as the minimum over INT32_MIN + entry,
template <bool MANY>
__device__ __forceinline__ void kv_lead(const KvPagesArgs &a, const uint32_t *first, const int *col, uint32_t from, uint32_t to) {
    for (uint32_t e = from + threadIdx.x * kKvEach; e < to; e += blockDim.x * kKvEach)
        kv_walk(a, first, col, to, e, [&](int, uint32_t e, int *, int p, bool) {
            if (KvShares<MANY>::load(a.shares + p) < 0) KvShares<MANY>::lower(a.shares + p, INT32_MIN + (int)e);
        });
}
//  3. the pages of those entries behind the free ones, from place `at` of the ring on; returns how many.  plain: every page was
//     named once and had no further owners, so all of them.
template <bool MANY>
__device__ __forceinline__ uint32_t kv_push(const KvPagesArgs &a, const uint32_t *first, const int *col, uint32_t from, uint32_t to,
                                            int64_t at, uint32_t *part, bool plain) {
    uint32_t back = 0;
    for (uint32_t base = from; base < to; base += blockDim.x * kKvEach) {
        int won[kKvEach];
        uint32_t wins = 0;
#pragma unroll
        for (int i = 0; i < kKvEach; ++i) won[i] = -1;
        kv_walk(a, first, col, to, base + threadIdx.x * kKvEach, [&](int i, uint32_t e, int *place, int p, bool middle) {
            if (plain || KvShares<MANY>::load(a.shares + p) == INT32_MIN + (int)e) won[i] = p, ++wins;
            if (middle) *place = -1;
        });
        uint32_t all;
        uint32_t rank = kv_block_scan(wins, part, &all) + back;
#pragma unroll
        for (int i = 0; i < kKvEach; ++i) {
            if (won[i] < 0) continue;
            a.ring[(at + rank++) % a.n_pages] = won[i];
            KvShares<MANY>::store(a.shares + won[i], 0);
        }
        back += all;
    }
    return back;
}

// The same passes by one workgroup over a list of one round, N entries per thread in order, read before.  Where no page that is
// given up has further owners and none is named twice -- every count was 0 -- all of them go back, and the second pass and its
// reads are left out; likewise where those with further owners keep some.
template <int N>
__device__ __forceinline__ uint32_t kv_one_round(const KvPagesArgs &a, const KvEntries<N> &x, int64_t at, uint32_t *part,
                                                 uint32_t &given) {
    const uint32_t e0 = threadIdx.x * N;
    int before[N];
    uint32_t mine = 0, wins = 0;
    bool plain = true, odd = false;
#pragma unroll
    for (int i = 0; i < N; ++i) before[i] = x.p[i] >= 0 ? KvShares<false>::less(a.shares + x.p[i]) : 0;
#pragma unroll
    for (int i = 0; i < N; ++i) mine += x.p[i] >= 0, plain = plain && before[i] == 0;
    bool won[N];
#pragma unroll
    for (int i = 0; i < N; ++i) won[i] = x.p[i] >= 0 && before[i] == 0;
    if (!__syncthreads_and(plain)) {
        int left[N];
#pragma unroll
        for (int i = 0; i < N; ++i) left[i] = x.p[i] >= 0 ? KvShares<false>::load(a.shares + x.p[i]) : 0;
#pragma unroll
        for (int i = 0; i < N; ++i) odd = odd || (left[i] < 0 && (left[i] != -1 || before[i] != 0));
        if (__syncthreads_or(odd)) {
#pragma unroll
            for (int i = 0; i < N; ++i)
                if (left[i] < 0) KvShares<false>::lower(a.shares + x.p[i], INT32_MIN + (int)(e0 + i));
            kv_lds_wait();
            __syncthreads();
#pragma unroll
            for (int i = 0; i < N; ++i)
                won[i] = left[i] < 0 && KvShares<false>::load(a.shares + x.p[i]) == INT32_MIN + (int)(e0 + i);
        }
    }
#pragma unroll
    for (int i = 0; i < N; ++i) wins += won[i];
    uint32_t all;                              // both numbers in one scan: at most 4096 each
    uint32_t rank = kv_block_scan(wins | mine << 16, part, &all) & 0xffff;
    given = all >> 16, all &= 0xffff;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        if (x.middle[i] && x.p[i] >= 0) *x.at[i] = -1;
        if (!won[i]) continue;
        a.ring[(at + rank++) % a.n_pages] = x.p[i];
        KvShares<false>::store(a.shares + x.p[i], 0);
    }
    return all;
}

// The first launch, one workgroup: ranges of entries per request by scans; then, if the list is short, all of it.  Bound by the
// latency of its chain lengths -> table -> shares -> scans -> entries -> counts -> scan -> ring: 64 requests after a drafted
// step, two pages each at most, 5.0 us (with a list 7.9); a list of 1024 entries 9.4, of 16384 without further owners 55 (with a
// search for first mentions 123).  Nothing but these ranges is kept in scratch memory: a page's count of further owners below
// zero says that it is free, and serves as the place of the minimum.  At most 4096 * 2^17 = 2^29 entries.
static __global__ __launch_bounds__(kKvTableThreads) void k_kv_release(KvReleaseArgs x) {
    const KvPagesArgs &a = x.p;
    __shared__ uint32_t s_first[PI_KV_MAX_REQ + 1];
    __shared__ int s_col[PI_KV_MAX_REQ];              // first column, | kKvMiddle
    __shared__ uint32_t s_part[kKvTableThreads / 64];
    __shared__ uint32_t s_denied;
    const int tid = threadIdx.x, n = a.n_req, per = (n + (int)blockDim.x - 1) / (int)blockDim.x, page = 1 << a.page_log;
    const int64_t room = (int64_t)a.max_pages << a.page_log;
    const int pool0 = a.pool[0], pool1 = a.pool[1];
    if (tid == 0) s_denied = 0;

    int c[kKvReqPerThread], f[kKvReqPerThread], t[kKvReqPerThread], old[kKvReqPerThread], end[kKvReqPerThread];
    bool bad[kKvReqPerThread], tail[kKvReqPerThread], split[kKvReqPerThread];
#pragma unroll
    for (int k = 0; k < kKvReqPerThread; ++k) {
        const int r = tid * per + k;
        const bool in = k < per && r < n;
        c[k] = in ? a.cached[r] : 0;
        f[k] = in ? x.from[r] : 0;
        t[k] = in && x.to ? x.to[r] : INT32_MAX;
    }
#pragma unroll
    for (int k = 0; k < kKvReqPerThread; ++k) {
        const int r = tid * per + k;
        f[k] = max(f[k], 0);
        bad[k] = c[k] < 0 || c[k] > room;
        tail[k] = k < per && r < n && !bad[k] && t[k] >= c[k] && f[k] < c[k];
        old[k] = tail[k] && (f[k] & (page - 1)) ? a.table[(int64_t)r * a.table_stride + (f[k] >> a.page_log)] : -1;
        end[k] = k >= per || r >= n || bad[k] || f[k] >= c[k] ? 0 : tail[k] ? (c[k] + page - 1) >> a.page_log : max(t[k], 0) >> a.page_log;
    }
    // With a request per thread the first pages that it gives up are read at once: there may be no others.
    int early[3] = {-1, -1, -1};
    if (per == 1) {
#pragma unroll
        for (int i = 0; i < 3; ++i) {
            const int col = (f[0] >> a.page_log) + i;
            if (col < end[0]) early[i] = a.table[(int64_t)tid * a.table_stride + col];
        }
    }
    int head = pool0 % a.n_pages;
    if (head < 0) head += a.n_pages;
    const int count = min(max(pool1, 0), a.n_pages);
    uint32_t asks = 0, total_asks, total;
#pragma unroll
    for (int k = 0; k < kKvReqPerThread; ++k) {
        split[k] = (uint32_t)old[k] < (uint32_t)a.n_pages && a.shares[old[k]] > 0;
        asks += split[k];
    }
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
    }
    if (denied) atomicAdd(&s_denied, denied);
    const uint32_t taken = min(total_asks, (uint32_t)count);
    if (per == 1 && __syncthreads_and(mine[0] <= 2)) {
        // two pages of a request at most
        const int skip = split[0] || !(f[0] & (page - 1)) ? 0 : 1;
        KvEntries<2> e;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            e.at[i] = a.table + (int64_t)tid * a.table_stride + (f[0] >> a.page_log) + skip + i;
            e.p[i] = (uint32_t)i < mine[0] ? skip ? early[i + 1] : early[i] : -1;
            if ((uint32_t)e.p[i] >= (uint32_t)a.n_pages) e.p[i] = -1;
            e.middle[i] = !tail[0];
        }
        uint32_t given;
        const uint32_t back = kv_one_round(a, e, (int64_t)head + count, s_part, given);
        if (tid < n) {
            x.copies[2 * tid] = split[0] ? old[0] : -1;
            x.copies[2 * tid + 1] = split[0] ? fresh[0] : -1;
            a.cached_next[tid] = tail[0] ? f[0] : c[0];
            if (split[0]) a.table[(int64_t)tid * a.table_stride + (f[0] >> a.page_log)] = fresh[0];
        }
        if (tid == 0) {
            a.pool_next[0] = (int)(((int64_t)head + taken) % a.n_pages);
            a.pool_next[1] = (int)min((int64_t)count - taken + back, (int64_t)a.n_pages);
            a.counts[0] = (int)given;
            a.counts[1] = (int)back;
            a.counts[2] = (int)taken;
            a.counts[3] = (int)s_denied;
            if (x.ws) x.ws[KvReleaseWs::kTotal] = 0;
        }
        return;
    }
    uint32_t at = kv_block_scan(entries, s_part, &total);       // (its barriers order s_col and the reads of the ring, too)
    // More than one round goes on to the launches behind, where there are any: 4100 entries 27 us, in two rounds here 29.
    const bool go_on = x.ws && total > blockDim.x * kKvEach;
#pragma unroll
    for (int k = 0; k < kKvReqPerThread; ++k) {
        const int r = tid * per + k;
        if (k >= per || r >= n) continue;
        x.copies[2 * r] = split[k] ? old[k] : -1;
        x.copies[2 * r + 1] = split[k] ? fresh[k] : -1;
        a.cached_next[r] = tail[k] ? f[k] : c[k];
        s_first[r] = at;
        if (go_on) {
            x.ws[KvReleaseWs::kFirst + r] = (int)at;
            x.ws[KvReleaseWs::kCol + r] = s_col[r];
            x.ws[KvReleaseWs::kFresh + r] = split[k] ? fresh[k] : INT32_MIN;
        }
        at += mine[k];
    }
    __syncthreads();
    if (x.ws && tid == 0) {
        x.ws[KvReleaseWs::kTotal] = go_on ? (int)total : 0;
        x.ws[KvReleaseWs::kHead] = head;
        x.ws[KvReleaseWs::kCount] = count;
        x.ws[KvReleaseWs::kTaken] = (int)taken;
        x.ws[KvReleaseWs::kDenied] = (int)s_denied;
        x.ws[KvReleaseWs::kGiven] = 0;
    }
    if (go_on) return;
    uint32_t back = 0, given = 0;
    if (total && total <= blockDim.x * kKvEach) {
        back = kv_one_round(a, kv_entries(a, s_first, s_col, total, tid * kKvEach), (int64_t)head + count, s_part, given);
        __syncthreads();
    } else if (total) {
        bool plain = true;
        const uint32_t mine = kv_give<false>(a, s_first, s_col, 0, total, plain);
        kv_block_scan(mine, s_part, &given);
        kv_lds_wait();
        plain = __syncthreads_and(plain);
        if (!plain) {
            kv_lead<false>(a, s_first, s_col, 0, total);
            kv_lds_wait();
            __syncthreads();
        }
        back = kv_push<false>(a, s_first, s_col, 0, total, (int64_t)head + count, s_part, plain);
        __syncthreads();
    }
#pragma unroll
    for (int k = 0; k < kKvReqPerThread; ++k)
        if (split[k]) a.table[(int64_t)(tid * per + k) * a.table_stride + (f[k] >> a.page_log)] = fresh[k];
    if (tid == 0) {
        a.pool_next[0] = (int)(((int64_t)head + taken) % a.n_pages);
        a.pool_next[1] = (int)min((int64_t)count - taken + back, (int64_t)a.n_pages);
        a.counts[0] = (int)given;
        a.counts[1] = (int)back;
        a.counts[2] = (int)taken;
        a.counts[3] = (int)s_denied;
    }
}

// The launches behind it, for a long list: each workgroup takes its share of the entries, in order.  PASS 0: owners less; 1:
// first entries; 2: how many of them; 3: their pages into the ring.  Each 5 to 9 us, most of that to start, fetch the ranges and
// find the entries: 1000 requests that give up 71 thousand entries, 36 us a pass (295 by the first workgroup alone).
template <int PASS>
__global__ __launch_bounds__(256) void k_kv_release_pass(KvReleaseArgs x) {
    const KvPagesArgs &a = x.p;
    __shared__ uint32_t s_first[PI_KV_MAX_REQ];
    __shared__ int s_col[PI_KV_MAX_REQ];
    __shared__ uint32_t s_part[4];
    const int tid = threadIdx.x, b = blockIdx.x;
    const uint32_t total = (uint32_t)x.ws[KvReleaseWs::kTotal];
    if (total == 0) return;
    for (int r = tid; r < a.n_req; r += 256) {
        s_first[r] = (uint32_t)x.ws[KvReleaseWs::kFirst + r];
        s_col[r] = x.ws[KvReleaseWs::kCol + r];
    }
    const uint32_t share = ((total + kKvReleaseGroups - 1) / kKvReleaseGroups + kKvEach - 1) & ~(uint32_t)(kKvEach - 1);
    const uint32_t from = min(b * share, total), to = min(from + share, total);
    __syncthreads();
    if constexpr (PASS == 0) {
        bool plain = false;
        const uint32_t given = kv_give<true>(a, s_first, s_col, from, to, plain);
        uint32_t all;
        kv_block_scan(given, s_part, &all);
        if (tid == 0 && all) atomicAdd(x.ws + KvReleaseWs::kGiven, (int)all);
    } else if constexpr (PASS == 1) {
        kv_lead<true>(a, s_first, s_col, from, to);
    } else if constexpr (PASS == 2) {
        uint32_t wins = 0, all;
        for (uint32_t e = from + tid * kKvEach; e < to; e += 256 * kKvEach)
            kv_walk(a, s_first, s_col, to, e,
                    [&](int, uint32_t e, int *, int p, bool) { wins += a.shares[p] == INT32_MIN + (int)e; });
        kv_block_scan(wins, s_part, &all);
        if (tid == 0) x.ws[KvReleaseWs::kWins + b] = (int)all;
    } else {
        uint32_t back, before = (uint32_t)x.ws[KvReleaseWs::kWins + tid];      // 256 threads, as many workgroups
        before = kv_block_scan(before, s_part, &back);
        __syncthreads();
        if (tid == b) s_part[0] = before;
        __syncthreads();
        before = s_part[0];
        __syncthreads();
        const int head = x.ws[KvReleaseWs::kHead], count = x.ws[KvReleaseWs::kCount];
        kv_push<true>(a, s_first, s_col, from, to, (int64_t)head + count + before, s_part, false);
        __syncthreads();
        // pages in the place of those that were cut inside of: by the workgroup whose entries begin with them
        for (int r = tid; r < a.n_req; r += 256) {
            const int fresh = x.ws[KvReleaseWs::kFresh + r];
            if (fresh != INT32_MIN && s_first[r] >= from && s_first[r] < to)
                a.table[(int64_t)r * a.table_stride + (s_col[r] & INT32_MAX)] = fresh;
        }
        if (b == 0 && tid == 0) {
            const int taken = x.ws[KvReleaseWs::kTaken];
            a.pool_next[0] = (int)(((int64_t)head + taken) % a.n_pages);
            a.pool_next[1] = (int)min((int64_t)count - taken + back, (int64_t)a.n_pages);
            a.counts[0] = x.ws[KvReleaseWs::kGiven];
            a.counts[1] = (int)back;
            a.counts[2] = taken;
            a.counts[3] = x.ws[KvReleaseWs::kDenied];
        }
    }
}

// Every workgroup finds out by scans which forks are made; they share out the shared entries, four per thread and round.  What is
// read here is not written here, unless the call works in place: then one workgroup reads all of it first.  Bound by the latency of
// its chain of loads: 48 forks that share 2500 entries, 7 us.
static __global__ __launch_bounds__(kKvTableThreads) void k_kv_fork(KvForkArgs x) {
    const KvPagesArgs &a = x.p;
    __shared__ uint32_t s_first[PI_KV_MAX_REQ + 1];
    __shared__ uint32_t s_pair[PI_KV_MAX_REQ];        // source | destination << 16
    __shared__ int s_claim[PI_KV_MAX_REQ];            // first fork to name a destination
    __shared__ uint32_t s_part[kKvTableThreads / 64];
    __shared__ uint32_t s_done;
    const int tid = threadIdx.x, threads = blockDim.x, n = x.n_fork, per = (n + threads - 1) / threads, page = 1 << a.page_log;
    const int64_t room = (int64_t)a.max_pages << a.page_log;
    const int pool0 = a.pool[0], pool1 = a.pool[1];
    if (tid == 0) s_done = 0;
    int s[kKvReqPerThread], d[kKvReqPerThread];
#pragma unroll
    for (int k = 0; k < kKvReqPerThread; ++k) {
        const int i = tid * per + k;
        const bool in = k < per && i < n;
        s[k] = in ? x.src[i] : -1;
        d[k] = in ? x.dst[i] : -1;
    }
    for (int r = tid; r < a.n_req; r += threads) s_claim[r] = INT32_MAX;
    __syncthreads();
    int len[kKvReqPerThread], there[kKvReqPerThread], old[kKvReqPerThread], fresh[kKvReqPerThread];
    bool ok[kKvReqPerThread], part[kKvReqPerThread];
#pragma unroll
    for (int k = 0; k < kKvReqPerThread; ++k) {
        if ((uint32_t)d[k] < (uint32_t)a.n_req) atomicMin(&s_claim[d[k]], tid * per + k);
        ok[k] = (uint32_t)s[k] < (uint32_t)a.n_req && (uint32_t)d[k] < (uint32_t)a.n_req && s[k] != d[k];
        len[k] = ok[k] ? a.cached[s[k]] : 0;
        there[k] = ok[k] ? a.cached[d[k]] : 0;
    }
    int head = pool0 % a.n_pages;
    if (head < 0) head += a.n_pages;
    const int count = min(max(pool1, 0), a.n_pages);
    __syncthreads();
    uint32_t asks = 0;
#pragma unroll
    for (int k = 0; k < kKvReqPerThread; ++k) {
        ok[k] = ok[k] && len[k] >= 0 && len[k] <= room && there[k] == 0 && s_claim[d[k]] == tid * per + k;
        part[k] = ok[k] && (len[k] & (page - 1));
        old[k] = part[k] ? a.table[(int64_t)s[k] * a.table_stride + (len[k] >> a.page_log)] : -1;
    }
#pragma unroll
    for (int k = 0; k < kKvReqPerThread; ++k) {
        if ((uint32_t)old[k] >= (uint32_t)a.n_pages) old[k] = -1;
        asks += old[k] >= 0;
    }
    uint32_t total_asks, total;
    uint32_t rank = kv_block_scan(asks, s_part, &total_asks);
    uint32_t entries = 0, mine[kKvReqPerThread];
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
        if (ok[k]) mine[k] = (uint32_t)(len[k] >> a.page_log);
        entries += mine[k];
        s_pair[i] = ok[k] ? (uint32_t)s[k] | (uint32_t)d[k] << 16 : 0u;
    }
    uint32_t done = 0;
#pragma unroll
    for (int k = 0; k < kKvReqPerThread; ++k) done += (uint32_t)__popcll(__ballot(k < per && tid * per + k < n && ok[k]));
    if ((tid & 63) == 0 && done) atomicAdd(&s_done, done);
    uint32_t at = kv_block_scan(entries, s_part, &total);
#pragma unroll
    for (int k = 0; k < kKvReqPerThread; ++k) {
        const int i = tid * per + k;
        if (k < per && i < n) s_first[i] = at;
        at += mine[k];
    }
    if (blockIdx.x == 0) {
        if (a.cached_next != a.cached)
            for (int r = tid; r < a.n_req; r += threads) a.cached_next[r] = a.cached[r];
        __syncthreads();
#pragma unroll
        for (int k = 0; k < kKvReqPerThread; ++k) {
            const int i = tid * per + k;
            if (k >= per || i >= n) continue;
            x.copies[2 * i] = old[k];
            x.copies[2 * i + 1] = fresh[k];
            if (!ok[k]) continue;
            a.cached_next[d[k]] = len[k];
            if (part[k]) a.table[(int64_t)d[k] * a.table_stride + (len[k] >> a.page_log)] = fresh[k];
        }
        if (tid == 0) {
            const uint32_t taken = min(total_asks, (uint32_t)count);
            a.pool_next[0] = (int)(((int64_t)head + taken) % a.n_pages);
            a.pool_next[1] = (int)((int64_t)count - taken);
            a.counts[0] = (int)s_done;
            a.counts[1] = (int)total;
            a.counts[2] = (int)taken;
            a.counts[3] = n - (int)s_done;
        }
    }
    __syncthreads();
    const uint32_t stride = gridDim.x * threads * kKvEach;
    for (uint32_t e0 = (blockIdx.x * threads + tid) * kKvEach; e0 < total; e0 += stride) {
        int i = kv_owner_of(s_first, n, e0);
        int *to[kKvEach], p[kKvEach];
#pragma unroll
        for (int j = 0; j < kKvEach; ++j) {
            const uint32_t e = e0 + j;
            to[j] = nullptr;
            if (e >= total) continue;
            while (i + 1 < n && s_first[i + 1] <= e) ++i;
            const uint32_t pair = s_pair[i], col = e - s_first[i];
            p[j] = a.table[(int64_t)(pair & 0xffff) * a.table_stride + col];
            to[j] = a.table + (int64_t)(pair >> 16) * a.table_stride + col;
        }
#pragma unroll
        for (int j = 0; j < kKvEach; ++j) {
            if (!to[j]) continue;
            *to[j] = p[j];
            if ((uint32_t)p[j] < (uint32_t)a.n_pages) atomicAdd(a.shares + p[j], 1);
        }
    }
}

struct KvCopyArgs {
    const int *copies;
    int n_pages;
    int64_t units;            // of 16 bytes, of one page's keys (as many of values)
    f32x4 *k, *v;
};

// Workgroup (pair and operand, part): 16 KB at a time, every gridDim.y-th.  Bound by HBM: 48 pages of 1 MB, 94 MB moved, 17.7 us
// a pass in a run of them.  The stores go past the caches (19.0 us otherwise; loads as well: 20.1).
static __global__ __launch_bounds__(256) void k_kv_copy(KvCopyArgs a) {
    const int i = blockIdx.x >> 1;
    const int from = a.copies[2 * i], to = a.copies[2 * i + 1];
    if ((uint32_t)from >= (uint32_t)a.n_pages || (uint32_t)to >= (uint32_t)a.n_pages || from == to) return;
    f32x4 *const base = blockIdx.x & 1 ? a.v : a.k;
    const f32x4 *const src = base + from * a.units;
    f32x4 *const dst = base + to * a.units;
    constexpr int kDeep = 4;
    for (int64_t u0 = (int64_t)blockIdx.y * (256 * kDeep) + threadIdx.x; u0 < a.units; u0 += (int64_t)gridDim.y * (256 * kDeep)) {
        f32x4 x[kDeep];
#pragma unroll
        for (int j = 0; j < kDeep; ++j)
            if (u0 + j * 256 < a.units) x[j] = src[u0 + j * 256];
#pragma unroll
        for (int j = 0; j < kDeep; ++j)
            if (u0 + j * 256 < a.units) __builtin_nontemporal_store(x[j], dst + u0 + j * 256);
    }
}

}  // namespace pik
