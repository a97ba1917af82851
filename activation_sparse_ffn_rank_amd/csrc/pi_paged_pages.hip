// pi_paged_pages.hip -- host side of pi_kv_release, pi_kv_fork and pi_kv_copy (include/pi_paged_kv.h).
#include "pi_paged_host.hpp"
#include "pi_paged_pages.hpp"

#include <algorithm>

namespace {

using namespace pik;

int check_pages(const pi_kv_pages *p) {
    if (!p || !p->cached || !p->free_ring || !p->pool || !p->block_table || !p->shares || !p->cached_next || !p->pool_next || !p->counts)
        return PI_ERR_NULL;
    if (p->n_req < 1 || p->n_req > PI_KV_MAX_REQ || page_log(p->page) < 0 || p->n_pages < 1 || p->max_pages < 1 ||
        p->max_pages > PI_KV_MAX_TABLE || p->table_stride < p->max_pages || (int64_t)p->n_pages * p->page > INT32_MAX ||
        (int64_t)p->max_pages * p->page > INT32_MAX)
        return PI_ERR_SHAPE;
    return PI_OK;
}

// By the entries that all tables have together: up to the first number a workgroup of few threads where requests are few, for its
// barriers' sake; up to the second one of many, as a list of thousands may come; past it, launches over the whole chip for long
// lists follow, which cost where there is none.  64 requests of 1024 pages, one workgroup and with the launches: 6.5 us and 11.2
// where a step gives nothing up, 18 and 26 where four requests end, 56 and 28 where sixteen do.  A list of 400 entries with 256
// threads 5.0 us, with 1024 6.5; one of 4096 46 and 18.
constexpr int64_t kFewEntries = 32768, kManyEntries = 131072;
int64_t entries_of(const pi_kv_pages *p) { return (int64_t)p->n_req * p->max_pages; }
bool long_lists(const pi_kv_pages *p) { return entries_of(p) > kManyEntries; }

size_t bytes_of(const pi_kv_pages *p) { return long_lists(p) ? KvReleaseWs::kInts * sizeof(int32_t) : 16; }

// Threads of a workgroup that holds four requests or forks each at most.
int threads_for(int n) { return n <= 256 ? 256 : kKvTableThreads; }

KvPagesArgs args_of(const pi_kv_pages *p) {
    return {p->n_req, page_log(p->page), p->n_pages, p->max_pages, p->table_stride, p->cached, p->free_ring, p->pool,
            p->block_table, p->shares, p->cached_next, p->pool_next, p->counts};
}

}  // namespace

extern "C" size_t pi_kv_pages_workspace_bytes(const pi_kv_pages *pages) { return check_pages(pages) ? 0 : bytes_of(pages); }

extern "C" int pi_kv_release(const pi_kv_pages *pages, const int32_t *drop_from, const int32_t *drop_to, int32_t *copies,
                             void *stream) {
    if (int rc = check_pages(pages)) return rc;
    if (!drop_from || !copies) return PI_ERR_NULL;
    if (!pages->ws || pages->ws_bytes < bytes_of(pages)) return PI_ERR_WORKSPACE;
    if (!aligned16(pages->ws)) return PI_ERR_ALIGN;
    const bool more = long_lists(pages);
    const KvReleaseArgs a{args_of(pages), drop_from, drop_to, copies, more ? static_cast<int32_t *>(pages->ws) : nullptr};
    hipStream_t st = static_cast<hipStream_t>(stream);
    const int threads = entries_of(pages) <= kFewEntries ? threads_for(pages->n_req) : kKvTableThreads;
    hipLaunchKernelGGL(k_kv_release, dim3(1), dim3(threads), 0, st, a);
    if (more) {
        hipLaunchKernelGGL(k_kv_release_pass<0>, dim3(kKvReleaseGroups), dim3(256), 0, st, a);
        hipLaunchKernelGGL(k_kv_release_pass<1>, dim3(kKvReleaseGroups), dim3(256), 0, st, a);
        hipLaunchKernelGGL(k_kv_release_pass<2>, dim3(kKvReleaseGroups), dim3(256), 0, st, a);
        hipLaunchKernelGGL(k_kv_release_pass<3>, dim3(kKvReleaseGroups), dim3(256), 0, st, a);
    }
    return hipGetLastError() == hipSuccess ? PI_OK : PI_ERR_HIP;
}

extern "C" int pi_kv_fork(const pi_kv_pages *pages, const int32_t *src, const int32_t *dst, int32_t n_fork, int32_t *copies,
                          void *stream) {
    if (int rc = check_pages(pages)) return rc;
    if (n_fork < 0 || n_fork > PI_KV_MAX_REQ) return PI_ERR_SHAPE;
    if (n_fork > 0 && (!src || !dst || !copies)) return PI_ERR_NULL;
    const KvForkArgs a{args_of(pages), src, dst, n_fork, copies};
    const bool in_place = pages->cached_next == pages->cached || pages->pool_next == pages->pool;
    const int threads = threads_for(n_fork);
    const int64_t rounds = ((int64_t)n_fork * pages->max_pages + threads * kKvEach - 1) / (threads * kKvEach);
    const int groups = in_place ? 1 : (int)std::min<int64_t>(32, std::max<int64_t>(1, rounds));
    hipLaunchKernelGGL(k_kv_fork, dim3(groups), dim3(threads), 0, static_cast<hipStream_t>(stream), a);
    return hipGetLastError() == hipSuccess ? PI_OK : PI_ERR_HIP;
}

extern "C" int pi_kv_copy(const pi_kv_cache *cache, const int32_t *copies, int32_t n, void *stream) {
    if (int rc = check_cache(cache)) return rc;
    if (n < 0 || n > PI_KV_MAX_TOKENS) return PI_ERR_SHAPE;
    if (n == 0) return PI_OK;
    if (!copies) return PI_ERR_NULL;
    const int64_t units = (int64_t)cache->n_kv * cache->page * cache->head_dim / 8;
    const KvCopyArgs a{copies, cache->n_pages, units, static_cast<f32x4 *>(cache->k_pages), static_cast<f32x4 *>(cache->v_pages)};
    // 16 KB a round: as many workgroups for a page as make 4096 of them all, the rounds shared out evenly
    const int64_t rounds = (units + 1023) / 1024, most = std::max<int64_t>(1, 4096 / (2 * (int64_t)n));
    const int64_t each = (rounds + most - 1) / most, parts = (rounds + each - 1) / each;
    hipLaunchKernelGGL(k_kv_copy, dim3((uint32_t)(2 * (int64_t)n), (uint32_t)parts), dim3(256), 0,
                       static_cast<hipStream_t>(stream), a);
    return hipGetLastError() == hipSuccess ? PI_OK : PI_ERR_HIP;
}
