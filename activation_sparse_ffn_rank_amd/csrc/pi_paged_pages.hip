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

KvPagesArgs args_of(const pi_kv_pages *p) {
    return {p->n_req, page_log(p->page), p->n_pages, p->max_pages, p->table_stride, p->cached, p->free_ring, p->pool,
            p->block_table, p->shares, p->cached_next, p->pool_next, p->counts};
}

}  // namespace

extern "C" int pi_kv_release(const pi_kv_pages *pages, const int32_t *drop_from, const int32_t *drop_to, int32_t *copies,
                             void *stream) {
    if (int rc = check_pages(pages)) return rc;
    if (!drop_from || !copies) return PI_ERR_NULL;
    const KvReleaseArgs a{args_of(pages), drop_from, drop_to, copies};
    hipLaunchKernelGGL(k_kv_release, dim3(1), dim3(kKvTableThreads), 0, static_cast<hipStream_t>(stream), a);
    return hipGetLastError() == hipSuccess ? PI_OK : PI_ERR_HIP;
}

extern "C" int pi_kv_fork(const pi_kv_pages *pages, const int32_t *src, const int32_t *dst, int32_t n_fork, int32_t *copies,
                          void *stream) {
    if (int rc = check_pages(pages)) return rc;
    if (n_fork < 0 || n_fork > PI_KV_MAX_REQ) return PI_ERR_SHAPE;
    if (n_fork > 0 && (!src || !dst || !copies)) return PI_ERR_NULL;
    const KvForkArgs a{args_of(pages), src, dst, n_fork, copies};
    hipLaunchKernelGGL(k_kv_fork, dim3(1), dim3(kKvTableThreads), 0, static_cast<hipStream_t>(stream), a);
    return hipGetLastError() == hipSuccess ? PI_OK : PI_ERR_HIP;
}

extern "C" int pi_kv_copy(const pi_kv_cache *cache, const int32_t *copies, int32_t n, void *stream) {
    if (int rc = check_cache(cache)) return rc;
    if (n < 0 || n > PI_KV_MAX_TOKENS) return PI_ERR_SHAPE;
    if (n == 0) return PI_OK;
    if (!copies) return PI_ERR_NULL;
    const int64_t units = (int64_t)cache->n_kv * cache->page * cache->head_dim / 8;
    const KvCopyArgs a{copies, cache->n_pages, units, static_cast<uint4 *>(cache->k_pages), static_cast<uint4 *>(cache->v_pages)};
    const int64_t parts = (units + 1023) / 1024, share = std::max<int64_t>(1, 2048 / (2 * (int64_t)n));
    hipLaunchKernelGGL(k_kv_copy, dim3((uint32_t)(2 * (int64_t)n), (uint32_t)std::min(parts, share)), dim3(256), 0,
                       static_cast<hipStream_t>(stream), a);
    return hipGetLastError() == hipSuccess ? PI_OK : PI_ERR_HIP;
}
