// pi_paged_verify.hip -- host side of pi_kv_verify (include/pi_paged_kv.h).
#include "pi_paged_host.hpp"
#include "pi_paged_verify.hpp"

#include <algorithm>

namespace {

using namespace pik;

int check_drafts(const pi_kv_drafts *d) {
    if (!d || !d->q_start || !d->tokens || !d->target || !d->u_accept || !d->u_next) return PI_ERR_NULL;
    if (d->n_req < 1 || d->n_req > PI_KV_MAX_REQ || d->rows < 1 || d->rows > PI_KV_MAX_TOKENS || d->vocab < 1 ||
        d->vocab > PI_KV_MAX_VOCAB || d->target_stride < (d->rows > 1 ? d->vocab : 0) ||
        (d->draft && d->draft_stride < (d->rows > 1 ? d->vocab : 0)))
        return PI_ERR_SHAPE;
    return PI_OK;
}

int pieces_of(const pi_kv_drafts *d) { return (d->vocab + kKvPiece - 1) / kKvPiece; }

// Tickets first, as many for any call, so that the calls that share a workspace find theirs at zero.
constexpr size_t kTicketBytes = PI_KV_MAX_REQ * sizeof(int32_t);
size_t bytes_of(const pi_kv_drafts *d) { return kTicketBytes + (size_t)d->n_req * pieces_of(d) * sizeof(double); }

}  // namespace

extern "C" size_t pi_kv_verify_workspace_bytes(const pi_kv_drafts *drafts) { return check_drafts(drafts) ? 0 : bytes_of(drafts); }

extern "C" int pi_kv_verify(const pi_kv_drafts *drafts, const int32_t *kv_len, int32_t *accepted, int32_t *next, int32_t *keep,
                            void *ws, size_t ws_bytes, void *stream) {
    if (int rc = check_drafts(drafts)) return rc;
    if (!accepted || !next || !kv_len != !keep) return PI_ERR_NULL;
    if (((reinterpret_cast<uintptr_t>(drafts->target) | reinterpret_cast<uintptr_t>(drafts->draft)) & 3u) != 0) return PI_ERR_ALIGN;
    if (!ws || ws_bytes < bytes_of(drafts)) return PI_ERR_WORKSPACE;
    if (!aligned16(ws)) return PI_ERR_ALIGN;
    KvVerifyArgs a{};
    a.n_req = drafts->n_req, a.rows = drafts->rows, a.vocab = drafts->vocab, a.pieces = pieces_of(drafts);
    a.p_stride = drafts->target_stride, a.q_stride = drafts->draft_stride;
    a.q_start = drafts->q_start, a.tokens = drafts->tokens, a.kv_len = kv_len;
    a.p = drafts->target, a.q = drafts->draft, a.u_accept = drafts->u_accept, a.u_next = drafts->u_next;
    a.accepted = accepted, a.next = next, a.keep = keep, a.tickets = static_cast<int32_t *>(ws);
    a.sums = reinterpret_cast<double *>(static_cast<char *>(ws) + kTicketBytes);
    // pieces a wave takes one after another: one while the chip holds all waves
    a.per_wave = 1;
    while (a.per_wave < 16 && (int64_t)a.n_req * a.pieces > (int64_t)a.per_wave * 8192) a.per_wave *= 2;
    hipStream_t st = static_cast<hipStream_t>(stream);
    const int groups = (a.pieces + 4 * a.per_wave - 1) / (4 * a.per_wave);
    hipLaunchKernelGGL(k_kv_verify, dim3(groups, a.n_req), dim3(256), 0, st, a);
    return hipGetLastError() == hipSuccess ? PI_OK : PI_ERR_HIP;
}
