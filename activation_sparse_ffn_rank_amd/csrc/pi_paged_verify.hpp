// pi_paged_verify.hpp -- gfx950 kernel that decides which drafted tokens stay and draws the next one (k_kv_verify).
//
// The acceptance tests need two numbers each; the sample needs one row of the target's probabilities and, after a
// rejection, one of the draft's.  That row is cut into pieces of kKvPiece entries whose weights the request's workgroups sum;
// the last of them to finish adds the sums up in order and reads the piece in which the running sum passes its mark once more.
#pragma once

#include "pi_paged.hpp"

namespace pik {

constexpr int kKvPieceLog = 10, kKvPiece = 1 << kKvPieceLog;
constexpr int kKvMaxPieces = PI_KV_MAX_VOCAB / kKvPiece;

struct KvVerifyArgs {
    int n_req, rows, vocab, pieces, per_wave;
    int64_t p_stride, q_stride;
    const int *q_start, *tokens, *kv_len;
    const float *p, *q, *u_accept, *u_next;
    int *accepted, *next, *keep;
    int *tickets;                  // [n_req] workgroups that have finished; zero between calls
    double *sums;                  // [n_req][pieces]
};

// Sums pass between workgroups of any XCD: written and read past the L2 of either.
__device__ __forceinline__ void kv_put(double *p, double x) { __hip_atomic_store(p, x, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT); }
__device__ __forceinline__ double kv_get(const double *p) {
    return __hip_atomic_load(const_cast<double *>(p), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

struct KvVerdict {
    int rows, accepted;            // of the request; rows = 0: none, or a range out of bounds
    int at;                        // the row after the accepted drafts
    bool rejected;
    int token;                     // the rejected draft
};
// Lanes test 64 drafts at a time.  All lanes return the same.
__device__ __forceinline__ KvVerdict kv_verdict(const KvVerifyArgs &a, int r, int lane) {
    KvVerdict x{0, 0, 0, false, -1};
    const int start = a.q_start[r], end = a.q_start[r + 1];
    if (start < 0 || end <= start || end > a.rows) return x;
    x.rows = end - start;
    for (int i0 = 0; i0 < x.rows - 1; i0 += 64) {
        const int i = i0 + lane, t = start + i;
        bool ok = true;
        int token = -1;
        if (i < x.rows - 1) {
            token = a.tokens[t + 1];
            ok = false;
            if ((uint32_t)token < (uint32_t)a.vocab) {
                const double q = a.q ? (double)a.q[t * a.q_stride + token] : 1.0;
                ok = (double)a.u_accept[t] * q < (double)a.p[t * a.p_stride + token];
            }
        }
        const uint64_t bad = __ballot(!ok);
        if (bad) {
            const int l = __builtin_ctzll(bad);
            x.accepted = i0 + l;
            x.rejected = true;
            x.token = bcast(token, l);
            break;
        }
        x.accepted = min(i0 + 64, x.rows - 1);
    }
    x.at = start + x.accepted;
    return x;
}

// Four neighbouring floats at a 4-byte aligned address.
struct KvQuad {
    float v[4];
} __attribute__((packed, aligned(4)));

// Weights of entries j .. j+3 of the row that is drawn from.  q NULL: all of the draft's probability is on `token`.
struct KvWeights {
    const float *p, *q;
    int vocab, token;              // token < 0: none is left out
    __device__ __forceinline__ double weight(double p_j, double q_j, int j) const {
        const double w = p_j - q_j;
        return w > 0.0 && j != token ? w : 0.0;            // (NaN: 0)
    }
    __device__ __forceinline__ void load(int j, KvQuad &x, KvQuad &y) const {
        y = KvQuad{{0.f, 0.f, 0.f, 0.f}};
        if (j + 4 <= vocab) {
            x = *reinterpret_cast<const KvQuad *>(p + j);
            if (q) y = *reinterpret_cast<const KvQuad *>(q + j);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                x.v[i] = j + i < vocab ? p[j + i] : 0.f;
                if (q) y.v[i] = j + i < vocab ? q[j + i] : 0.f;
            }
        }
    }
};
__device__ __forceinline__ KvWeights kv_weights_of(const KvVerifyArgs &a, const KvVerdict &v, bool rest) {
    return {a.p + v.at * a.p_stride, rest && a.q ? a.q + v.at * a.q_stride : nullptr, a.vocab, rest && !a.q ? v.token : -1};
}

__device__ __forceinline__ double kv_wave_sum(double x) {
#pragma unroll
    for (int b = 1; b < 64; b <<= 1) x += __shfl_xor(x, b);
    return x;
}

// Sum of piece i of a row, by one wave.
__device__ __forceinline__ double kv_piece_sum(const KvWeights &w, int i, int lane) {
    constexpr int kLoads = kKvPiece / 256;
    KvQuad x[kLoads], y[kLoads];
    const int j0 = (i << kKvPieceLog) + lane * 4;
#pragma unroll
    for (int k = 0; k < kLoads; ++k) w.load(j0 + k * 256, x[k], y[k]);
    double sum = 0.0;
#pragma unroll
    for (int k = 0; k < kLoads; ++k)
#pragma unroll
        for (int e = 0; e < 4; ++e) sum += w.weight(x[k].v[e], y[k].v[e], j0 + k * 256 + e);
    return kv_wave_sum(sum);
}

// Sum over the threads before this one, in a fixed order; *total: of all.  sums: one per thread.
__device__ __forceinline__ double kv_block_sums(double x, double *sums, double *part, double *total) {
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, waves = blockDim.x >> 6;
#pragma unroll
    for (int b = 1; b < 64; b <<= 1) {
        const double y = __shfl_up(x, b);
        if (lane >= b) x += y;
    }
    __syncthreads();                       // what the call before left may still be read
    if (lane == 63) part[wave] = x;
    __syncthreads();
    double before = 0.0, all = 0.0;
    for (int w = 0; w < waves; ++w) {
        before += w < wave ? part[w] : 0.0;
        all += part[w];
    }
    *total = all;
    sums[tid] = before + x;
    __syncthreads();
    return tid ? sums[tid - 1] : 0.0;
}

// The lowest thread's `first` that is not INT32_MAX, else the highest thread's `last` that is not -1, else -1; both grow with the
// thread.  (By votes: minima in LDS took 5 us here, a step per lane.)  found: two ints per wave.
__device__ __forceinline__ int kv_first_or_last(int first, int last, int *found) {
    const int wave = threadIdx.x >> 6, waves = blockDim.x >> 6;
    const uint64_t some = __ballot(first != INT32_MAX), any = __ballot(last >= 0);
    if ((threadIdx.x & 63) == 0) {
        found[2 * wave] = INT32_MAX;
        found[2 * wave + 1] = -1;
    }
    if (some) found[2 * wave] = bcast(first, __builtin_ctzll(some));
    if (any) found[2 * wave + 1] = bcast(last, 63 - __builtin_clzll(any));
    __syncthreads();
    int low = INT32_MAX, high = -1;
    for (int w = 0; w < waves; ++w) {
        low = min(low, found[2 * w]);
        high = max(high, found[2 * w + 1]);
    }
    return low != INT32_MAX ? low : high;
}

// Bound by HBM for many requests (96 of them, two rows of 100003 each, 77 MB: 19.1 us a pass, of which the row sums end at about
// 14), by latency for few: one request, 32000 tokens, 7.3 us, of which verdict 1, sums 1.5, their way to the last workgroup 2, its
// sums, piece and draw 2.
// Workgroup (group of pieces, request).  The last one of a request draws: an entry without weight is never taken, and where
// rounding leaves none above the mark it is the last one with weight.
static __global__ __launch_bounds__(256) void k_kv_verify(KvVerifyArgs a) {
    __shared__ double s_part[4], s_sums[256], s_before;
    __shared__ int s_found[2][8], s_end;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, r = blockIdx.y;
    const float u_next = a.u_next[r];
    // Every workgroup has read this before the last one writes `keep`, which may lie in its place (tickets between).
    const int keys = a.kv_len ? a.kv_len[r] : INT32_MAX;
    const KvVerdict v = kv_verdict(a, r, lane);
    if (v.rows == 0) {                     // (no tickets: this workgroup's lengths are its own)
        if (tid == 0 && blockIdx.x == 0) {
            a.accepted[r] = 0;
            a.next[r] = -1;
            if (a.keep) a.keep[r] = keys > 0 ? keys : INT32_MAX;
        }
        return;
    }
    // A step that refuses a request gives it no keys: its scores stand for nothing, and its cache has none of its rows.
    const bool refused = keys < v.rows;
    KvWeights w = kv_weights_of(a, v, v.rejected);
    double *const sums = a.sums + (int64_t)r * a.pieces;
    if (!refused) {
        const int from = (blockIdx.x * 4 + wave) * a.per_wave, to = min(from + a.per_wave, a.pieces);
        for (int i = from; i < to; ++i) {
            const double sum = kv_piece_sum(w, i, lane);
            if (lane == 0) kv_put(sums + i, sum);
        }
    }
    kv_lds_wait();                         // this wave's sums are out
    __syncthreads();                       // ... and so are the others'
    if (gridDim.x > 1) {
        if (tid == 0) s_end = atomicAdd(a.tickets + r, 1) == (int)gridDim.x - 1;
        __syncthreads();
        if (!s_end) return;
        if (tid == 0) a.tickets[r] = 0;
    }
    if (tid == 0) {
        a.accepted[r] = refused ? 0 : v.accepted;
        if (refused) a.next[r] = a.tokens[a.q_start[r]];
        if (a.keep) a.keep[r] = refused ? INT32_MAX : keys - (v.rows - 1 - v.accepted);
    }
    if (refused) return;
    const int per = (a.pieces + 255) / 256, i0 = tid * per, i1 = min(i0 + per, a.pieces);
    double upto, total, one;               // one: of the thread's first piece, most often its only one
    for (bool again = false;; again = true) {
        one = i0 < i1 ? kv_get(sums + i0) : 0.0;
        double mine = one;
        for (int i = i0 + 1; i < i1; ++i) mine += kv_get(sums + i);
        upto = kv_block_sums(mine, s_sums, s_part, &total);
        if (total > 0.0 || again || !v.rejected) break;
        // nothing is left of the rest: the target's own weights
        w = kv_weights_of(a, v, false);
        for (int i = wave; i < a.pieces; i += 4) {
            const double sum = kv_piece_sum(w, i, lane);
            if (lane == 0) kv_put(sums + i, sum);
        }
        kv_lds_wait();
        __syncthreads();
    }
    if (!(total > 0.0)) {
        if (tid == 0) a.next[r] = -1;
        return;
    }
    const double mark = (double)u_next * total;
    // the first of this thread's pieces to pass the mark, and its last one, with the sums before them
    int first = INT32_MAX, last = -1;
    double to_first = 0.0, to_last = 0.0;
    for (int i = i0; i < i1; ++i) {
        const double x = i == i0 ? one : kv_get(sums + i);
        if (!(x > 0.0)) continue;
        last = i, to_last = upto;
        if (first == INT32_MAX && upto + x > mark) first = i, to_first = upto;
        upto += x;
    }
    const int piece = kv_first_or_last(first, last, s_found[0]);
    if (piece == first) s_before = to_first;
    else if (piece == last) s_before = to_last;
    const int j0 = (piece << kKvPieceLog) + tid * 4;
    KvQuad x, y;
    w.load(j0, x, y);
    double each[4], sum = 0.0;
#pragma unroll
    for (int e = 0; e < 4; ++e) sum += each[e] = w.weight(x.v[e], y.v[e], j0 + e);
    double at = kv_block_sums(sum, s_sums, s_part, &total) + s_before;      // (its barriers order s_before, too)
    first = INT32_MAX, last = -1;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        at += each[e];
        if (!(each[e] > 0.0)) continue;
        last = j0 + e;
        if (first == INT32_MAX && at > mark) first = j0 + e;
    }
    const int token = kv_first_or_last(first, last, s_found[1]);
    if (tid == 0) a.next[r] = token;
}

}  // namespace pik
