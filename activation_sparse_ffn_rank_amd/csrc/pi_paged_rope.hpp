// pi_paged_rope.hpp -- gfx950 kernel of the append with rotary positions and head norms (k_kv_rope).
//
// A head of 16 L elements (L = 4, 8 or 16) is held by L neighbouring lanes, 16 elements each in two 16-byte pieces that
// hold both elements of 8 pairs: elements 8l .. 8l+7 and the same rot_dim/2 further on for halves (those past rot_dim alike, their own
// half further on), the same HD/2 further on for neighbours.  Either piece of the lanes of a head is contiguous.  The mean of the
// squares is a sum over L lanes, and a rotation touches one lane's registers only.
#pragma once

#include "pi_paged.hpp"

namespace pik {

struct KvRopeArgs {
    int n_req, total_q, n_q, n_kv, page_log, n_slots, rot, norm;
    int per_wave, parts;              // heads that a group of lanes takes one after another; waves that share out a token's heads
    int v_groups, v_tile;             // workgroups that transpose values, numbered first, and tokens of each
    float scale, eps;
    int64_t q_ts, q_hs, k_ts, k_hs, v_ts, v_hs, o_ts, o_hs;
    const uint16_t *q, *k, *v, *q_weight, *k_weight;
    const double *freq;
    const int *slots, *q_start, *kv_len;
    uint16_t *q_out, *k_pages, *v_pages;
};

// q_start is searched 64 entries at a time, by all lanes of a wave: the number of starts at or before a row names its request.  For
// a row's heads and for its values alike, so that with starts that decrease, where a search may miss a row's range, both
// leave it out.  This lane's share of the first search: the start of every step-th request, with one request a lane its end and
// keys, too.
struct KvStarts {
    int step, start, end, m;
};
__device__ __forceinline__ KvStarts kv_starts(const KvRopeArgs &a, int lane) {
    const int step = (a.n_req + 63) / 64, at = lane * step;
    const bool in = at < a.n_req, all = step == 1 && in;
    return {step, in ? a.q_start[at] : INT32_MAX, all ? a.q_start[at + 1] : 0, all ? a.kv_len[at] : 0};
}
__device__ __forceinline__ int kv_starts_upto(int start, int t) { return __popcll(__ballot(start <= t)); }
__device__ __forceinline__ bool kv_in_range(const KvRopeArgs &a, int t, int start, int end) {
    return start >= 0 && t >= start && t < end && end <= a.total_q;
}

// Where packed row t stands (in: it belongs to a request).
struct KvPlace {
    bool in;
    int64_t pos;
};
__device__ __forceinline__ KvPlace kv_place(const KvRopeArgs &a, int t, int lane) {
    const KvStarts s = kv_starts(a, lane);
    int start = s.start, end = s.end, m = s.m;
    int l = kv_starts_upto(start, t) - 1;
    if (l < 0) return {false, 0};
    if (s.step > 1) {
        const int r = l * s.step + lane;
        const bool in = lane < s.step && r < a.n_req;
        start = in ? a.q_start[r] : INT32_MAX, end = in ? a.q_start[r + 1] : 0, m = in ? a.kv_len[r] : 0;
        l = kv_starts_upto(start, t) - 1;
        if (l < 0) return {false, 0};                    // (starts that decrease)
    }
    start = bcast(start, l), end = bcast(end, l), m = bcast(m, l);
    return {kv_in_range(a, t, start, end), (int64_t)m - end + t};
}

// Which of rows t .. t + n - 1 (n <= 32) belong to one, a bit each, by the same searches; the second one in 64 requests from the
// first group on, a window that the next rows' groups mostly lie in.
__device__ __forceinline__ uint32_t kv_rows_in(const KvRopeArgs &a, const KvStarts &s, int t, int n, int lane) {
    int start = s.start, end = s.end, base = INT32_MIN / 2;
    uint32_t in = 0;
#pragma unroll 1
    for (int i = 0; i < n; ++i) {
        int l = kv_starts_upto(s.start, t + i) - 1;
        if (l < 0) continue;
        if (s.step > 1) {
            int off = l * s.step - base;
            if (off < 0 || off + s.step > 64) {
                base = l * s.step, off = 0;
                const int r = base + lane;
                start = r < a.n_req ? a.q_start[r] : INT32_MAX, end = r < a.n_req ? a.q_start[r + 1] : 0;
            }
            l = __popcll(__ballot(start <= t + i) & ((~0ull >> (64 - s.step)) << off)) - 1;
            if (l < 0) continue;
            l += off;
        }
        in |= (uint32_t)kv_in_range(a, t + i, bcast(start, l), bcast(end, l)) << i;
    }
    return in;
}

template <class T>
__device__ __forceinline__ void kv_floats(uint4 w, float (&x)[8]) {
    const typename T::v8 v = __builtin_bit_cast(typename T::v8, w);
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = (float)v[i];
}
template <class T>
__device__ __forceinline__ uint4 kv_halves(const float (&x)[8]) {
    return make_uint4(kv_pack<T>(x[0], x[1]), kv_pack<T>(x[2], x[3]), kv_pack<T>(x[4], x[5]), kv_pack<T>(x[6], x[7]));
}

// Sum over groups of L neighbouring lanes (4, 8, 16).
template <int L>
__device__ __forceinline__ float kv_lane_sum(float x) {
    auto add = [](float x, float y) { return x + y; };
#define KV_DPP(ctrl) __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, x), ctrl, 0xF, 0xF, true))
    x = add(x, KV_DPP(0xB1));                        // lane ^ 1
    x = add(x, KV_DPP(0x4E));                        // lane ^ 2
    if (L >= 8) x = add(x, KV_DPP(0x141));           // 7 - lane of 8
    if (L >= 16) x = add(x, KV_DPP(0x140));          // 15 - lane of 16
#undef KV_DPP
    return x;
}

// TT tokens of one kv head's values, transposed through LDS as k_kv_append does.
template <int HD, int TT>
__device__ __forceinline__ void kv_values(const KvRopeArgs &a, uint32_t *s_v) {
    constexpr int per = HD / 8, kLdsRow = HD / 2 + 1, kRows = TT / 4, kLoads = (TT * per + 255) / 256;
    __shared__ uint32_t s_in[4];                     // rows that belong to a request, by the waves that look for them
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int h = blockIdx.x % a.n_kv, t0 = blockIdx.x / a.n_kv * TT, nt = min(TT, a.total_q - t0);
    const int t = tid & (TT - 1);
    const KvStarts starts = kv_starts(a, lane);
    const uint32_t slot = t < nt ? (uint32_t)a.slots[t0 + t] : 0xffffffffu;
    uint4 x[kLoads];
#pragma unroll
    for (int k = 0; k < kLoads; ++k) {
        const int i = tid + 256 * k, u = i / per, ch = i - u * per;
        if (u < nt) x[k] = ld16(a.v + (t0 + u) * a.v_ts + h * a.v_hs + ch * 8);
    }
    // With a request a lane it takes one vote to see that no start decreases; then all rows between the first and the last of them
    // belong to one, if no range leaves the rows.  (Each row looked for in turn, whatever the starts: 4096 tokens of 96 heads
    // 124.8 us a pass and 122 so, 16 of 32 heads 4.4 us of kernel and 4.1.)
    const int first = bcast(starts.start, 0), end = bcast(starts.end, (a.n_req - 1) & 63);
    const bool plain = starts.step == 1 && !__any(lane < a.n_req && starts.start > starts.end) && first >= 0 && end <= a.total_q;
    bool in = t0 + t >= first && t0 + t < end;
    if (!plain) s_in[wave] = kv_rows_in(a, starts, t0 + wave * kRows, kRows, lane);
#pragma unroll
    for (int k = 0; k < kLoads; ++k) {
        const int i = tid + 256 * k, u = i / per, ch = i - u * per;
        if (u >= nt) break;
        uint32_t *const d = s_v + u * kLdsRow + ch * 4;
        d[0] = x[k].x, d[1] = x[k].y, d[2] = x[k].z, d[3] = x[k].w;
    }
    __syncthreads();
    if (!plain) in = s_in[t / kRows] >> (t % kRows) & 1;
    if (slot >= (uint32_t)a.n_slots || !in) return;
    const int64_t pg = slot >> a.page_log, off = slot & ((1u << a.page_log) - 1);
    uint16_t *const vp = a.v_pages + (((pg * a.n_kv + h) * HD) << a.page_log) + off;
    for (int d = tid / TT; d < HD / 2; d += 256 / TT) {
        const uint32_t w = s_v[t * kLdsRow + d];
        vp[(int64_t)(2 * d) << a.page_log] = (uint16_t)w;
        vp[(int64_t)(2 * d + 1) << a.page_log] = (uint16_t)(w >> 16);
    }
}

// Workgroups below v_groups take values.  The others: a wave takes one token and some of its query and key heads, 64 / L side by
// side, which it finds next to one another in memory, some rounds of them one after another.  Its lanes compute the cosines and
// sines of a pair each (heads of 256: two) and hand them round through LDS.  (A wave of 16 tokens side by side, each lane with the
// angles of its own pairs, was slower: 24 ragged requests of 2440 tokens, 128/8 heads of 64, 36 us and 30 so; 16 tokens of 32 + 32
// heads 5.1 and 3.7, the least of a trace.)  Queries and keys are stored past the caches: the same ragged rows 30 -> 24 us by
// themselves; together with an attention that reads them at once 2440 ragged rows on 3000 keys take 225 us and 219 with ordinary
// stores of the queries, 1024 rows of 32 heads on 2048 keys 96 and 97.  Norms and rotations are fp32,
// rounded once.  Bound by HBM: 4096 tokens of 96 + 96 heads of 128, 604 MB in 122 us (4.9 TB/s), the ragged rows 115 MB in 24;
// few tokens by the chain q_start -> place -> sines -> store.
template <class T, int HD, bool PAIRS>
__global__ __launch_bounds__(256) void k_kv_rope(KvRopeArgs a) {
    constexpr int L = HD / 16, kSide = 64 / L;
    extern __shared__ uint32_t s_v[];                // values: [v_tile][HD/2 + 1]; others: [wave][2][HD/2] cosines, sines
    if ((int)blockIdx.x < a.v_groups) {
        if (a.v_tile == 64) kv_values<HD, 64>(a, s_v);
        else kv_values<HD, 16>(a, s_v);
        return;
    }
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int w = ((int)blockIdx.x - a.v_groups) * 4 + wave;
    const int part = w % a.parts, t = w / a.parts;
    if (t >= a.total_q) return;
    const int l = lane & (L - 1), g = lane / L, heads = a.n_q + a.n_kv;
    const int hp = part * a.per_wave * kSide, h0 = hp + g, h1 = min(hp + a.per_wave * kSide, heads);
    const int rest = l - a.rot / 16;                                        // of those not turned
    const bool turned0 = PAIRS ? 8 * l < a.rot : rest < 0, turned1 = PAIRS ? HD / 2 + 8 * l < a.rot : rest < 0;
    const int at0 = PAIRS || rest < 0 ? 8 * l : a.rot + 8 * rest;
    const int at1 = at0 + (PAIRS ? HD / 2 : rest < 0 ? a.rot / 2 : (HD - a.rot) / 2);
    const uint16_t *const qs = a.q + t * a.q_ts, *const ks = a.k + t * a.k_ts;
    auto source = [&](int h) { return h < a.n_q ? qs + h * a.q_hs : ks + (h - a.n_q) * a.k_hs; };
    // the first heads' elements, frequencies, weights and slot are on their way while the row's place is found
    uint4 r0 = zero4(), r1 = zero4(), qw0 = zero4(), qw1 = zero4(), kw0 = zero4(), kw1 = zero4();
    if (h0 < h1) {
        r0 = ld16(source(h0) + at0);
        r1 = ld16(source(h0) + at1);
    }
    const uint32_t slot = (uint32_t)a.slots[t];
    constexpr int kPer = HD == 256 ? 2 : 1;
    double freq[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) freq[i] = 2 * (lane + 64 * i) < a.rot ? a.freq[lane + 64 * i] : 0.0;
    if (a.norm && a.q_weight) qw0 = ld16(a.q_weight + at0), qw1 = ld16(a.q_weight + at1);
    if (a.norm && a.k_weight) kw0 = ld16(a.k_weight + at0), kw1 = ld16(a.k_weight + at1);
    const KvPlace place = kv_place(a, t, lane);
    if (!place.in) return;
    float c[8], s[8];
    if (a.rot) {
        float *const cs = reinterpret_cast<float *>(s_v) + wave * HD, *const ss = cs + HD / 2;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            // the angle in turns, less whole ones, in 64 bits: far positions have few bits behind the point
            double x = (double)place.pos * (freq[i] * 0.15915494309189535);
            x -= rint(x);
            float sine, cosine;
            sincospif(2.f * (float)x, &sine, &cosine);
            if (2 * (lane + 64 * i) < HD) cs[lane + 64 * i] = cosine * a.scale, ss[lane + 64 * i] = sine * a.scale;
        }
        __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
        __builtin_amdgcn_wave_barrier();
        __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
        const int p0 = PAIRS ? 4 * l : turned0 ? 8 * l : 0, p1 = PAIRS ? HD / 4 + 4 * l : p0 + 4;
#pragma unroll
        for (int i = 0; i < 4; ++i) c[i] = cs[p0 + i], s[i] = ss[p0 + i], c[4 + i] = cs[p1 + i], s[4 + i] = ss[p1 + i];
    }
    const bool stored = slot < (uint32_t)a.n_slots;
    const int64_t pg = slot >> a.page_log, off = slot & ((1u << a.page_log) - 1);
    uint16_t *const qd = a.q_out + t * a.o_ts, *const kd = a.k_pages + (((pg * a.n_kv) << a.page_log) + off) * HD;
    for (int h = h0; h < h1; h += kSide) {
        const bool key = h >= a.n_q;
        float x0[8], x1[8];
        kv_floats<T>(r0, x0);
        kv_floats<T>(r1, x1);
        if (h + kSide < h1) {                                               // the next heads'
            r0 = ld16(source(h + kSide) + at0);
            r1 = ld16(source(h + kSide) + at1);
        }
        if (a.norm) {
            float sum = 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i) sum += x0[i] * x0[i] + x1[i] * x1[i];
            const float f = 1.f / sqrtf(kv_lane_sum<L>(sum) * (1.f / HD) + a.eps);
#pragma unroll
            for (int i = 0; i < 8; ++i) x0[i] *= f, x1[i] *= f;
            if (key ? a.k_weight != nullptr : a.q_weight != nullptr) {
                float w0[8], w1[8];
                kv_floats<T>(key ? kw0 : qw0, w0);
                kv_floats<T>(key ? kw1 : qw1, w1);
#pragma unroll
                for (int i = 0; i < 8; ++i) x0[i] *= w0[i], x1[i] *= w1[i];
            }
        }
        auto turn = [&](float &p, float &q, int i) {
            const float u = p * c[i] - q * s[i], v = p * s[i] + q * c[i];
            p = u, q = v;
        };
        if (PAIRS) {
            if (turned0)
#pragma unroll
                for (int i = 0; i < 4; ++i) turn(x0[2 * i], x0[2 * i + 1], i);
            if (turned1)
#pragma unroll
                for (int i = 0; i < 4; ++i) turn(x1[2 * i], x1[2 * i + 1], 4 + i);
        } else if (turned0) {
#pragma unroll
            for (int i = 0; i < 8; ++i) turn(x0[i], x1[i], i);
        }
        if (key && !stored) continue;
        uint16_t *const dst = key ? kd + ((int64_t)(h - a.n_q) << a.page_log) * HD : qd + h * a.o_hs;
        __builtin_nontemporal_store(__builtin_bit_cast(f32x4, kv_halves<T>(x0)), reinterpret_cast<f32x4 *>(dst + at0));
        __builtin_nontemporal_store(__builtin_bit_cast(f32x4, kv_halves<T>(x1)), reinterpret_cast<f32x4 *>(dst + at1));
    }
}

}  // namespace pik
