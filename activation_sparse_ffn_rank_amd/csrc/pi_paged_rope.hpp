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
    int tok_log;                      // log2 of the tokens that a wave takes side by side
    int per_wave;                     // heads that a group of lanes takes one after another
    int q_parts, k_parts;             // waves that share out the query heads of a token group, and the kv heads
    int v_groups, v_tile;             // workgroups that transpose values, numbered first, and tokens of each
    float scale, eps;
    int64_t q_ts, q_hs, k_ts, k_hs, v_ts, v_hs, o_ts, o_hs;
    const uint16_t *q, *k, *v, *q_weight, *k_weight;
    const double *freq;
    const int *slots, *q_start, *kv_len;
    uint16_t *q_out, *k_pages, *v_pages;
};

struct KvPlace {
    bool in;             // the row belongs to a request
    int64_t pos;
};
// Where the packed rows t0, t0 + 1, .. of a wave's lane groups stand; `mine` is this lane's.  q_start is searched 64 entries
// at a time.
__device__ __forceinline__ KvPlace kv_place(const KvRopeArgs &a, int t0, int tokens, int mine, int lane) {
    KvPlace x{false, 0};
    const int step = (a.n_req + 63) / 64;
    const int s1 = lane * step < a.n_req ? a.q_start[lane * step] : INT32_MAX;
    const int e1 = lane < a.n_req ? a.q_start[lane + 1] : 0, m1 = lane < a.n_req ? a.kv_len[lane] : 0;
    for (int i = 0; i < tokens; ++i) {
        const int t = t0 + i;
        int r = __popcll(__ballot(s1 <= t)) - 1;
        if (r < 0) continue;
        int start = bcast(s1, r), end, m;
        if (step == 1) {
            end = bcast(e1, r), m = bcast(m1, r);
        } else {
            const int at = r * step + lane;
            const int s2 = lane < step && at < a.n_req ? a.q_start[at] : INT32_MAX;
            const int l = __popcll(__ballot(s2 <= t)) - 1;
            if (l < 0) continue;                         // (starts that decrease)
            start = bcast(s2, l);
            r = r * step + l;
            end = a.q_start[r + 1], m = a.kv_len[r];
        }
        if (i == mine) {
            x.in = start >= 0 && t >= start && t < end && end <= a.total_q;
            x.pos = (int64_t)m - end + t;
        }
    }
    return x;
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
    constexpr int per = HD / 8, kLdsRow = HD / 2 + 1;
    const int tid = threadIdx.x, h = blockIdx.x % a.n_kv, t0 = blockIdx.x / a.n_kv * TT, nt = min(TT, a.total_q - t0);
    const int t = tid & (TT - 1);
    const uint32_t slot = t < nt ? (uint32_t)a.slots[t0 + t] : 0xffffffffu;
    const int first = a.q_start[0], end = a.q_start[a.n_req];
#pragma unroll
    for (int i = tid; i < TT * per; i += 256) {
        const int u = i / per, ch = i - u * per;
        if (u >= nt) break;
        const uint4 x = ld16(a.v + (t0 + u) * a.v_ts + h * a.v_hs + ch * 8);
        uint32_t *const d = s_v + u * kLdsRow + ch * 4;
        d[0] = x.x, d[1] = x.y, d[2] = x.z, d[3] = x.w;
    }
    __syncthreads();
    if (slot >= (uint32_t)a.n_slots || t0 + t < first || t0 + t >= end) return;
    const int64_t pg = slot >> a.page_log, off = slot & ((1u << a.page_log) - 1);
    uint16_t *const vp = a.v_pages + (((pg * a.n_kv + h) * HD) << a.page_log) + off;
    for (int d = tid / TT; d < HD / 2; d += 256 / TT) {
        const uint32_t w = s_v[t * kLdsRow + d];
        vp[(int64_t)(2 * d) << a.page_log] = (uint16_t)w;
        vp[(int64_t)(2 * d + 1) << a.page_log] = (uint16_t)(w >> 16);
    }
}

// Workgroups below v_groups take values.  The others: a wave takes 2^tok_log tokens and, one after another, some of their query or
// key heads, whose angles it computes once.
template <class T, int HD, bool PAIRS>
__global__ __launch_bounds__(256) void k_kv_rope(KvRopeArgs a) {
    constexpr int L = HD / 16;
    extern __shared__ uint32_t s_v[];                // [v_tile][HD/2 + 1]
    if ((int)blockIdx.x < a.v_groups) {
        if (a.v_tile == 64) kv_values<HD, 64>(a, s_v);
        else kv_values<HD, 16>(a, s_v);
        return;
    }
    const int tid = threadIdx.x, lane = tid & 63;
    const int w = ((int)blockIdx.x - a.v_groups) * 4 + (tid >> 6), parts = a.q_parts + a.k_parts;
    const int tokens = 1 << a.tok_log, side = (64 / L) >> a.tok_log;        // heads side by side
    const int part = w % parts, t0 = w / parts << a.tok_log;
    if (t0 >= a.total_q) return;
    const int l = lane & (L - 1), g = lane / L, mine = g & (tokens - 1), t = min(t0 + mine, a.total_q - 1);
    const bool keys = part >= a.q_parts;
    const int heads = keys ? a.n_kv : a.n_q, n = a.per_wave * side;
    const int hp = (keys ? part - a.q_parts : part) * n, h0 = hp + (g >> a.tok_log), h1 = min(hp + n, heads);
    const int rest = l - a.rot / 16;                                        // of those not turned
    const bool turned0 = PAIRS ? 8 * l < a.rot : rest < 0, turned1 = PAIRS ? HD / 2 + 8 * l < a.rot : rest < 0;
    const int at0 = PAIRS || rest < 0 ? 8 * l : a.rot + 8 * rest;
    const int at1 = at0 + (PAIRS ? HD / 2 : rest < 0 ? a.rot / 2 : (HD - a.rot) / 2);
    const uint16_t *const src = keys ? a.k + t * a.k_ts : a.q + t * a.q_ts;
    const int64_t src_hs = keys ? a.k_hs : a.q_hs;
    // the first head's elements, frequencies and weights are on their way while the row's place is found
    uint4 r0 = ld16(src + min(h0, heads - 1) * src_hs + at0), r1 = ld16(src + min(h0, heads - 1) * src_hs + at1);
    uint32_t slot = keys ? (uint32_t)a.slots[t] : 0u;
    double freq[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) freq[i] = 0.0;
    if (turned0)
#pragma unroll
        for (int i = 0; i < 4; ++i) freq[i] = a.freq[(PAIRS ? 4 : 8) * l + i];
    if (turned1)
#pragma unroll
        for (int i = 0; i < 4; ++i) freq[4 + i] = a.freq[(PAIRS ? HD / 4 + 4 * l : 8 * l + 4) + i];
    float w0[8], w1[8];
    const uint16_t *const weight = keys ? a.k_weight : a.q_weight;
    if (a.norm && weight) {
        kv_floats<T>(ld16(weight + at0), w0);
        kv_floats<T>(ld16(weight + at1), w1);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) w0[i] = w1[i] = 1.f;
    }
    const KvPlace place = kv_place(a, t0, tokens, mine, lane);
    if (!place.in || (keys && slot >= (uint32_t)a.n_slots)) return;
    float c[8], s[8];
#pragma unroll
    for (int half = 0; half < 2; ++half)
        if (half ? turned1 : turned0) {
#pragma unroll
            for (int i = 4 * half; i < 4 * half + 4; ++i) {
                // the angle in turns, less whole ones, in 64 bits: far positions have few bits behind the point
                double x = (double)place.pos * (freq[i] * 0.15915494309189535);
                x -= rint(x);
                sincospif(2.f * (float)x, &s[i], &c[i]);
                s[i] *= a.scale, c[i] *= a.scale;
            }
        }
    const int64_t pg = slot >> a.page_log, off = slot & ((1u << a.page_log) - 1);
    uint16_t *const dst = keys ? a.k_pages + (((pg * a.n_kv) << a.page_log) + off) * HD : a.q_out + t * a.o_ts;
    const int64_t dst_hs = keys ? (int64_t)HD << a.page_log : a.o_hs;
    for (int h = h0; h < h1; h += side) {
        float x0[8], x1[8];
        kv_floats<T>(r0, x0);
        kv_floats<T>(r1, x1);
        if (h + side < h1) {                                                // the next head's
            r0 = ld16(src + (h + side) * src_hs + at0);
            r1 = ld16(src + (h + side) * src_hs + at1);
        }
        if (a.norm) {
            float sum = 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i) sum += x0[i] * x0[i] + x1[i] * x1[i];
            const float f = 1.f / sqrtf(kv_lane_sum<L>(sum) * (1.f / HD) + a.eps);
#pragma unroll
            for (int i = 0; i < 8; ++i) x0[i] *= f * w0[i], x1[i] *= f * w1[i];
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
        *reinterpret_cast<uint4 *>(dst + h * dst_hs + at0) = kv_halves<T>(x0);
        *reinterpret_cast<uint4 *>(dst + h * dst_hs + at1) = kv_halves<T>(x1);
    }
}

}  // namespace pik
