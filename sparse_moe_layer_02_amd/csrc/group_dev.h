// group_dev.h - selection with expert groups for one token by one wavefront.
//
//   score  s_e = softmax(l)_e, sigmoid(l_e) or sqrt(softplus(l_e)), in fp64,
//          rounded once to fp32; key_e = fp32(s_e + b_e)
//   group  score = the sum (fp32) of the group's group_top best keys; the
//          topk_group best groups stay (equal scores: lower group first, NaN
//          last, as for experts)
//   select top-k keys among the experts of those groups (rank order)
//   weight scale * s_j / sum_sel s (0 if the sum is 0), or scale * s_j
//
// Lane l holds experts l, l + 64, ... as route_dev.h's selection does, and
// the k rounds are the same.  The group scores need a group's keys side by
// side: the wavefront lays its keys out in LDS and lane g scans group g.
#pragma once
#include "common.h"
#include "kernels.h"
#include "route_dev.h"

#pragma clang fp contract(off)

namespace moe {

// The fp32 value of pack_key's upper half (NaN for 0).
__device__ __forceinline__ float unpack_ord(uint32_t ord) {
    if (ord == 0u) return __uint_as_float(0x7FC00000u);
    return __uint_as_float((ord & 0x80000000u) ? ord & 0x7FFFFFFFu : ~ord);
}

// keys: E words of LDS of this wavefront's own.  Returns the expert of rank
// `lane` in lanes 0..k-1, its weight in *w_lane.
template <int KPL>
__device__ __forceinline__ int group_topk_token(const float* __restrict__ lrow, const float* __restrict__ bias, int E,
                                                int k, int score_kind, float route_scale, const GroupArgs& g,
                                                uint32_t* keys, int32_t* __restrict__ idx_out,
                                                float* __restrict__ w_out, float* w_lane = nullptr) {
    const int lane = lane_id();
    float sc[KPL];
    uint64_t key[KPL];
#pragma unroll
    for (int j = 0; j < KPL; ++j) sc[j] = lane + WAVE * j < E ? lrow[lane + WAVE * j] : -INFINITY;
    if (score_kind == MOE_SCORE_SOFTMAX) {
        float m = -INFINITY;
#pragma unroll
        for (int j = 0; j < KPL; ++j) m = fmaxf(m, sc[j]);
        // (DPP shifts read 0 from outside a row; the maximum of the non-negative
        // and the negative part is taken on orderable integers instead)
        const uint32_t mu = __float_as_uint(m);
        const uint32_t om = wave_max_u32((mu & 0x80000000u) ? ~mu : (mu | 0x80000000u));
        m = unpack_ord(om);
        double ex[KPL], sum = 0.0;
#pragma unroll
        for (int j = 0; j < KPL; ++j) {
            ex[j] = lane + WAVE * j < E ? exp((double)sc[j] - (double)m) : 0.0;
            sum += ex[j];
        }
        sum = wave_sum_f64(sum);
#pragma unroll
        for (int j = 0; j < KPL; ++j) sc[j] = (float)(ex[j] / sum);
    } else {
#pragma unroll
        for (int j = 0; j < KPL; ++j) sc[j] = router_score(score_kind, sc[j]);
    }
#pragma unroll
    for (int j = 0; j < KPL; ++j) {
        const int e = lane + WAVE * j;
        key[j] = e < E ? pack_key(bias ? sc[j] + bias[e] : sc[j], e) : 0ull;
    }
    if (g.n_group > 1 && g.topk_group < g.n_group) {
        const int S = E / g.n_group;
#pragma unroll
        for (int j = 0; j < KPL; ++j)
            if (lane + WAVE * j < E) keys[lane + WAVE * j] = (uint32_t)(key[j] >> 32);
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");  // the wavefront's own writes before its reads
        __builtin_amdgcn_wave_barrier();
        uint64_t mine = 0;  // group `lane`: orderable score, then the lower index
        if (lane < g.n_group) {
            uint32_t b0 = 0, b1 = 0;
            int s = lane % S;  // staggered starts: the lanes' reads spread over the banks
            for (int i = 0; i < S; ++i) {
                const uint32_t v = keys[lane * S + s];
                b1 = max(b1, min(b0, v));
                b0 = max(b0, v);
                s = s + 1 == S ? 0 : s + 1;
            }
            const float best = unpack_ord(b0);
            mine = pack_key(g.group_top == 2 && S > 1 ? best + unpack_ord(b1) : best, lane);
        }
        int rank = 0;
        for (int q = 0; q < g.n_group; ++q) {
            const uint64_t o = ((uint64_t)(uint32_t)__builtin_amdgcn_readlane((uint32_t)(mine >> 32), q) << 32) |
                               (uint32_t)__builtin_amdgcn_readlane((uint32_t)mine, q);
            rank += o > mine;
        }
        const uint64_t keep = __ballot(lane < g.n_group && rank < g.topk_group);
#pragma unroll
        for (int j = 0; j < KPL; ++j) {
            const int e = lane + WAVE * j;
            const int grp = (int)(((float)e + 0.5f) * g.inv_size);  // e / S (exact: E <= 1024)
            if (e < E && !((keep >> grp) & 1)) key[j] = 0ull;
        }
    }
    // descending within the lane, then k rounds of wave maxima (route_dev.h)
#pragma unroll
    for (int i = 1; i < KPL; ++i) {
#pragma unroll
        for (int j = i; j > 0; --j) {
            const bool sw = key[j] > key[j - 1];
            const uint64_t ka = key[j - 1], kb = key[j];
            const float sa = sc[j - 1], sb = sc[j];
            key[j - 1] = sw ? kb : ka;
            key[j] = sw ? ka : kb;
            sc[j - 1] = sw ? sb : sa;
            sc[j] = sw ? sa : sb;
        }
    }
    int my_idx = 0;
    float my_s = 0.0f;
    double S = 0.0;
    for (int r = 0; r < k; ++r) {
        const uint32_t hi = (uint32_t)(key[0] >> 32), lo = (uint32_t)key[0];
        // a NaN key's upper half is 0, as a dropped expert's whole key is: the
        // index half decides between them too, and is never 0 for a real key
        const uint32_t M = wave_max_u32(hi);
        const uint64_t cand = __ballot(hi == M);
        int win;
        if (__popcll(cand) == 1) {
            win = __ffsll((unsigned long long)cand) - 1;
        } else {
            const uint32_t L = wave_max_u32(hi == M ? lo : 0u);
            win = __ffsll((unsigned long long)__ballot(hi == M && lo == L)) - 1;
        }
        const int e = (int)(0xFFFFFFFFu - (uint32_t)__builtin_amdgcn_readlane(lo, win));
        const float s_sel = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(sc[0]), win));
        if (lane == win) {
#pragma unroll
            for (int j = 0; j + 1 < KPL; ++j) {
                key[j] = key[j + 1];
                sc[j] = sc[j + 1];
            }
            key[KPL - 1] = 0ull;
            sc[KPL - 1] = 0.0f;
        }
        S += (double)s_sel;
        if (lane == r) {
            my_idx = e;
            my_s = s_sel;
        }
    }
    const double num = (double)my_s * (double)route_scale;
    const float w = !g.normalise ? (float)num : S > 0.0 ? (float)(((double)my_s / S) * (double)route_scale) : 0.0f;
    if (lane < k) {
        idx_out[lane] = my_idx;
        w_out[lane] = w;
    }
    if (w_lane) *w_lane = w;
    return my_idx;
}

}  // namespace moe
