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
// side: the wavefront lays its keys out in LDS and as many lanes as there are
// for each group scan it together.
//
// Bound by instruction issue: a wavefront per token, 64 of them in turn on each
// SIMD for 65536 tokens (256 experts, 8 groups, top-8: 96 us with the library
// exponential and division and one lane scanning each group, 80 us here, about
// 600 vector instructions a token; a bitwise search for the k-th key over
// ballots in place of the k rounds took as many).  group_select.hip puts four
// tokens into a wavefront where there are that many (54 us).
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

// e^x for |x| up to 708 (further out: as at 708) to about one unit in the last
// place: x = n ln2 + r, the Taylor series of e^r to r^12 (|r| <= ln2 / 2: the next
// term is below 2^-52), scaled by 2^n.  NaN is the caller's.
__device__ __forceinline__ double exp_f64(double x) {
    x = fmin(fmax(x, -708.0), 708.0);
    const double n = rint(x * 1.4426950408889634);
    double r = __fma_rn(-n, 0x1.62e42fefa39efp-1, x);  // ln2 in two parts; the fused product is exact
    r = __fma_rn(-n, 0x1.abc9e3b39803fp-56, r);
    double p = 1.0 / 479001600.0;
    p = __fma_rn(p, r, 1.0 / 39916800.0);
    p = __fma_rn(p, r, 1.0 / 3628800.0);
    p = __fma_rn(p, r, 1.0 / 362880.0);
    p = __fma_rn(p, r, 1.0 / 40320.0);
    p = __fma_rn(p, r, 1.0 / 5040.0);
    p = __fma_rn(p, r, 1.0 / 720.0);
    p = __fma_rn(p, r, 1.0 / 120.0);
    p = __fma_rn(p, r, 1.0 / 24.0);
    p = __fma_rn(p, r, 1.0 / 6.0);
    p = __fma_rn(p, r, 0.5);
    p = __fma_rn(p, r, 1.0);
    p = __fma_rn(p, r, 1.0);
    return ldexp(p, (int)n);
}
// 1 / d for finite normal d: the hardware's estimate and two Newton steps.
__device__ __forceinline__ double rcp_f64(double d) {
    double r = __builtin_amdgcn_rcp(d);
    r = __fma_rn(__fma_rn(-d, r, 1.0), r, r);
    return __fma_rn(__fma_rn(-d, r, 1.0), r, r);
}

// Logits sc[j] to scores; in(j): sc[j] is a real expert's (others hold -inf).
// rmax, rsum: maximum of an orderable word and fp64 sum over the lanes that
// share the token.
template <int N, class In, class Max, class Sum>
__device__ __forceinline__ void group_scores(float (&sc)[N], int score_kind, In in, Max rmax, Sum rsum) {
    if (score_kind == MOE_SCORE_SOFTMAX) {
        float m = -INFINITY;
#pragma unroll
        for (int j = 0; j < N; ++j) m = fmaxf(m, sc[j]);
        // (DPP shifts read 0 from outside a row; the maximum of the non-negative
        // and the negative part is taken on orderable integers instead)
        const uint32_t mu = __float_as_uint(m);
        const uint32_t om = rmax((mu & 0x80000000u) ? ~mu : (mu | 0x80000000u));
        m = unpack_ord(om);
        double ex[N], sum = 0.0;
#pragma unroll
        for (int j = 0; j < N; ++j) {
            const double x = (double)sc[j] - (double)m;  // NaN for a NaN logit, and for all if m is infinite
            ex[j] = in(j) ? (x != x ? x : exp_f64(x)) : 0.0;
            sum += ex[j];
        }
        sum = rsum(sum);
        const double inv = sum != sum ? sum : rcp_f64(sum);  // sum >= 1
#pragma unroll
        for (int j = 0; j < N; ++j) sc[j] = (float)(ex[j] * inv);
    } else if (score_kind == MOE_SCORE_SIGMOID) {
#pragma unroll
        for (int j = 0; j < N; ++j) {
            const float s = (float)rcp_f64(1.0 + exp_f64(-(double)sc[j]));
            sc[j] = sc[j] != sc[j] ? sc[j] : s;
        }
    } else {
#pragma unroll
        for (int j = 0; j < N; ++j) sc[j] = router_score(score_kind, sc[j]);
    }
}

// Orderable score of a group from its two best keys, then the lower group.
__device__ __forceinline__ uint64_t group_key(uint32_t b0, uint32_t b1, bool two, int grp) {
    const float best = unpack_ord(b0);
    return pack_key(two ? best + unpack_ord(b1) : best, grp);
}
__device__ __forceinline__ void merge_best2(uint32_t& b0, uint32_t& b1, uint32_t c0, uint32_t c1) {
    b1 = max(min(b0, c0), max(b1, c1));
    b0 = max(b0, c0);
}
// Weight of a selected score (S: the sum of the selected ones).
__device__ __forceinline__ float group_weight(float s, double S, float route_scale, int normalise) {
    const double num = (double)s * (double)route_scale;
    return !normalise ? (float)num : S > 0.0 ? (float)(((double)s / S) * (double)route_scale) : 0.0f;
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
    group_scores<KPL>(sc, score_kind, [&](int j) { return lane + WAVE * j < E; },
                      [](uint32_t v) { return wave_max_u32(v); }, [](double v) { return wave_sum_f64(v); });
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
        // lpg lanes (a power of two) scan each group: lane g lpg + i its keys i, i + lpg, ...
        int lpg = 1;
        while (2 * lpg * g.n_group <= WAVE) lpg *= 2;
        const int grp_l = lane / lpg;
        uint32_t b0 = 0, b1 = 0;
        if (grp_l < g.n_group) {
            const uint32_t* kg = keys + grp_l * S;
            for (int i = lane % lpg; i < S; i += lpg) {
                const uint32_t v = kg[i];
                b1 = max(b1, min(b0, v));
                b0 = max(b0, v);
            }
        }
        for (int o = 1; o < lpg; o *= 2) {
            const uint32_t c0 = (uint32_t)__shfl_xor((int)b0, o), c1 = (uint32_t)__shfl_xor((int)b1, o);
            merge_best2(b0, b1, c0, c1);
        }
        const uint64_t mine = grp_l < g.n_group ? group_key(b0, b1, g.group_top == 2 && S > 1, grp_l) : 0ull;
        int rank = 0;
        for (int q = 0; q < g.n_group; ++q) {
            const uint64_t o = ((uint64_t)(uint32_t)__builtin_amdgcn_readlane((uint32_t)(mine >> 32), q * lpg) << 32) |
                               (uint32_t)__builtin_amdgcn_readlane((uint32_t)mine, q * lpg);
            rank += o > mine;
        }
        const uint64_t keep = __ballot(grp_l < g.n_group && rank < g.topk_group);
#pragma unroll
        for (int j = 0; j < KPL; ++j) {
            const int e = lane + WAVE * j;
            const int grp = (int)(((float)e + 0.5f) * g.inv_size);  // e / S (exact: E <= 1024)
            if (e < E && !((keep >> (grp * lpg)) & 1)) key[j] = 0ull;
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
    const float w = group_weight(my_s, S, route_scale, g.normalise);
    if (lane < k) {
        idx_out[lane] = my_idx;
        w_out[lane] = w;
    }
    if (w_lane) *w_lane = w;
    return my_idx;
}

}  // namespace moe
