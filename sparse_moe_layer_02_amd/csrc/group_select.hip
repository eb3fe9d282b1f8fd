// group_select.hip - top-k selection with expert groups and softmax scores
// (group_dev.h): one wavefront per token, or for many tokens four per wavefront.
#include "common.h"
#include "group_dev.h"
#include "f8_dev.h"
#include "kernels.h"

#pragma clang fp contract(off)

namespace moe {

template <int KPL>
__global__ __launch_bounds__(256) void group_topk_kernel(SelectArgs a, GroupArgs g) {
    __shared__ uint32_t keys[4][KPL * WAVE];
    const int wave = wave_index(), t = blockIdx.x * 4 + wave;
    if (t >= a.T) return;
    group_topk_token<KPL>(a.logits + (size_t)t * a.E, a.bias, a.E, a.k, a.score, a.route_scale, g, keys[wave],
                          a.topk_idx + (size_t)t * a.k, a.topk_w + (size_t)t * a.k);
}

// Four tokens per wavefront, 16 lanes each; lane l of a row holds experts l C ..
// l C + C - 1, so that a group is whole lanes, the maxima stay in a DPP row and
// lower lane and lower register are the lower index.  Keys are the orderable
// words alone (a real expert's at least 1; 0: dropped, or selected already).
//
// Bound by instruction issue as group_topk_kernel is, with the rounds' and the
// groups' instructions shared by four tokens.
template <int C>
__global__ __launch_bounds__(256) void group_topk_rows_kernel(SelectArgs a, GroupArgs g) {
    constexpr int E = 16 * C;
    typedef float lf4 __attribute__((ext_vector_type(4), aligned(4)));  // (logits and bias: 4-byte aligned)
    __shared__ __attribute__((aligned(16))) float s_sc[4][4][E];
    __shared__ int s_idx[4][4][16];
    const int wave = wave_index(), lane = lane_id(), row = lane / 16, l = lane % 16;
    const int t0 = (blockIdx.x * 4 + wave) * 4, t = t0 + row;
    if (t0 >= a.T) return;
    const float* lr = a.logits + (size_t)min(t, a.T - 1) * E + l * C;
    float sc[C];
#pragma unroll
    for (int q = 0; q < C / 4; ++q) {
        const lf4 v = reinterpret_cast<const lf4*>(lr)[q];
        sc[4 * q] = v.x; sc[4 * q + 1] = v.y; sc[4 * q + 2] = v.z; sc[4 * q + 3] = v.w;
    }
    group_scores<C>(sc, a.score, [](int) { return true; }, [](uint32_t v) { return row16_max_u32(v); }, [](double v) {
        v += dpp_f64<0x128>(v);  // row rotations: every lane of the row has the sum
        v += dpp_f64<0x124>(v);
        v += dpp_f64<0x122>(v);
        return v + dpp_f64<0x121>(v);
    });
    uint32_t key[C];
#pragma unroll
    for (int j = 0; j < C; ++j) key[j] = (uint32_t)(pack_key(a.bias ? sc[j] + a.bias[l * C + j] : sc[j], 0) >> 32);
    float* ts = s_sc[wave][row];
    int* ti = s_idx[wave][row];
#pragma unroll
    for (int q = 0; q < C / 4; ++q)
        *reinterpret_cast<float4*>(ts + l * C + 4 * q) = make_float4(sc[4 * q], sc[4 * q + 1], sc[4 * q + 2], sc[4 * q + 3]);
    bool keep = true;
    if (g.topk_group < g.n_group) {
        const int lg = 16 / g.n_group, grp = l / lg;  // lanes of a group
        uint32_t b0 = 0, b1 = 0;
#pragma unroll
        for (int j = 0; j < C; ++j) {
            b1 = max(b1, min(b0, key[j]));
            b0 = max(b0, key[j]);
        }
        for (int o = 1; o < lg; o *= 2) {
            const uint32_t c0 = (uint32_t)__shfl_xor((int)b0, o), c1 = (uint32_t)__shfl_xor((int)b1, o);
            merge_best2(b0, b1, c0, c1);
        }
        const uint64_t mine = group_key(b0, b1, g.group_top == 2, grp);
        int rank = 0;
        for (int q = 0; q < g.n_group; ++q) {
            const int from = 16 * row + q * lg;
            const uint64_t o = ((uint64_t)(uint32_t)__shfl((int)(mine >> 32), from) << 32) | (uint32_t)__shfl((int)mine, from);
            rank += o > mine;
        }
        keep = rank < g.topk_group;
    }
#pragma unroll
    for (int j = 0; j < C; ++j) key[j] = keep ? max(key[j], 1u) : 0u;
    for (int r = 0; r < a.k; ++r) {
        uint32_t m = key[0];
#pragma unroll
        for (int j = 1; j < C; ++j) m = max(m, key[j]);
        const uint32_t M = row16_max_u32(m);
        const uint32_t tops = (uint32_t)(__ballot(m == M) >> (16 * row)) & 0xFFFFu;
        bool done = l != __ffs((int)tops) - 1;
        const bool mine = !done;
        int sel = 0;
#pragma unroll
        for (int j = 0; j < C; ++j) {
            const bool hit = !done && key[j] == M;
            sel = hit ? j : sel;
            key[j] = hit ? 0u : key[j];
            done = done || hit;
        }
        if (mine) ti[r] = l * C + sel;
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");  // the wavefront's own writes before its reads
    __builtin_amdgcn_wave_barrier();
    double S = 0.0;
    for (int r = 0; r < a.k; ++r) S += (double)ts[ti[r]];
    if (l < a.k && t < a.T) {
        const int e = ti[l];
        a.topk_idx[(size_t)t * a.k + l] = e;
        a.topk_w[(size_t)t * a.k + l] = group_weight(ts[e], S, a.route_scale, g.normalise);
    }
}

// Four tokens per wavefront: whole lanes per group, a rank per lane, and enough
// tokens to fill the device with a quarter of the wavefronts (us, one / four
// tokens per wavefront, top-8 of 8 groups: 256 experts, sigmoid: 4096 tokens 8.7
// / 9.2, 16384 23.2 / 16.5, 65536 79.7 / 53.7; 128 experts, softmax: 7.2 / 6.9,
// 18.4 / 11.0, 58.8 / 28.5).
static bool rows_fit(const SelectArgs& a, const GroupArgs& g) {
    const bool groups = g.topk_group == g.n_group || 16 % g.n_group == 0;
    return a.T >= 8192 && a.E % 64 == 0 && a.E <= 256 && a.k <= 16 && groups;
}

hipError_t launch_group_topk(const SelectArgs& a, const GroupArgs& g, hipStream_t st, const KTime& kt) {
    if (rows_fit(a, g)) {
        const dim3 grid((a.T + 15) / 16);
        if (a.E == 64) launch_kernel(group_topk_rows_kernel<4>, grid, 256, st, kt, a, g);
        else if (a.E == 128) launch_kernel(group_topk_rows_kernel<8>, grid, 256, st, kt, a, g);
        else if (a.E == 192) launch_kernel(group_topk_rows_kernel<12>, grid, 256, st, kt, a, g);
        else launch_kernel(group_topk_rows_kernel<16>, grid, 256, st, kt, a, g);
        return hipGetLastError();
    }
    const int kpl = (a.E + WAVE - 1) / WAVE;
    const dim3 grid((a.T + 3) / 4);
    if (kpl <= 1) launch_kernel(group_topk_kernel<1>, grid, 256, st, kt, a, g);
    else if (kpl <= 2) launch_kernel(group_topk_kernel<2>, grid, 256, st, kt, a, g);
    else if (kpl <= 3) launch_kernel(group_topk_kernel<3>, grid, 256, st, kt, a, g);
    else if (kpl <= 4) launch_kernel(group_topk_kernel<4>, grid, 256, st, kt, a, g);
    else if (kpl <= 8) launch_kernel(group_topk_kernel<8>, grid, 256, st, kt, a, g);
    else launch_kernel(group_topk_kernel<16>, grid, 256, st, kt, a, g);
    return hipGetLastError();
}

}  // namespace moe
