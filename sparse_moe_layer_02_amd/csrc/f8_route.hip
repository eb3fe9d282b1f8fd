// f8_route.hip - the routing of few tokens through an e4m3 or int8 layer, in two
// launches.
//
// 1. Router logits, a workgroup per expert: 1024 threads of four columns each,
// so that up to 4096 columns of the expert's row and of every token are in
// flight at once (fp64 sums in a fixed tree order, rounded once).  8 tokens x
// 192 experts x 4096: 4.9 us; route.hip's 256 threads, which go round four
// times, 17.5 us.
//
// 2. Selection, token->expert grouping and the quantisation of x.  Each is
// microseconds of latency for a single workgroup's work, and the expert
// kernels wait for all three; in launches of their own they took 15 us of a
// one-token layer's 96.  Workgroup 0 selects (a wavefront per token) and groups
// (permute_dev.h, over the indices it keeps in LDS); the others quantise the
// rows of x: 8.3 us (10.1 with a scan each for offsets, experts and tiles).
#include "common.h"
#include "group_dev.h"
#include "kernels.h"
#include "permute_dev.h"
#include "i8_quantize_dev.h"
#include "quantize_dev.h"
#include "route_dev.h"

#pragma clang fp contract(off)

namespace moe {

constexpr int FR_WAVES = F8_ROUTE_MAX_T;  // a wavefront per token
constexpr int FR_TOK = 8;                 // tokens per pass of the router

__global__ __launch_bounds__(FR_WAVES * WAVE) void f8_router_kernel(const uint16_t* __restrict__ x,
                                                                    const float* __restrict__ wr, int T, int d, int E,
                                                                    float* __restrict__ logits) {
    __shared__ double part[FR_WAVES][FR_TOK];
    const int e = blockIdx.x, t0 = blockIdx.y * FR_TOK, nt = min(FR_TOK, T - t0), tid = threadIdx.x;
    const float* w = wr + (size_t)e * d;
    double acc[FR_TOK];
#pragma unroll
    for (int t = 0; t < FR_TOK; ++t) acc[t] = 0.0;
    for (int c = 4 * tid; c < d; c += 4 * FR_WAVES * WAVE) {
        const float4 v = *reinterpret_cast<const float4*>(w + c);
        uint2 u[FR_TOK];
#pragma unroll
        for (int t = 0; t < FR_TOK; ++t)  // (tokens past the last repeat it; not stored)
            u[t] = *reinterpret_cast<const uint2*>(x + (size_t)(t0 + min(t, nt - 1)) * d + c);
#pragma unroll
        for (int t = 0; t < FR_TOK; ++t) {
            acc[t] = __fma_rn((double)bf16_lo(u[t].x), (double)v.x, acc[t]);
            acc[t] = __fma_rn((double)bf16_hi(u[t].x), (double)v.y, acc[t]);
            acc[t] = __fma_rn((double)bf16_lo(u[t].y), (double)v.z, acc[t]);
            acc[t] = __fma_rn((double)bf16_hi(u[t].y), (double)v.w, acc[t]);
        }
    }
#pragma unroll
    for (int t = 0; t < FR_TOK; ++t) {
        if (t < nt) {
            const double s = wave_sum_f64(acc[t]);
            if (lane_id() == 0) part[tid / WAVE][t] = s;
        }
    }
    __syncthreads();
    if (tid < nt) {
        double s = part[0][tid];
#pragma unroll
        for (int q = 1; q < FR_WAVES; ++q) s += part[q][tid];
        logits[(size_t)(t0 + tid) * E + e] = (float)s;
    }
}

static_assert(FR_WAVES * WAVE == 1024 && F8_ROUTE_MAX_T * 32 < 1024, "emit_lists_few: threads, assignments");

// The rows of x in the workgroups behind the first: e4m3 codes by blocks of 128
// columns, int8 codes by rows; how many workgroups.
__device__ __forceinline__ void quantize_rest(const QuantArgs& q) {
    quantize_blocks<MOE_DT_BF16>(q, (int64_t)(blockIdx.x - 1) * (FR_WAVES * 4) + threadIdx.x / 16,
                                 (int64_t)(gridDim.x - 1) * (FR_WAVES * 4));
}
__device__ __forceinline__ void quantize_rest(const TokenQuantArgs& q) {
    quantize_token_rows<MOE_DT_BF16, FR_WAVES * WAVE>(q, blockIdx.x - 1, gridDim.x - 1);
}
static int64_t rest_blocks(const QuantArgs& q) {
    return ((int64_t)q.rows * f8_scale_ld(q.cols) + FR_WAVES * 4 - 1) / (FR_WAVES * 4);
}
static int64_t rest_blocks(const TokenQuantArgs& q) { return q.rows; }

template <int KPL, class Q>
__global__ __launch_bounds__(FR_WAVES * WAVE) void f8_route_kernel(SelectArgs s, GroupArgs g, bool grouped, PermArgs p, Q q) {
    if (blockIdx.x > 0) {
        quantize_rest(q);
        return;
    }
    __shared__ uint32_t s_key[FR_WAVES][KPL * WAVE];
    __shared__ int32_t s_idx[FR_WAVES * 32];
    __shared__ int cnt[1024];
    __shared__ int smem[17];
    const int tid = threadIdx.x, lane = lane_id(), wave = wave_index(), E = s.E, n = s.T * s.k;
    if (wave < s.T) {
        const float* l = s.logits + (size_t)wave * E;
        int32_t* oi = s.topk_idx + (size_t)wave * s.k;
        float* ow = s.topk_w + (size_t)wave * s.k;
        int my;
        if (grouped) my = group_topk_token<KPL>(l, s.bias, E, s.k, s.score, s.route_scale, g, s_key[wave], oi, ow);
        else my = topk_token<KPL, 0>(l, s.bias, E, s.k, s.score, s.route_scale, oi, ow);
        if (lane < s.k) s_idx[wave * s.k + lane] = my;
    }
    cnt[tid] = 0;
    __syncthreads();
    p.topk_idx = s_idx;
    if (tid < n) atomicAdd(&cnt[s_idx[tid]], 1);
    __syncthreads();
    int off;
    emit_lists_few(p, cnt[tid], smem, &off);
    cnt[tid] = off;  // becomes the scatter cursor
    __syncthreads();
    if (tid < WAVE) scatter_range(p, 0, n, cnt);
}

hipError_t launch_f8_router(const RouteArgs& a, hipStream_t st, const KTime& kt) {
    const dim3 grid(a.E, (a.T + FR_TOK - 1) / FR_TOK);
    launch_kernel(f8_router_kernel, grid, FR_WAVES * WAVE, st, kt, static_cast<const uint16_t*>(a.x), a.wr, a.T, a.d, a.E,
                  a.logits);
    return hipGetLastError();
}

template <class Q>
static hipError_t route_launch(const SelectArgs& s, const GroupArgs& g, bool grouped, const PermArgs& p, const Q& q,
                               hipStream_t st, const KTime& kt) {
    const dim3 grid(1 + (unsigned)rest_blocks(q));
    if (s.E <= 256) launch_kernel(f8_route_kernel<4, Q>, grid, FR_WAVES * WAVE, st, kt, s, g, grouped, p, q);
    else launch_kernel(f8_route_kernel<16, Q>, grid, FR_WAVES * WAVE, st, kt, s, g, grouped, p, q);
    return hipGetLastError();
}

hipError_t launch_f8_route(const SelectArgs& s, const GroupArgs& g, bool grouped, const PermArgs& p, const QuantArgs& q,
                           hipStream_t st, const KTime& kt) {
    return route_launch(s, g, grouped, p, q, st, kt);
}
hipError_t launch_i8_route(const SelectArgs& s, const GroupArgs& g, bool grouped, const PermArgs& p, const TokenQuantArgs& q,
                           hipStream_t st, const KTime& kt) {
    return route_launch(s, g, grouped, p, q, st, kt);
}

}  // namespace moe
