// f8_stream.hip - e4m3 products for few activation rows: out[m, n] = x_m W_n.
//
// Bound by the weight bytes, each read once, and at these sizes by latency.
// The weights go from memory straight into the registers of the wavefront
// that uses them, in the order the matrix instruction takes them, so neither
// LDS nor a barrier stands between HBM and the multiply.  A wavefront owns 16
// NR weight rows; the 128 columns that share a scale are one step, whose codes
// are widened to bf16 (exact) and multiplied on the matrix cores with fp32
// sums (f8_dev.h: why not the 8-bit instruction; its rate is not needed
// here).  A step's sum is multiplied by the activation row's power-of-two scale
// (exact) and added with the weight block's fp32 scale.  Lane l reads columns
// 16 (l / 16) .. +15 of both 64-column halves, so a load touches 64 consecutive
// bytes of 16 rows; the activation rows are read the same way (their order in
// K is free as long as both operands agree).
#include "common.h"
#include "dma_dev.h"
#include "f8_dev.h"
#include "gemm_dev.h"
#include "kernels.h"

namespace moe {
namespace {

constexpr int SW = 8;  // wavefronts per workgroup

template <bool NT>
__device__ __forceinline__ f8_u4 f8_ld(const uint8_t* p) {
    if constexpr (NT) return __builtin_nontemporal_load(reinterpret_cast<const f8_u4*>(p));
    else return *reinterpret_cast<const f8_u4*>(p);
}

// Fragments of U steps of 128 columns: NR weight row tiles, NT activation row tiles.
template <int NR, int NT, int U>
struct F8Frag {
    f8_u4 w[U][NR][2], x[U][NT][2];
    uint32_t e[U][NT];
};

// acc[r][t] += the products over the 128-column steps [kb0, kb1).  wp, xp:
// this lane's rows; ep: their scale bytes; sp: the weight rows' block scales
// (wave-uniform).  kb1 may be the step that K ends in: its columns past K
// count as zeros and are not read.
template <int NR, int NT, int U>
__device__ __forceinline__ void f8_stream(const uint8_t* const (&wp)[NR], const float* const (&sp)[NR],
                                          const uint8_t* const (&xp)[NT], const uint8_t* const (&ep)[NT], int kb0,
                                          int kb1, int K, f8_f4 (&acc)[NR][NT]) {
    using Frag = F8Frag<NR, NT, U>;
    const int lo = 16 * (lane_id() / 16), kfull = K / F8_BLK, kbe = min(kb1, kfull);
    auto load = [&](Frag& f, int kb) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int k = min(kb + u, kbe - 1);  // (steps past the end repeat the last; not used)
            const size_t o = (size_t)k * F8_BLK + lo;
#pragma unroll
            for (int r = 0; r < NR; ++r) {
                f.w[u][r][0] = f8_ld<true>(wp[r] + o);
                f.w[u][r][1] = f8_ld<true>(wp[r] + o + 64);
            }
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                f.x[u][t][0] = f8_ld<false>(xp[t] + o);
                f.x[u][t][1] = f8_ld<false>(xp[t] + o + 64);
                f.e[u][t] = ep[t][k];
            }
        }
        pin();
    };
    auto step = [&](const f8_u4 (&w)[NR][2], const f8_u4 (&x)[NT][2], const uint32_t (&e)[NT], int k) {
        F8Wide ww[NR];
        float s[NR];
#pragma unroll
        for (int r = 0; r < NR; ++r) {
            ww[r] = f8_widen(w[r][0], w[r][1]);
            s[r] = f8_uniform(sp[r], k);
        }
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            const F8Wide xw = f8_widen(x[t][0], x[t][1]);
            const float sx = f8_scale_value(e[t]);
#pragma unroll
            for (int r = 0; r < NR; ++r) {
                const f8_f4 p = f8_dot16(ww[r], xw, f8_f4{0.f, 0.f, 0.f, 0.f});
#pragma unroll
                for (int v = 0; v < 4; ++v) acc[r][t][v] = fmaf(s[r], p[v] * sx, acc[r][t][v]);
            }
        }
    };
    auto compute = [&](const Frag& f, int kb) {
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (kb + u < kbe) step(f.w[u], f.x[u], f.e[u], kb + u);
    };
    if (kb0 < kbe) {
        Frag a, b;
        load(a, kb0);
        for (int kb = kb0; kb < kbe; kb += 2 * U) {
            if (kb + U < kbe) load(b, kb + U);
            compute(a, kb);
            if (kb + U < kbe) {
                if (kb + 2 * U < kbe) load(a, kb + 2 * U);
                compute(b, kb + U);
            }
        }
    }
    if (kb0 <= kfull && kfull < kb1) {  // the step that K ends in
        const int k0 = kfull * F8_BLK + lo;
        const f8_u4 zero = f8_u4{0, 0, 0, 0};
        f8_u4 w[NR][2], x[NT][2];
        uint32_t e[NT];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const bool in = k0 + 64 * h < K;  // K is a multiple of 16
#pragma unroll
            for (int r = 0; r < NR; ++r) {
                w[r][h] = zero;
                if (in) w[r][h] = f8_ld<true>(wp[r] + k0 + 64 * h);
            }
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                x[t][h] = zero;
                if (in) x[t][h] = f8_ld<false>(xp[t] + k0 + 64 * h);
            }
        }
#pragma unroll
        for (int t = 0; t < NT; ++t) e[t] = ep[t][kfull];
        step(w, x, e, kfull);
    }
}

// ---------------------------------------------------------------------------
// dense: 16 RB output columns per workgroup, K split over KS = SW / RB
// wavefronts whose partial sums are added in LDS in a fixed order.
// ---------------------------------------------------------------------------
template <int NT, int RB, int OF>
__global__ __launch_bounds__(64 * SW) void f8_dense_stream_kernel(BlockArgs a) {
    constexpr int KS = SW / RB;
    __shared__ f8_f4 part[KS > 1 ? KS - 1 : 1][RB][NT][WAVE];
    const int lane = lane_id(), wave = wave_index(), rb = wave % RB, ks = wave / RB;
    const int c0 = (blockIdx.x * RB + rb) * 16, m0 = blockIdx.y * 16 * NT, KB = f8_blocks(a.k);
    const bool live = c0 < a.n;
    f8_f4 acc[1][NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) acc[0][t] = f8_f4{0.f, 0.f, 0.f, 0.f};
    if (live) {
        const uint8_t* wp[1] = {a.wq + (size_t)min(c0 + lane % 16, a.n - 1) * a.k};
        const float* sp[1] = {a.ws + (size_t)(c0 / F8_BLK) * KB};
        const uint8_t *xp[NT], *ep[NT];
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            const size_t r = (size_t)min(m0 + 16 * t + lane % 16, a.m - 1);
            xp[t] = a.xq + r * a.k;
            ep[t] = a.xe + r * f8_scale_ld(a.k);
        }
        const int per = (KB + KS - 1) / KS;
        f8_stream<1, NT, NT <= 2 ? 4 : 2>(wp, sp, xp, ep, ks * per, min(KB, (ks + 1) * per), a.k, acc);
    }
    if constexpr (KS > 1) {
        if (ks > 0)
#pragma unroll
            for (int t = 0; t < NT; ++t) part[ks - 1][rb][t][lane] = acc[0][t];
        __syncthreads();
        if (ks > 0) return;
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int s = 0; s < KS - 1; ++s) acc[0][t] += part[s][rb][t][lane];
    }
    const int c = c0 + 4 * (lane / 16);
    if (c >= a.n) return;
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        const int r = m0 + 16 * t + lane % 16;
        if (r >= a.m) continue;
        const float v[4] = {acc[0][t][0], acc[0][t][1], acc[0][t][2], acc[0][t][3]};
        f8_store4<OF>(a.out, (size_t)r * a.n + c, a.n - c, v, a.n % 4 == 0);
    }
}

template <int NT, int RB>
hipError_t dense_launch(const BlockArgs& a, hipStream_t st) {
    const dim3 grid((a.n + 16 * RB - 1) / (16 * RB), (a.m + 16 * NT - 1) / (16 * NT));
    if (a.odt == MOE_DT_BF16) f8_dense_stream_kernel<NT, RB, MOE_DT_BF16><<<grid, 64 * SW, 0, st>>>(a);
    else f8_dense_stream_kernel<NT, RB, MOE_DT_F32><<<grid, 64 * SW, 0, st>>>(a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_block_matmul(const BlockArgs& a, hipStream_t st) {
    if (a.m > 128) return launch_block_matmul_tile(a, st);
    if (a.m <= 16) return dense_launch<1, 1>(a, st);
    if (a.m <= 32) return dense_launch<2, 2>(a, st);
    return dense_launch<4, 4>(a, st);
}

}  // namespace moe
