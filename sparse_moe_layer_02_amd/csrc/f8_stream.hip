// f8_stream.hip - e4m3 products for few activation rows (or few results):
// out[m, n] = x_m W_n.
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

// A lane's 32 columns of one activation row: 16 from each 64-column half, as
// codes, or as bf16 or fp32 values that are quantised here (few rows: the
// launch that would do it first costs more than every workgroup doing it).
template <int XF>
struct F8Act {
    static constexpr int N = XF == MOE_DT_F8B128 ? 1 : XF == MOE_DT_BF16 ? 2 : 4;  // 16-byte pieces per half
    static constexpr int SIZE = XF == MOE_DT_F8B128 ? 1 : XF == MOE_DT_BF16 ? 2 : 4;
    f8_u4 v[2][N];
    uint32_t e;  // scale byte (codes)

    __device__ __forceinline__ void load(const uint8_t* row, const uint8_t* scales, int kb, int lo, int K) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int c = kb * F8_BLK + 64 * h + lo;
#pragma unroll
            for (int q = 0; q < N; ++q) {
                v[h][q] = f8_u4{0, 0, 0, 0};
                if (c < K) v[h][q] = f8_ld<false>(row + (size_t)c * SIZE + 16 * q);  // K is a multiple of 16
            }
        }
        if constexpr (XF == MOE_DT_F8B128) e = scales[kb];
    }
    // codes of both halves; their scale in s
    __device__ __forceinline__ F8Wide widen(float& s) const {
        if constexpr (XF == MOE_DT_F8B128) {
            s = f8_scale_value(e);
            return f8_widen(v[0][0], v[1][0]);
        } else {
            float x[2][16];
            uint32_t m = 0;
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    if constexpr (XF == MOE_DT_BF16) {
                        const uint32_t p = v[h][j / 8][j / 2 % 4];
                        x[h][j] = j % 2 ? bf16_hi(p) : bf16_lo(p);
                    } else {
                        x[h][j] = __uint_as_float(v[h][j / 4][j % 4]);
                    }
                    m = max(m, f8_abs_bits(x[h][j]));
                }
            // the block's other columns are in the lanes 16, 32 and 48 away
            m = max(m, (uint32_t)__shfl_xor((int)m, 16));
            m = max(m, (uint32_t)__shfl_xor((int)m, 32));
            const uint32_t byte = f8_scale_byte(m);
            const float inv = f8_inv_scale(byte);
            f8_u4 c[2];
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    c[h][q] = f8_pack4(x[h][4 * q], x[h][4 * q + 1], x[h][4 * q + 2], x[h][4 * q + 3], inv, byte);
            s = f8_scale_value(byte);
            return f8_widen(c[0], c[1]);
        }
    }
};

// Fragments of U steps of 128 columns: NR weight row tiles, NT activation row tiles.
template <int NR, int NT, int U, int XF>
struct F8Frag {
    f8_u4 w[U][NR][2];
    F8Act<XF> x[U][NT];
};

// acc[r][t] += the products over the 128-column steps [kb0, kb1).  wp, xp:
// this lane's rows; ep: their scale bytes; sp: the weight rows' block scales
// (wave-uniform).  kb1 may be the step that K ends in: its columns past K
// count as zeros and are not read.
template <int NR, int NT, int U, int XF>
__device__ __forceinline__ void f8_stream(const uint8_t* const (&wp)[NR], const float* const (&sp)[NR],
                                          const uint8_t* const (&xp)[NT], const uint8_t* const (&ep)[NT], int kb0,
                                          int kb1, int K, f8_f4 (&acc)[NR][NT]) {
    using Frag = F8Frag<NR, NT, U, XF>;
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
            for (int t = 0; t < NT; ++t) f.x[u][t].load(xp[t], ep[t], k, lo, 1 << 30);
        }
        pin();
    };
    auto step = [&](const f8_u4 (&w)[NR][2], const F8Act<XF> (&x)[NT], int k) {
        F8Wide ww[NR];
        float s[NR];
#pragma unroll
        for (int r = 0; r < NR; ++r) {
            ww[r] = f8_widen(w[r][0], w[r][1]);
            s[r] = f8_uniform(sp[r], k);
        }
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            float sx;
            const F8Wide xw = x[t].widen(sx);
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
            if (kb + u < kbe) step(f.w[u], f.x[u], kb + u);
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
        f8_u4 w[NR][2];
        F8Act<XF> x[NT];
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int r = 0; r < NR; ++r) {
                w[r][h] = f8_u4{0, 0, 0, 0};
                if (k0 + 64 * h < K) w[r][h] = f8_ld<true>(wp[r] + k0 + 64 * h);
            }
#pragma unroll
        for (int t = 0; t < NT; ++t) x[t].load(xp[t], ep[t], kfull, lo, K);
        step(w, x, kfull);
    }
}

// 16 NR output columns per workgroup, K split over its SW wavefronts, whose
// partial sums are added in LDS in a fixed order.
template <int NT, int NR, int OF, int XF>
__global__ __launch_bounds__(64 * SW) void f8_dense_stream_kernel(BlockArgs a) {
    __shared__ f8_f4 part[SW][NR][NT][WAVE];
    const int lane = lane_id(), wave = wave_index();
    const int c0 = blockIdx.x * 16 * NR, m0 = blockIdx.y * 16 * NT, KB = f8_blocks(a.k);
    f8_f4 acc[NR][NT];
    const uint8_t* wp[NR];
    const float* sp[NR];
    const uint8_t *xp[NT], *ep[NT];
#pragma unroll
    for (int r = 0; r < NR; ++r) {
        wp[r] = a.wq + (size_t)min(c0 + 16 * r + lane % 16, a.n - 1) * a.k;
        sp[r] = a.ws + (size_t)(min(c0 + 16 * r, a.n - 1) / F8_BLK) * KB;
#pragma unroll
        for (int t = 0; t < NT; ++t) acc[r][t] = f8_f4{0.f, 0.f, 0.f, 0.f};
    }
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        const size_t r = (size_t)min(m0 + 16 * t + lane % 16, a.m - 1);
        xp[t] = a.xq + r * a.k * F8Act<XF>::SIZE;
        ep[t] = XF == MOE_DT_F8B128 ? a.xe + r * f8_scale_ld(a.k) : nullptr;
    }
    const int per = (KB + SW - 1) / SW;
    constexpr int U = XF == MOE_DT_F8B128 ? 4 / NR : XF == MOE_DT_BF16 ? 2 : 1;  // steps in flight: what the registers hold
    f8_stream<NR, NT, U, XF>(wp, sp, xp, ep, wave * per, min(KB, (wave + 1) * per), a.k, acc);
#pragma unroll
    for (int r = 0; r < NR; ++r)
#pragma unroll
        for (int t = 0; t < NT; ++t) part[wave][r][t][lane] = acc[r][t];
    __syncthreads();
    // wavefront w adds the partial sums of the (r, t) tiles w, w + SW, ...
    for (int q = wave; q < NR * NT; q += SW) {
        const int r = q / NT, t = q % NT;
        f8_f4 s = part[0][r][t][lane];
#pragma unroll
        for (int w = 1; w < SW; ++w) s += part[w][r][t][lane];
        const int c = c0 + 16 * r + 4 * (lane / 16), row = m0 + 16 * t + lane % 16;
        if (c >= a.n || row >= a.m) continue;
        const float v[4] = {s[0], s[1], s[2], s[3]};
        f8_store4<OF>(a.out, (size_t)row * a.n + c, a.n - c, v, a.n % 4 == 0);
    }
}

template <int NT, int NR, int XF>
hipError_t dense_launch(const BlockArgs& a, hipStream_t st) {
    const dim3 grid((a.n + 16 * NR - 1) / (16 * NR), (a.m + 16 * NT - 1) / (16 * NT));
    if (a.odt == MOE_DT_BF16) f8_dense_stream_kernel<NT, NR, MOE_DT_BF16, XF><<<grid, 64 * SW, 0, st>>>(a);
    else f8_dense_stream_kernel<NT, NR, MOE_DT_F32, XF><<<grid, 64 * SW, 0, st>>>(a);
    return hipGetLastError();
}

}  // namespace

// Rows that are quantised by the product itself: every workgroup of 16 output
// columns does it again, so few rows and few workgroups (us against a launch of
// its own first, bf16 rows: n x k 6144 x 2048: 1 row 7.7 / 10.5, 16 rows 10.2 /
// 13.8; 4096 x 6144: 9.8 / 9.8, 14.3 / 14.3; 24576 x 6144: 57 / 52, 78 / 70; fp32
// rows, twice the bytes, 4096 x 6144: 1 row 9.6 / 9.7, 8 rows 13.9 / 12.4).
bool block_matmul_takes(int xdt, int m, int n) {
    return n <= 8192 && m <= (xdt == MOE_DT_BF16 ? 16 : 4);
}

// Up to 48 rows here, more in LDS tiles (us at n x k 4096 x 6144: 1 row 9.1
// against 20.3 for the smallest tiles, 24 rows 16.7 / 20.3, 128 rows 33.9 / 23.1;
// 48 rows of 4096 x 4096 13.1 / 16.2, 77 rows of 6144 x 2048 16.9 / 9.9), unless
// the sum over k is long and there are so few results that all workgroups here
// run at once, its eight wavefronts sharing the sum: 256 rows of 512 x 2048 7.8 /
// 8.7 (fp32 results 7.6 / 10.8), 77 of 1024 x 6144 17.6 / 18.5 (17.2 / 25.5), but
// 512 of 1024 x 2048 13.6 / 8.9 and, at 512 columns, 128 of 1024 5.4 / 5.1.
hipError_t launch_block_matmul(const BlockArgs& a, hipStream_t st) {
    if (a.xdt == MOE_DT_BF16) return dense_launch<1, 1, MOE_DT_BF16>(a, st);
    if (a.xdt == MOE_DT_F32) return dense_launch<1, 1, MOE_DT_F32>(a, st);
    if (a.m <= 16) return dense_launch<1, 1, MOE_DT_F8B128>(a, st);
    const bool few = (long)((a.m + 31) / 32) * ((a.n + 31) / 32) <= 256 && a.k >= 1024;
    if (a.m <= 48 || few) return dense_launch<2, 2, MOE_DT_F8B128>(a, st);
    return launch_block_matmul_tile(a, st);
}

}  // namespace moe
