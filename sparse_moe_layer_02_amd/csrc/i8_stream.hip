// i8_stream.hip - int8 products for few activation rows.
//
//   dense:    out[m, n] = x_m W_n
//   gate/up:  h[r, c] = silu(x_r Wg_c) (x_r Wu_c), fp32
//   down:     y[t] = shared row + sum_j w_j (h_j Wd^T), with the combine
//
// Bound by the weight bytes, each read once, and at these sizes by latency.
// The weights go from memory straight into the registers of the wavefront that
// uses them, in the order the matrix instruction takes them, so neither LDS nor a
// barrier stands between HBM and the multiply.  A step is 64 columns of K: lane l
// holds columns 16 (l / 16) .. + 15 of weight row l % 16 and of activation row
// l % 16, and the 16 x 16 x 64 instruction adds their products in int32.  Sums
// are exact, so K is split as the sizes suggest; the partial sums meet in LDS.
// Rows that no expert has repeat the last one; their results are not stored.
//
// Column tails: a load past the end of K re-reads the row's last 16 columns, and
// the activation operand is zero there.
#include "common.h"
#include "dma_dev.h"
#include "gemm_dev.h"
#include "i8_dev.h"
#include "kernels.h"

namespace moe {
namespace {

constexpr int SW = 8;  // wavefronts per workgroup
constexpr int SK = 64; // columns of a step
// Steps loaded at once.  A wavefront's share of K is a multiple of them: with 8 at
// once and 12 for a wavefront the loads past its end, repeats of its last step,
// cost more than they hid (1 x 4096 x 6144: 9.7 us, 7.3 so; non-temporal loads 7.9;
// two groups ahead in place of one 8.1; 24576 x 6144: 30 us, 5.0 TB/s).
constexpr int UU = 4;
constexpr int I8_FUSE_VALUES = 24 * 1024;  // values a workgroup quantises itself, at most (their codes lie in LDS)

__device__ __forceinline__ i32x4_t ld_codes(const int8_t* p) { return *reinterpret_cast<const i32x4_t*>(p); }
__device__ __forceinline__ i32x4_t dot16(i32x4_t w, i32x4_t x, i32x4_t c) {
    return __builtin_amdgcn_mfma_i32_16x16x64_i8(w, x, c, 0, 0, 0);
}

// The products of steps [s0, s1) of NR blocks of 16 weight rows and NT of 16
// activation rows.  wp: this lane's weight rows; x(t, c): columns c .. c + 15 of its
// activation row, from memory, or from LDS (LX) once between() has put them
// there.  U steps are in flight while the U before them are multiplied, the first
// before between().
template <int NR, int NT, int U, bool LX>
struct Frag {
    i32x4_t w[U][NR], x[LX ? 1 : U][NT];
};
template <int NR, int NT, int U, bool LX, class X, class Between>
__device__ __forceinline__ void stream(const int8_t* const (&wp)[NR], X x, int s0, int s1, int K,
                                       i32x4_t (&acc)[NR][NT], Between between) {
    typedef Frag<NR, NT, U, LX> F;
    const int lo = 16 * (lane_id() / 16);
    auto load = [&](F& f, int s) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int c = min(SK * min(s + u, s1 - 1) + lo, K - 16);
#pragma unroll
            for (int r = 0; r < NR; ++r) f.w[u][r] = ld_codes(wp[r] + c);
            if constexpr (!LX) {
#pragma unroll
                for (int t = 0; t < NT; ++t) f.x[u][t] = x(t, c);
            }
        }
        pin();
    };
    auto compute = [&](const F& f, int s) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (s + u >= s1) break;
            const int c = SK * (s + u) + lo;
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                i32x4_t v;
                if constexpr (LX) v = x(t, min(c, K - 16));
                else v = f.x[u][t];
                if (c >= K) v = i32x4_t{0, 0, 0, 0};
#pragma unroll
                for (int r = 0; r < NR; ++r) acc[r][t] = dot16(f.w[u][r], v, acc[r][t]);
            }
        }
    };
    F a, b;
    if (s0 < s1) load(a, s0);
    between();
    for (int s = s0; s < s1; s += 2 * U) {
        if (s + U < s1) load(b, s + U);
        compute(a, s);
        if (s + U < s1) {
            if (s + 2 * U < s1) load(a, s + 2 * U);
            compute(b, s + U);
        }
    }
}

// Rows of fp32 or bf16 as codes in LDS by the whole workgroup (few rows: every
// workgroup doing it costs less than a launch that does it first).  The
// wavefronts share a row while there are fewer than SW.  top: a word per row.
template <int XF>
__device__ __forceinline__ void rows_to_lds(const void* x, int rows, int cols, size_t ldx, int8_t* codes, int ldq,
                                            uint32_t* top, float* scales) {
    const int lane = lane_id(), wave = wave_index();
    int wpr = SW;  // wavefronts per row
    while (wpr > 1 && wpr * rows > SW) wpr >>= 1;
    const int part = wave % wpr, first = wave / wpr, step = SW / wpr;
    constexpr int KEEP = 2;  // groups of 8 columns that stay in registers
    float v[KEEP][8];
    if ((int)threadIdx.x < rows) top[threadIdx.x] = 0u;
    __syncthreads();
    for (int r = first; r < rows; r += step) {
        uint32_t m = 0;
#pragma unroll
        for (int j = 0; j < KEEP; ++j) {
            const int c = 8 * (WAVE * (part + wpr * j) + lane);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[j][i] = 0.0f;
            if (c < cols) i8_load8<XF>(x, r * ldx + c, v[j]);
            m = max(m, i8_max8(v[j]));
        }
        for (int c = 8 * (WAVE * (part + wpr * KEEP) + lane); c < cols; c += 8 * WAVE * wpr) {
            float u[8];
            i8_load8<XF>(x, r * ldx + c, u);
            m = max(m, i8_max8(u));
        }
        m = wave_max_u32(m);
        if (lane == 0) atomicMax(&top[r], m);
    }
    __syncthreads();
    for (int r = first; r < rows; r += step) {
        const float s = i8_scale(top[r]);
        const I8Scale p = i8_scale_parts(s);
        if (part == 0 && lane == 0) scales[r] = s;
        int8_t* q = codes + r * ldq;
#pragma unroll
        for (int j = 0; j < KEEP; ++j) {
            const int c = 8 * (WAVE * (part + wpr * j) + lane);
            if (c < cols) {
                if (rows > step) i8_load8<XF>(x, r * ldx + c, v[j]);  // (the registers hold the wavefront's last row)
                *reinterpret_cast<uint2*>(q + c) = i8_codes8(v[j], p);
            }
        }
        for (int c = 8 * (WAVE * (part + wpr * KEEP) + lane); c < cols; c += 8 * WAVE * wpr) {
            float u[8];
            i8_load8<XF>(x, r * ldx + c, u);
            *reinterpret_cast<uint2*>(q + c) = i8_codes8(u, p);
        }
    }
    __syncthreads();
}

// 16 NR output columns x 16 NT rows per workgroup, K split over its wavefronts.
// XF: codes, or rows that are quantised here (all of them in one workgroup's LDS).
template <int NT, int NR, int OF, int XF>
__global__ __launch_bounds__(WAVE * SW) void i8_dense_stream_kernel(ChannelArgs a) {
    constexpr bool LX = XF != MOE_DT_I8CH;
    extern __shared__ __attribute__((aligned(16))) int8_t codes[];  // [m, k], LX
    __shared__ i32x4_t part[SW][NR][NT][WAVE];
    __shared__ uint32_t top[LX ? 16 : 1];
    __shared__ float scales[LX ? 16 : 1];
    const int lane = lane_id(), wave = wave_index();
    const int c0 = blockIdx.x * 16 * NR, m0 = blockIdx.y * 16 * NT, steps = (a.k + SK - 1) / SK;
    i32x4_t acc[NR][NT];
    const int8_t* wp[NR];
    int xr[NT];
#pragma unroll
    for (int r = 0; r < NR; ++r) {
        wp[r] = a.wq + (size_t)min(c0 + 16 * r + lane % 16, a.n - 1) * a.k;
#pragma unroll
        for (int t = 0; t < NT; ++t) acc[r][t] = i32x4_t{0, 0, 0, 0};
    }
#pragma unroll
    for (int t = 0; t < NT; ++t) xr[t] = min(m0 + 16 * t + lane % 16, a.m - 1);
    const int per = (steps + SW * UU - 1) / (SW * UU) * UU, s0 = wave * per, s1 = min(steps, s0 + per);
    if constexpr (LX) {
        stream<NR, NT, UU, true>(
            wp, [&](int t, int c) { return *reinterpret_cast<const i32x4_t*>(codes + xr[t] * a.k + c); }, s0, s1, a.k, acc,
            [&] { rows_to_lds<XF>(a.x, a.m, a.k, a.k, codes, a.k, top, scales); });
    } else {
        const int8_t* xp[NT];
#pragma unroll
        for (int t = 0; t < NT; ++t) xp[t] = static_cast<const int8_t*>(a.x) + (size_t)xr[t] * a.k;
        stream<NR, NT, UU, false>(wp, [&](int t, int c) { return ld_codes(xp[t] + c); }, s0, s1, a.k, acc, [] {});
    }
#pragma unroll
    for (int r = 0; r < NR; ++r)
#pragma unroll
        for (int t = 0; t < NT; ++t) part[wave][r][t][lane] = acc[r][t];
    __syncthreads();
    // wavefront w adds the partial sums of the (r, t) tiles w, w + SW, ...
    for (int q = wave; q < NR * NT; q += SW) {
        const int r = q / NT, t = q % NT;
        i32x4_t s = part[0][r][t][lane];
#pragma unroll
        for (int w = 1; w < SW; ++w) s += part[w][r][t][lane];
        const int c = c0 + 16 * r + 4 * (lane / 16), row = m0 + 16 * t + lane % 16;
        if (c >= a.n || row >= a.m) continue;
        const float sx = LX ? scales[row] : a.xs[row];
        float v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = (float)s[i] * sx * a.ws[min(c + i, a.n - 1)];
        f8_store4<OF>(a.out, (size_t)row * a.n + c, a.n - c, v, a.n % 4 == 0);
    }
}

template <int NT, int NR, int XF>
hipError_t dense_launch(const ChannelArgs& a, hipStream_t st) {
    const dim3 grid((a.n + 16 * NR - 1) / (16 * NR), (a.m + 16 * NT - 1) / (16 * NT));
    const size_t lds = XF == MOE_DT_I8CH ? 0 : (size_t)a.m * a.k;
    if (a.odt == MOE_DT_BF16) i8_dense_stream_kernel<NT, NR, MOE_DT_BF16, XF><<<grid, WAVE * SW, lds, st>>>(a);
    else i8_dense_stream_kernel<NT, NR, MOE_DT_F32, XF><<<grid, WAVE * SW, lds, st>>>(a);
    return hipGetLastError();
}

}  // namespace

// Rows that are quantised by the product itself.
bool channel_matmul_takes(int m, int n, int k) { return m <= 16 && (int64_t)m * k <= I8_FUSE_VALUES && n <= 8192; }

hipError_t launch_channel_matmul(const ChannelArgs& a, hipStream_t st) {
    if (a.xdt == MOE_DT_BF16) return dense_launch<1, 1, MOE_DT_BF16>(a, st);
    if (a.xdt == MOE_DT_F32) return dense_launch<1, 1, MOE_DT_F32>(a, st);
    if (a.m <= 16) return dense_launch<1, 1, MOE_DT_I8CH>(a, st);
    const bool few = (long)((a.m + 31) / 32) * ((a.n + 31) / 32) <= 256 && a.k >= 1024;
    if (a.m <= 48 || few) return dense_launch<2, 2, MOE_DT_I8CH>(a, st);
    return launch_channel_matmul_tile(a, st);
}

}  // namespace moe
