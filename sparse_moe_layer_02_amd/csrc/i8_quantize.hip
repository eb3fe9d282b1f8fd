// i8_quantize.hip - rows of fp32 or bf16 to int8 codes with one fp32 scale per
// row (i8_dev.h has the rounding).
//
// Bound by memory: 2 (or 4) bytes read, 1 written per value.  A workgroup takes
// a row; its values stay in registers between the maximum and the codes, so the
// row is read once (rows longer than that are read again).
#include "common.h"
#include "i8_dev.h"
#include "kernels.h"

namespace moe {
namespace {

constexpr int QT = 256;  // threads per row
constexpr int QN = 4;    // groups of 8 columns a thread keeps

template <int XF>
__device__ __forceinline__ void load8(const void* x, size_t at, float (&v)[8]) {
    if constexpr (XF == MOE_DT_BF16) {
        const uint4 u = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(x) + at);
        v[0] = bf16_lo(u.x); v[1] = bf16_hi(u.x); v[2] = bf16_lo(u.y); v[3] = bf16_hi(u.y);
        v[4] = bf16_lo(u.z); v[5] = bf16_hi(u.z); v[6] = bf16_lo(u.w); v[7] = bf16_hi(u.w);
    } else {
        const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(x) + at);
        const float4 u = p[0], w = p[1];
        v[0] = u.x; v[1] = u.y; v[2] = u.z; v[3] = u.w;
        v[4] = w.x; v[5] = w.y; v[6] = w.z; v[7] = w.w;
    }
}
__device__ __forceinline__ uint32_t max8(const float (&v)[8]) {
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) m = max(m, f8_abs_bits(v[j]));
    return m;
}
__device__ __forceinline__ uint2 codes8(const float (&v)[8], const I8Scale& p) {
    return make_uint2(i8_pack4(v[0], v[1], v[2], v[3], p), i8_pack4(v[4], v[5], v[6], v[7], p));
}

template <int XF>
__global__ __launch_bounds__(QT) void quantize_tokens_kernel(TokenQuantArgs a) {
    __shared__ uint32_t part[2][QT / WAVE];
    int at = 0;
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x, at ^= 1) {
        const int cols = row < a.rows0 ? a.cols : a.cols1;
        const size_t in = (size_t)row * a.ldx;
        int8_t* out = a.q + (size_t)row * a.ldq;
        float v[QN][8];
        uint32_t m = 0;
#pragma unroll
        for (int j = 0; j < QN; ++j) {
            const int c = 8 * (QT * j + threadIdx.x);
            if (c < cols) {
                load8<XF>(a.x, in + c, v[j]);
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) v[j][i] = 0.0f;
            }
        }
#pragma unroll
        for (int j = 0; j < QN; ++j) m = max(m, max8(v[j]));
        for (int c = 8 * (QT * QN + threadIdx.x); c < cols; c += 8 * QT) {
            float u[8];
            load8<XF>(a.x, in + c, u);
            m = max(m, max8(u));
        }
        m = wave_max_u32(m);
        // (two sets in turn: a row's maxima are read while the next row's are written)
        if (lane_id() == 0) part[at][threadIdx.x / WAVE] = m;
        __syncthreads();
        m = part[at][0];
#pragma unroll
        for (int w = 1; w < QT / WAVE; ++w) m = max(m, part[at][w]);
        const float s = i8_scale(m);
        const I8Scale p = i8_scale_parts(s);
        if (threadIdx.x == 0) a.s[row] = s;
#pragma unroll
        for (int j = 0; j < QN; ++j) {
            const int c = 8 * (QT * j + threadIdx.x);
            if (c < cols) *reinterpret_cast<uint2*>(out + c) = codes8(v[j], p);
        }
        for (int c = 8 * (QT * QN + threadIdx.x); c < cols; c += 8 * QT) {
            float u[8];
            load8<XF>(a.x, in + c, u);
            *reinterpret_cast<uint2*>(out + c) = codes8(u, p);
        }
    }
}

}  // namespace

hipError_t launch_quantize_tokens(const TokenQuantArgs& a, hipStream_t st, const KTime& kt) {
    const int grid = (int)(a.rows < 65536 ? a.rows : 65536);
    if (a.xdt == MOE_DT_BF16) launch_kernel(quantize_tokens_kernel<MOE_DT_BF16>, grid, QT, st, kt, a);
    else launch_kernel(quantize_tokens_kernel<MOE_DT_F32>, grid, QT, st, kt, a);
    return hipGetLastError();
}

}  // namespace moe
