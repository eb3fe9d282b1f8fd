// quantize_dev.h - rows of fp32 or bf16 to e4m3 codes with one power-of-two
// scale per 128 columns (f8_dev.h has the rounding).
//
// Bound by memory: 2 (or 4) bytes read, 1 + 1/128 written per value, no
// reuse (4096 x 6144 bf16: 14 us, 5.4 TB/s).  A 16-lane row of a wavefront takes
// one 128-column block, eight columns per lane (one or two 16-byte loads, one
// 8-byte store), so the block's maximum is four DPP steps and nothing goes
// through LDS.
#pragma once
#include "common.h"
#include "f8_dev.h"
#include "kernels.h"

namespace moe {

// Blocks first, first + stride, ... of the rows, 16 lanes each (every lane of a
// 16-lane row passes the same `first`).
template <int XF>
__device__ __forceinline__ void quantize_blocks(const QuantArgs& a, int64_t first, int64_t stride) {
    const int nb = f8_scale_ld(a.cols);  // blocks per row, padding included
    const int64_t n = (int64_t)a.rows * nb;
    const int l = threadIdx.x % 16;
    for (int64_t i = first; i < n; i += stride) {
        const int64_t row = i / nb;
        const int b = (int)(i - row * nb), c = b * F8_BLK + 8 * l;
        float v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = 0.0f;
        if (c < a.cols) {  // cols is a multiple of 16: a lane's eight columns are all in or all out
            if constexpr (XF == MOE_DT_BF16) {
                const uint4 u = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.x) + row * a.ldx + c);
                v[0] = bf16_lo(u.x); v[1] = bf16_hi(u.x); v[2] = bf16_lo(u.y); v[3] = bf16_hi(u.y);
                v[4] = bf16_lo(u.z); v[5] = bf16_hi(u.z); v[6] = bf16_lo(u.w); v[7] = bf16_hi(u.w);
            } else {
                const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(a.x) + row * a.ldx + c);
                const float4 u = p[0], w = p[1];
                v[0] = u.x; v[1] = u.y; v[2] = u.z; v[3] = u.w;
                v[4] = w.x; v[5] = w.y; v[6] = w.z; v[7] = w.w;
            }
        }
        uint32_t m = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) m = max(m, f8_abs_bits(v[j]));
        const uint32_t byte = f8_scale_byte(row16_max_u32(m));
        const float inv = f8_inv_scale(byte);
        if (c < a.cols)
            *reinterpret_cast<uint2*>(a.q + row * (int64_t)a.cols + c) =
                make_uint2(f8_pack4(v[0], v[1], v[2], v[3], inv, byte), f8_pack4(v[4], v[5], v[6], v[7], inv, byte));
        if (l == 0) a.e[row * nb + b] = (uint8_t)byte;
    }
}

}  // namespace moe
