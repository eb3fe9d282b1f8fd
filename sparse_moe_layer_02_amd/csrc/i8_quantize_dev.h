// i8_quantize_dev.h - rows of fp32 or bf16 to int8 codes by a workgroup per row
// (i8_dev.h has the rounding).
//
// Bound by memory: 2 (or 4) bytes read, 1 written per value.  A row's values stay
// in registers between the maximum and the codes, so it is read once (what is
// longer than the registers hold is read again).  4096 x 6144 bf16: 16.6 us, 4.5 TB/s
// read and written, as a large copy.
#pragma once
#include "common.h"
#include "i8_dev.h"
#include "kernels.h"

namespace moe {

constexpr int QN = 4;  // groups of 8 columns a thread keeps

// Rows first, first + stride, ... (the same in every thread of a workgroup of QT).
template <int XF, int QT>
__device__ __forceinline__ void quantize_token_rows(const TokenQuantArgs& a, int64_t first, int64_t stride) {
    __shared__ uint32_t part[2][QT / WAVE];
    int at = 0;
    for (int64_t row = first; row < a.rows; row += stride, at ^= 1) {
        const int cols = row < a.rows0 ? a.cols : a.cols1;
        const size_t in = (size_t)row * a.ldx;
        int8_t* out = a.q + (size_t)row * a.ldq;
        float v[QN][8];
        uint32_t m = 0;
#pragma unroll
        for (int j = 0; j < QN; ++j) {
            const int c = 8 * (QT * j + threadIdx.x);
            if (c < cols) {
                i8_load8<XF>(a.x, in + c, v[j]);
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) v[j][i] = 0.0f;
            }
        }
#pragma unroll
        for (int j = 0; j < QN; ++j) m = max(m, i8_max8(v[j]));
        for (int c = 8 * (QT * QN + threadIdx.x); c < cols; c += 8 * QT) {
            float u[8];
            i8_load8<XF>(a.x, in + c, u);
            m = max(m, i8_max8(u));
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
            if (c < cols) *reinterpret_cast<uint2*>(out + c) = i8_codes8(v[j], p);
        }
        for (int c = 8 * (QT * QN + threadIdx.x); c < cols; c += 8 * QT) {
            float u[8];
            i8_load8<XF>(a.x, in + c, u);
            *reinterpret_cast<uint2*>(out + c) = i8_codes8(u, p);
        }
    }
}

}  // namespace moe
