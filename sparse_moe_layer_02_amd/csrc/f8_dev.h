// f8_dev.h - device building blocks of the 8-bit operators (e4m3 codes, one
// power-of-two scale per 128 columns of a row, one fp32 scale per 128 x 128
// block of a weight matrix).
//
// Row scale.  For a block of 128 values with largest magnitude a, s is the
// smallest power of two with a <= 448 s (448 is e4m3's largest value), at
// least 2^-126, and 1 for a block of zeros; it is kept as its e8m0 byte
// (exponent + 127).  x / s is then exact in fp32 unless it falls below fp32's
// normal range, far under e4m3's smallest step, so the only rounding is the
// conversion to e4m3 (nearest, ties to even), and the codes do not depend on
// how the quotient is computed.  A block that holds a NaN or an infinity gets
// the e8m0 byte 255 (NaN) and NaN codes: whatever reads it becomes NaN.
#pragma once
#include "common.h"

namespace moe {

constexpr int F8_BLK = 128;  // columns (and weight rows) that share a scale

typedef int i32x8_t __attribute__((ext_vector_type(8)));
typedef uint32_t f8_u4 __attribute__((ext_vector_type(4)));
typedef float f8_f4 __attribute__((ext_vector_type(4)));
typedef float f8_f16 __attribute__((ext_vector_type(16)));

// Bytes of one row's scales: one per 128 columns, padded to whole dwords.
__host__ __device__ __forceinline__ int f8_scale_ld(int cols) { return (cols + 4 * F8_BLK - 1) / (4 * F8_BLK) * 4; }
__host__ __device__ __forceinline__ int f8_blocks(int n) { return (n + F8_BLK - 1) / F8_BLK; }

// e8m0 byte of the scale, from the largest |x| bit pattern of the block
// (NaN patterns are above infinity's, so one integer maximum finds both).
__device__ __forceinline__ uint32_t f8_scale_byte(uint32_t amax) {
    if (amax >= 0x7F800000u) return 255u;
    if (amax == 0u) return 127u;
    // a = m 2^e with m in [1, 2): 448 = 1.75 * 2^8
    const int b = (int)(amax >> 23) - 8 + ((amax & 0x7FFFFFu) > 0x600000u ? 1 : 0);
    return (uint32_t)max(b, 1);
}
// 1 / s of a scale byte (1 .. 247)
__device__ __forceinline__ float f8_inv_scale(uint32_t byte) { return __uint_as_float((254u - byte) << 23); }

// Four codes of x[0..3] * inv; NaN codes for a block whose byte is 255.
__device__ __forceinline__ uint32_t f8_pack4(float a, float b, float c, float d, float inv, uint32_t byte) {
    int v = __builtin_amdgcn_cvt_pk_fp8_f32(a * inv, b * inv, 0, false);
    v = __builtin_amdgcn_cvt_pk_fp8_f32(c * inv, d * inv, v, true);
    return byte == 255u ? 0x7F7F7F7Fu : (uint32_t)v;
}

__device__ __forceinline__ uint32_t f8_abs_bits(float x) { return __float_as_uint(x) & 0x7FFFFFFFu; }

// Maximum over each 16-lane row, in every lane of the row (row rotations).
__device__ __forceinline__ uint32_t row16_max_u32(uint32_t v) {
    v = max(v, dpp_u32<0x128>(v));
    v = max(v, dpp_u32<0x124>(v));
    v = max(v, dpp_u32<0x122>(v));
    v = max(v, dpp_u32<0x121>(v));
    return v;
}

// Sixteen zero bytes: where a copy lane past the end of K reads.
__device__ const uint32_t f8_zeros[4] = {0u, 0u, 0u, 0u};

__device__ __forceinline__ i32x8_t f8_join(f8_u4 lo, f8_u4 hi) {
    return __builtin_bit_cast(i32x8_t, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
}

// A weight block's scale by a scalar load (wave-uniform address; the weights
// are never written by a kernel that reads them).
__device__ __forceinline__ float f8_uniform(const float* p, int i) {
    return reinterpret_cast<const __attribute__((address_space(4))) float*>(reinterpret_cast<uintptr_t>(p))[i];
}

// fp32 value of a scale byte (0 stands for 2^-127, 255 for NaN).
__device__ __forceinline__ float f8_scale_value(uint32_t byte) {
    return __uint_as_float(byte == 255u ? 0x7FC00000u : byte == 0u ? 0x00400000u : byte << 23);
}

// ---------------------------------------------------------------------------
// Products of e4m3 operands on the matrix cores.  Both operands hold the
// columns in the same order, so any order is right.
//
// The 8-bit instructions do not add in fp32: of every 8 consecutive columns'
// products each is cut (towards zero) to 13 bits below the largest one's
// leading bit before they are summed (measured on the device with one large
// and one small product; the groups of 8 and the accumulator add in fp32).
// That is 1.5e-5 of the result for normal operands (2-norm), 6e-5 for rows of
// silu(g) u, and up to 7 * 2^-13 of the largest product of every 8: not an fp32
// sum.  So:
//  - f8_dot16 / f8_dot32 widen the codes to bf16 (exact) and use the bf16
//    instructions, whose sums are fp32, at half the rate: for fp32 results, and
//    for everything in the layers (a code of the SwiGLU intermediate that falls
//    on the other side of its rounding is off by a whole step: with the 8-bit
//    instruction a 4096-token layer's fp32 y was off by 1.1e-3, now 8e-5);
//  - f8_mfma32 is the 8-bit instruction, for products that are rounded to bf16
//    (1.6e-3) next.
//
// D of the 16 x 16 forms: column (activation row) lane % 16, rows (weight rows)
// 4 (lane / 16) + v; of the 32 x 32 forms: column lane % 32, rows
// 8 (v / 4) + 4 (lane / 32) + v % 4.
// ---------------------------------------------------------------------------
// (scale: a power of two that multiplies the values)
__device__ __forceinline__ bf16x8_t f8_widen8(uint32_t lo, uint32_t hi, float scale = 1.0f) {
    bf16x2_t p[4];
    p[0] = __builtin_bit_cast(bf16x2_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, scale, false));
    p[1] = __builtin_bit_cast(bf16x2_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, scale, true));
    p[2] = __builtin_bit_cast(bf16x2_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, scale, false));
    p[3] = __builtin_bit_cast(bf16x2_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, scale, true));
    bf16x8_t r;
    __builtin_memcpy(&r, p, 16);
    return r;
}

// 32 codes of a lane's row as bf16: four operands of the bf16 instructions.
struct F8Wide {
    bf16x8_t v[4];
};
__device__ __forceinline__ F8Wide f8_widen(f8_u4 a, f8_u4 b, float scale = 1.0f) {
    return F8Wide{{f8_widen8(a.x, a.y, scale), f8_widen8(a.z, a.w, scale), f8_widen8(b.x, b.y, scale),
                   f8_widen8(b.z, b.w, scale)}};
}
__device__ __forceinline__ f8_f4 f8_dot16(const F8Wide& w, const F8Wide& x, f8_f4 c) {
#pragma unroll
    for (int j = 0; j < 4; ++j) c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w.v[j], x.v[j], c, 0, 0, 0);
    return c;
}
__device__ __forceinline__ f8_f16 f8_dot32(const F8Wide& w, const F8Wide& x, f8_f16 c) {
#pragma unroll
    for (int j = 0; j < 4; ++j) c = __builtin_amdgcn_mfma_f32_32x32x16_bf16(w.v[j], x.v[j], c, 0, 0, 0);
    return c;
}

// The 8-bit instruction; it applies the activation rows' e8m0 scales (byte
// SEL of `e`; the scale of the weight operand is 1).
constexpr int F8_ONE = 0x7F7F7F7F;
template <int SEL>
__device__ __forceinline__ f8_f16 f8_mfma32(i32x8_t w, i32x8_t x, f8_f16 c, uint32_t e) {
    return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(w, x, c, 0, 0, 0, F8_ONE, SEL, (int)e);
}

// Four adjacent results of a row (left: columns up to the row's end; wide: the
// row's start and the column are multiples of 4).
template <int OF>
__device__ __forceinline__ void f8_store4(void* out, size_t at, int left, const float (&v)[4], bool wide) {
    if constexpr (OF == MOE_DT_BF16) {
        uint16_t* p = static_cast<uint16_t*>(out) + at;
        if (wide) {
            *reinterpret_cast<uint2*>(p) = make_uint2(f32_to_bf16(v[0]) | (uint32_t)f32_to_bf16(v[1]) << 16,
                                                      f32_to_bf16(v[2]) | (uint32_t)f32_to_bf16(v[3]) << 16);
        } else {
            for (int j = 0; j < 4; ++j)
                if (j < left) p[j] = f32_to_bf16(v[j]);
        }
    } else {
        float* p = static_cast<float*>(out) + at;
        if (wide) {
            *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
        } else {
            for (int j = 0; j < 4; ++j)
                if (j < left) p[j] = v[j];
        }
    }
}

}  // namespace moe
