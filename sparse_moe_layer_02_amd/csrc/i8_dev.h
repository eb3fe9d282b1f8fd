// i8_dev.h - device building blocks of the int8 operators (codes with one fp32
// scale per activation row and one per weight row).
//
// Row scale.  s is the fp32 value nearest to a / 127, a the row's largest
// magnitude, at least 2^-120, and 1 for a row of zeros.  A code is the integer
// nearest to x / s, ties to even, decided exactly (i8_code), so codes do not
// depend on how the quotient is computed.  A row that holds a NaN or an infinity
// gets the scale NaN and codes 0: whatever reads it becomes NaN.
//
// Products of codes are summed in int32 by the matrix cores: exact while
// 128 * 128 * K < 2^31 (MOE_I8_MAX_K).  The only roundings of a product are the
// sum's to fp32 and the multiplications by the two scales.
#pragma once
#include "common.h"
#include "f8_dev.h"

namespace moe {

typedef int i32x4_t __attribute__((ext_vector_type(4)));

constexpr float I8_MIN_SCALE = 0x1p-120f;

// Scale of a row from the largest |x| bit pattern (NaN patterns are above
// infinity's, so one integer maximum finds both).
__device__ __forceinline__ float i8_scale(uint32_t amax) {
    if (amax >= 0x7F800000u) return __uint_as_float(0x7FC00000u);
    if (amax == 0u) return 1.0f;
    return fmaxf(__fdiv_rn(__uint_as_float(amax), 127.0f), I8_MIN_SCALE);
}

// What the codes of a row need of its scale.
struct I8Scale {
    float s, inv, half, below;  // below: the value under half
    bool none;                  // a NaN scale
};
__device__ __forceinline__ I8Scale i8_scale_parts(float s) {
    const float h = 0.5f * s;
    return I8Scale{s, __fdiv_rn(1.0f, s), h, __uint_as_float(__float_as_uint(h) - 1u), s != s};
}
// The code of x in the low byte.  m holds the integer nearest to x inv (one
// rounding, at 1.5 * 2^23, where the step is 1); x / s lies within 2^-16 of x inv,
// so that integer is off by one at most, and only next to a border.  The
// remainder x - n s then decides: next to a border it is a multiple of half a
// step of s of about half of s, which fp32 holds, so the fused product is exact.
__device__ __forceinline__ uint32_t i8_code(float x, const I8Scale& p) {
    constexpr float MAGIC = 12582912.0f;
    const float m = __fmaf_rn(x, p.inv, MAGIC);
    const float e = __fmaf_rn(-(m - MAGIC), p.s, x);
    const uint32_t b = __float_as_uint(m);
    const float lim = b & 1u ? p.below : p.half;  // an odd integer gives way at the border itself
    return b + (e > lim ? 1u : 0u) - (e < -lim ? 1u : 0u);
}
__device__ __forceinline__ uint32_t i8_pack4(float a, float b, float c, float d, const I8Scale& p) {
    // v_perm: bytes 0-3 of the second operand are 0-3, of the first 4-7
    const uint32_t lo = __builtin_amdgcn_perm(i8_code(b, p), i8_code(a, p), 0x0c0c0400u);
    const uint32_t hi = __builtin_amdgcn_perm(i8_code(d, p), i8_code(c, p), 0x04000c0cu);
    return p.none ? 0u : lo | hi;
}

// Eight columns of a row (16-byte aligned), their largest |x| bits, their codes.
template <int XF>
__device__ __forceinline__ void i8_load8(const void* x, size_t at, float (&v)[8]) {
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
__device__ __forceinline__ uint32_t i8_max8(const float (&v)[8]) {
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) m = max(m, f8_abs_bits(v[j]));
    return m;
}
__device__ __forceinline__ uint2 i8_codes8(const float (&v)[8], const I8Scale& p) {
    return make_uint2(i8_pack4(v[0], v[1], v[2], v[3], p), i8_pack4(v[4], v[5], v[6], v[7], p));
}

// Four adjacent scales of weight rows (any 4-byte alignment).
__device__ __forceinline__ f8_f4 i8_scales4(const float* p) {
    f8_f4 v;
    __builtin_memcpy(&v, p, 16);
    return v;
}

}  // namespace moe
