// tile_dev.h - building blocks of the kernels that multiply tiles of 8-bit rows
// through LDS (f8_tile.hip, i8_tile.hip): the tile's shape, the copies of its
// stages, the lanes' places in a stage, and the way of the results to memory.
#pragma once
#include <utility>

#include "common.h"
#include "dma_dev.h"
#include "f8_dev.h"
#include "gemm_dev.h"
#include "kernels.h"

namespace moe {
namespace {

// Tile shapes: GM x GN wavefronts (GM along the activation rows, GN along the
// weight rows), each NB x NJ blocks of 32 x 32, NST stages in LDS.
template <int NB_, int NJ_, int GM_, int GN_, int NST_>
struct Shape {
    static constexpr int NB = NB_, NJ = NJ_, GM = GM_, GN = GN_, NST = NST_;
    static constexpr int W = GM * GN;              // wavefronts
    static constexpr int BM = 32 * NB * GM;        // activation rows
    static constexpr int WR = 32 * NJ, TN = WR * GN;         // weight rows per wavefront, per tile
    static constexpr int WB = TN * F8_BLK, XB = BM * F8_BLK; // bytes of a stage
    static constexpr int WQ = WB / 1024 / W;                 // 1 KB copies per wavefront and stage
    static constexpr int XQ = (XB / 1024 + W - 1) / W;       // (at most)
    static_assert(WQ * 1024 * W == WB, "weight copies");
    static constexpr int WAVES = NST * (WB + XB) <= 80 * 1024 && W == 8 ? 4 : 2;  // per SIMD: two workgroups where LDS has room
};

// A wave-uniform pointer in scalar registers (where the compiler cannot see it).
template <class P>
__device__ __forceinline__ const P* uniform_ptr(const P* p) {
    const uint64_t u = reinterpret_cast<uint64_t>(p);
    const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)u), hi = __builtin_amdgcn_readfirstlane((uint32_t)(u >> 32));
    return reinterpret_cast<const P*>(((uint64_t)hi << 32) | lo);
}
__device__ __forceinline__ __amdgpu_buffer_rsrc_t tile_buffer(const uint8_t* p) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(p), 0, 0xFFFFFFFF, 0x00020000);
}
template <bool NT = false>  // NT: non-temporal
__device__ __forceinline__ void buffer_copy16(__amdgpu_buffer_rsrc_t r, uint32_t off, int k0, uint8_t* dst) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void*)(dst), 16, (int)off, k0, 0, NT ? 2 : 0);
}

// Copy lane l of copy c fills row 8 c + l / 8, slot l % 8.
__device__ __forceinline__ int copy_row(int c, int lane) { return 8 * c + (lane >> 3); }
__device__ __forceinline__ int copy_chunk(int row, int lane) { return 16 * ((lane & 7) ^ pair_swz(row)); }

// Byte offsets of the four 16-byte chunks a lane multiplies in a stage, from the
// first row of a block of 32 rows (the swizzle repeats every 16 rows, so they
// serve every block): row lane % 32, chunks 2 (lane / 32) + {0, 1, 4, 5}.
struct F8Lane {
    uint32_t o[4];
};
__device__ __forceinline__ F8Lane tile_lane(int lane) {
    F8Lane f;
#pragma unroll
    for (int k = 0; k < 4; ++k)
        f.o[k] = (lane & 31) * F8_BLK + (((4 * (k >> 1) + 2 * (lane >> 5) + (k & 1)) ^ pair_swz(lane & 31)) << 4);
    return f;
}

// f(ic<0>()), ..., f(ic<N - 1>()): indices that are constants from the start.
template <class F, int... I>
__device__ __forceinline__ void each_of(F f, std::integer_sequence<int, I...>) {
    (f(ic<I>()), ...);
}
template <int N, class F>
__device__ __forceinline__ void each(F f) {
    each_of(f, std::make_integer_sequence<int, N>());
}

// The ring's stages as separate objects: the compiler then knows that reading
// one does not wait for the copies into another.
#define F8_TILE_LDS(S)                                                                         \
    __shared__ __attribute__((aligned(1024))) uint8_t W0[S::WB];                               \
    __shared__ __attribute__((aligned(1024))) uint8_t W1[S::WB];                               \
    __shared__ __attribute__((aligned(1024))) uint8_t W2[S::NST > 2 ? S::WB : 16];             \
    __shared__ __attribute__((aligned(1024))) uint8_t W3[S::NST > 3 ? S::WB : 16];             \
    __shared__ __attribute__((aligned(1024))) uint8_t X0[S::XB];                               \
    __shared__ __attribute__((aligned(1024))) uint8_t X1[S::XB];                               \
    __shared__ __attribute__((aligned(1024))) uint8_t X2[S::NST > 2 ? S::XB : 16];             \
    __shared__ __attribute__((aligned(1024))) uint8_t X3[S::NST > 3 ? S::XB : 16];             \
    uint8_t* const WS[4] = {W0, W1, W2, W3};                                                   \
    uint8_t* const XS[4] = {X0, X1, X2, X3}

// f(the first N of S)
template <int N, class F>
__device__ __forceinline__ void ring(uint8_t* const (&S)[4], F f) {
    if constexpr (N == 2) {
        uint8_t* const R[2] = {S[0], S[1]};
        f(R);
    } else if constexpr (N == 3) {
        uint8_t* const R[3] = {S[0], S[1], S[2]};
        f(R);
    } else {
        f(S);
    }
}

// Results to memory through LDS, so that eight lanes store 128 consecutive bytes
// of a row (a lane holds four columns of a row per eight; straight from the
// registers, 2772 x 4096 x 192 to fp32 took 32 us and now 22, to bf16 18 / 17, to
// 4089 columns, whose rows start anywhere, 39 / 23; 4096 x 4096 x 6144 7% less, the
// down product of 4096 tokens 5%).  A wavefront's region holds 32
// rows of 128 bytes, 16-byte chunks swizzled by row.
constexpr int OUT_REGION = 32 * 128;
template <class S>
__device__ __forceinline__ uint8_t* out_region(uint8_t* const (&WS)[4], int wave) {
    constexpr int PER = S::WB / OUT_REGION;  // regions in a stage's weight buffer
    static_assert(2 * PER >= S::W, "room for every wavefront");
    if constexpr (PER >= S::W) return WS[0] + wave * OUT_REGION;
    else return (wave < PER ? WS[0] : WS[1]) + wave % PER * OUT_REGION;
}
__device__ __forceinline__ int out_chunk(int row, int c) { return row * 128 + 16 * (c ^ (row & 7)); }
// (the wavefront's own LDS accesses keep their order; this keeps the compiler to it)
__device__ __forceinline__ void out_fence() { __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront"); }
// The lane's 16 fp32 results of a block: one activation row, 32 columns with the other half's.
__device__ __forceinline__ void out_put_f32(uint8_t* R, int lane, const f8_f16& p) {
#pragma unroll
    for (int q = 0; q < 4; ++q)
        *reinterpret_cast<f8_f4*>(R + out_chunk(lane & 31, 2 * q + (lane >> 5))) = f8_f4{p[4 * q], p[4 * q + 1], p[4 * q + 2], p[4 * q + 3]};
}
// The same rounded to bf16, as columns 32 j .. + 31 of the region's 64.
__device__ __forceinline__ void out_put_bf16(uint8_t* R, int lane, int j, const f8_f16& p) {
#pragma unroll
    for (int q = 0; q < 4; ++q)
        *reinterpret_cast<uint2*>(R + out_chunk(lane & 31, 4 * j + q) + 8 * (lane >> 5)) =
            make_uint2(f32_to_bf16(p[4 * q]) | (uint32_t)f32_to_bf16(p[4 * q + 1]) << 16,
                       f32_to_bf16(p[4 * q + 2]) | (uint32_t)f32_to_bf16(p[4 * q + 3]) << 16);
}
// Rows of the region (the first `rows`, `left` columns of BYTES / sizeof(E)) to
// `out`, n elements per row, in units of U.
template <class E, class U, int BYTES>
__device__ __forceinline__ void out_rows(const uint8_t* R, int lane, E* out, size_t n, int rows, int left) {
    constexpr int PER = BYTES / sizeof(U), ROWS = WAVE / PER, EU = sizeof(U) / sizeof(E);  // lanes per row, rows at once
#pragma unroll
    for (int s = 0; s < 32 / ROWS; ++s) {
        const int r = ROWS * s + lane / PER, u = lane % PER;
        const U v = *reinterpret_cast<const U*>(R + out_chunk(r, u * (int)sizeof(U) / 16) + u * sizeof(U) % 16);
        if (r < rows && u * EU < left) *reinterpret_cast<U*>(out + r * n + u * EU) = v;
    }
}

// Whether a tile holds all rows of its expert.
template <int BM>
__device__ __forceinline__ bool one_tile(const FfnArgs& f, const TileRows& tr) {
    return tr.g == f.E ? f.T <= BM : f.offsets[tr.g + 1] - f.offsets[tr.g] <= BM;
}

}  // namespace
}  // namespace moe
