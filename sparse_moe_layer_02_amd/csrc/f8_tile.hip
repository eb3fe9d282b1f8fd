// f8_tile.hip - e4m3 products for many activation rows per weight matrix.
//
//   gate/up:  h[r, c] = silu(x_r Wg_c) (x_r Wu_c), quantised per 128 columns
//   down:     slot_out[f, :] = w_f (h_r Wd^T)
//   dense:    out[m, n] = x_m W_n
//
// A workgroup of eight wavefronts computes 32 NB GM activation rows x 256
// weight rows (gate/up: 128 gate and the same 128 up rows, so that a tile holds
// whole scale blocks of h); GM wavefronts along the activation rows, 8 / GM
// along the weight rows, each NB x GM blocks of 32 x 32.  A stage is one step of 128
// columns, the width of a scale block: 128-byte rows, copied straight from
// global memory into LDS (eight whole cache lines per copy instruction, 16-byte
// chunks swizzled by row as dma_dev.h describes), in a ring of NST stages behind
// one barrier per stage.  A block's partial sum over the stage starts from zero
// on the matrix cores and is added with the weight block's fp32 scale, which is
// uniform over the block (one v_fma per 16 x 64 results, an SGPR operand); the
// activation rows' e8m0 scales are applied by the matrix instruction.
//
// WIDE: the codes are widened to bf16 and the sums are fp32 (f8_dev.h); taken
// for fp32 results.  Otherwise the 8-bit instruction, twice the rate, for
// results that are rounded to bf16 or e4m3 next.
//
// A tile computes only the 32-row blocks that hold rows: blocks are dealt to the
// two wavefront rows in turn, and each wavefront runs the K loop built for its
// number of live blocks.
#include "common.h"
#include "dma_dev.h"
#include "f8_dev.h"
#include "gemm_dev.h"
#include "kernels.h"

namespace moe {
namespace {

constexpr int TW = 8;              // wavefronts
constexpr int TN = 256;            // weight rows per tile
constexpr int TWB = TN * F8_BLK;   // bytes of one stage's weight rows
constexpr int TWC = TWB / 1024 / TW;  // 1 KB weight copies per wavefront and stage

// Tile shapes: NB blocks of 32 activation rows per wavefront, GM wavefronts
// along them, NST stages in LDS (what 160 KB hold).
template <int NB_, int GM_, int NST_>
struct Shape {
    static constexpr int NB = NB_, GM = GM_, NST = NST_;
    static constexpr int BM = 32 * NB * GM;        // activation rows
    static constexpr int GN = TW / GM;             // wavefronts along the weight rows
    static constexpr int WR = TN / GN;             // weight rows per wavefront: GM blocks of 32
    static constexpr int XB = BM * F8_BLK;         // bytes of one stage's activation rows
    static constexpr int XCP = XB / 1024;          // 1 KB copies of them
    static constexpr int XQ = (XCP + TW - 1) / TW; // at most, per wavefront
};
typedef Shape<1, 1, 4> Rows32;
typedef Shape<2, 1, 3> Rows64;
typedef Shape<2, 2, 3> Rows128;
typedef Shape<4, 2, 2> Rows256;

// Per-lane sources of one tile.
template <class S>
struct F8Tile {
    static constexpr int NB = S::NB;
    const uint8_t* wsrc[TWC];  // weight row bytes this copy lane fetches at K = 0
    const uint8_t* xsrc[S::XQ];// activation row bytes
    int wch, xch;              // the lane's 16-byte chunk in a stage row (weights, activations), in bytes
    const uint8_t* ep[NB];     // scale bytes of the lane's activation row in each live block
    const float* sp[2];        // block scales of the wavefront's weight rows (gate/up: of gate, of up)
    int K, nst;
};

// Copy lane l of copy c fills row 8 c + l / 8, slot l % 8.
__device__ __forceinline__ int copy_row(int c, int lane) { return 8 * c + (lane >> 3); }
__device__ __forceinline__ int copy_chunk(int row, int lane) { return 16 * ((lane & 7) ^ pair_swz(row)); }

// 32 codes of row r: columns 64 h + 32 (lane / 32) .. + 31 of the stage.
struct F8Row {
    f8_u4 a, b;
};
__device__ __forceinline__ F8Row tile_row(const uint8_t* S, int r, int h) {
    const int c = 4 * h + 2 * (lane_id() >> 5), sw = pair_swz(r);
    const uint8_t* p = S + r * F8_BLK;
    return F8Row{*reinterpret_cast<const f8_u4*>(p + ((c ^ sw) << 4)), *reinterpret_cast<const f8_u4*>(p + (((c + 1) ^ sw) << 4))};
}

// The K loop of one wavefront with L live blocks and XC activation copies per
// stage; acc[i][j]: block i (activation rows) x weight row block j.  SPLIT: the
// wavefront's one weight block holds 16 gate rows and 16 up rows.
template <class S, int L, int XC, bool WIDE, bool SPLIT>
__device__ __forceinline__ void tile_loop(const F8Tile<S>& g, uint8_t* const (&W)[S::NST], uint8_t* const (&X)[S::NST],
                                          f8_f16 (&acc)[S::NB][S::GM]) {
    constexpr int NST = S::NST, NB = S::NB, NJ = S::GM;
    const int lane = lane_id(), wave = wave_index(), mh = wave / S::GN, wn = wave % S::GN, l32 = lane & 31;
    constexpr int NC = TWC + XC;
    const int last = g.nst - 1, ktail = g.K & (F8_BLK - 1);
    auto issue = [&](uint8_t* w, uint8_t* x, int kb) {
        kb = min(kb, last);  // (stages past the end re-read the last; not used)
        const int k0 = kb * F8_BLK;
        if (kb == last && ktail) {  // columns past K come from a row of zeros
#pragma unroll
            for (int q = 0; q < TWC; ++q)
                copy16(g.wch < ktail ? g.wsrc[q] + k0 : reinterpret_cast<const uint8_t*>(f8_zeros), w + (q * TW + wave) * 1024);
#pragma unroll
            for (int q = 0; q < XC; ++q)
                copy16(g.xch < ktail ? g.xsrc[q] + k0 : reinterpret_cast<const uint8_t*>(f8_zeros), x + (q * TW + wave) * 1024);
            return;
        }
#pragma unroll
        for (int q = 0; q < TWC; ++q) copy16(g.wsrc[q] + k0, w + (q * TW + wave) * 1024);
#pragma unroll
        for (int q = 0; q < XC; ++q) copy16(g.xsrc[q] + k0, x + (q * TW + wave) * 1024);
    };
    uint32_t ev[NB], en[NB];
#pragma unroll
    for (int i = 0; i < L; ++i) en[i] = *reinterpret_cast<const uint32_t*>(g.ep[i]);
#pragma unroll
    for (int s = 0; s < NST - 1; ++s) issue(W[s], X[s], s);
    float sw[2];
    sw[0] = f8_uniform(g.sp[0], 0);
    sw[1] = f8_uniform(g.sp[1], 0);
    auto stage = [&](auto bb, auto ss, int kb) {
        constexpr int B = decltype(bb)::value;    // LDS stage
        constexpr int SEL = decltype(ss)::value;  // kb % 4: byte of the activation scales
        wait_vm<(NST - 2) * NC>();
        barrier_nofence();
        issue(W[(B + NST - 1) % NST], X[(B + NST - 1) % NST], kb + NST - 1);
        if constexpr (SEL == 0) {
#pragma unroll
            for (int i = 0; i < L; ++i) {
                ev[i] = en[i];
                en[i] = *reinterpret_cast<const uint32_t*>(g.ep[i] + (kb + 4 <= last ? kb + 4 : 0));
            }
        }
        const float s0 = sw[0], s1 = sw[1];
        sw[0] = f8_uniform(g.sp[0], min(kb + 1, last));
        sw[1] = f8_uniform(g.sp[1], min(kb + 1, last));
        if constexpr (L > 0) {
            F8Row w[NJ][2];
#pragma unroll
            for (int j = 0; j < NJ; ++j)
#pragma unroll
                for (int h = 0; h < 2; ++h) w[j][h] = tile_row(W[B], S::WR * wn + 32 * j + l32, h);
            F8Wide ww[NJ][2];
            if constexpr (WIDE) {
#pragma unroll
                for (int j = 0; j < NJ; ++j)
#pragma unroll
                    for (int h = 0; h < 2; ++h) ww[j][h] = f8_widen(w[j][h].a, w[j][h].b);
            }
#pragma unroll
            for (int i = 0; i < L; ++i) {
                const int xr = 32 * (mh + S::GM * i) + l32;
                const F8Row x0 = tile_row(X[B], xr, 0), x1 = tile_row(X[B], xr, 1);
                auto add = [&](const f8_f16& p, int j) {
#pragma unroll
                    for (int v = 0; v < 16; ++v)
                        acc[i][j][v] = fmaf((SPLIT ? v >= 8 : j > 0) ? s1 : s0, p[v], acc[i][j][v]);
                };
                if constexpr (WIDE) {
                    const F8Wide v0 = f8_widen(x0.a, x0.b), v1 = f8_widen(x1.a, x1.b);
                    const float sx = f8_scale_value((ev[i] >> (8 * SEL)) & 255u);
#pragma unroll
                    for (int j = 0; j < NJ; ++j) add(f8_dot32(ww[j][1], v1, f8_dot32(ww[j][0], v0, f8_f16{})) * sx, j);
                } else {
                    const i32x8_t v0 = f8_join(x0.a, x0.b), v1 = f8_join(x1.a, x1.b);
#pragma unroll
                    for (int j = 0; j < NJ; ++j) {
                        const f8_f16 p = f8_mfma32<SEL>(f8_join(w[j][0].a, w[j][0].b), v0, f8_f16{}, ev[i]);
                        add(f8_mfma32<SEL>(f8_join(w[j][1].a, w[j][1].b), v1, p, ev[i]), j);
                    }
                }
            }
            wait_lgkm0();  // this stage's reads are done before the next barrier releases its refill
        }
    };
    // twelve (four) stages run through every pair of LDS stage and scale byte
    constexpr int CYC = NST == 3 ? 12 : 4;
    for (int kb = 0; kb < g.nst; kb += CYC) {
#define F8_STAGE(n) \
    if constexpr (n < CYC) { if (kb + n < g.nst) stage(ic<(n) % NST>(), ic<(n) % 4>(), kb + n); }
        F8_STAGE(0) F8_STAGE(1) F8_STAGE(2) F8_STAGE(3) F8_STAGE(4) F8_STAGE(5)
        F8_STAGE(6) F8_STAGE(7) F8_STAGE(8) F8_STAGE(9) F8_STAGE(10) F8_STAGE(11)
#undef F8_STAGE
    }
    wait_vm<0>();  // no copy may still be writing LDS when the workgroup ends
}

// Runs the loop built for this wavefront's live blocks (rows of the tile: nrows).
// A round of activation copies of the eight wavefronts covers 64 rows.
template <class S, bool WIDE, bool SPLIT>
__device__ __forceinline__ void tile_run(const F8Tile<S>& g, int nrows, uint8_t* const (&W)[S::NST],
                                         uint8_t* const (&X)[S::NST], f8_f16 (&acc)[S::NB][S::GM]) {
    const int wave = wave_index(), nblk = (nrows + 31) / 32, live = (nblk - wave / S::GN + S::GM - 1) / S::GM;
    auto run = [&](auto l, auto xc) { tile_loop<S, decltype(l)::value, decltype(xc)::value, WIDE, SPLIT>(g, W, X, acc); };
    if constexpr (S::GM == 2) {
        if constexpr (S::NB == 4) {
            if (nblk > 6) return live == 4 ? run(ic<4>(), ic<4>()) : run(ic<3>(), ic<4>());
            if (nblk > 4) return live == 3 ? run(ic<3>(), ic<3>()) : run(ic<2>(), ic<3>());
        }
        if (nblk > 2) return live == 2 ? run(ic<2>(), ic<2>()) : run(ic<1>(), ic<2>());
        return live == 1 ? run(ic<1>(), ic<1>()) : run(ic<0>(), ic<1>());
    } else if constexpr (S::NB == 2) {
        return live == 2 ? run(ic<2>(), ic<1>()) : run(ic<1>(), ic<1>());
    } else {  // four copies of 8 rows: the first four wavefronts
        return wave < 4 ? run(ic<1>(), ic<1>()) : run(ic<1>(), ic<0>());
    }
}

// The ring's stages as separate objects: the compiler then knows that reading
// one does not wait for the copies into another.
#define F8_TILE_LDS(S)                                                                         \
    __shared__ __attribute__((aligned(1024))) uint8_t W0[TWB];                                 \
    __shared__ __attribute__((aligned(1024))) uint8_t W1[TWB];                                 \
    __shared__ __attribute__((aligned(1024))) uint8_t W2[S::NST > 2 ? TWB : 16];               \
    __shared__ __attribute__((aligned(1024))) uint8_t W3[S::NST > 3 ? TWB : 16];               \
    __shared__ __attribute__((aligned(1024))) uint8_t X0[S::XB];                               \
    __shared__ __attribute__((aligned(1024))) uint8_t X1[S::XB];                               \
    __shared__ __attribute__((aligned(1024))) uint8_t X2[S::NST > 2 ? S::XB : 16];             \
    __shared__ __attribute__((aligned(1024))) uint8_t X3[S::NST > 3 ? S::XB : 16];             \
    uint8_t* const WS[4] = {W0, W1, W2, W3};                                                   \
    uint8_t* const XS[4] = {X0, X1, X2, X3}

template <class S, bool WIDE, bool SPLIT>
__device__ __forceinline__ void tile_go(const F8Tile<S>& g, int nrows, uint8_t* const (&WS)[4], uint8_t* const (&XS)[4],
                                        f8_f16 (&acc)[S::NB][S::GM]) {
#pragma unroll
    for (int i = 0; i < S::NB; ++i)
#pragma unroll
        for (int j = 0; j < S::GM; ++j) acc[i][j] = f8_f16{};
    if constexpr (S::NST == 2) {
        uint8_t* const W[2] = {WS[0], WS[1]};
        uint8_t* const X[2] = {XS[0], XS[1]};
        tile_run<S, WIDE, SPLIT>(g, nrows, W, X, acc);
    } else if constexpr (S::NST == 3) {
        uint8_t* const W[3] = {WS[0], WS[1], WS[2]};
        uint8_t* const X[3] = {XS[0], XS[1], XS[2]};
        tile_run<S, WIDE, SPLIT>(g, nrows, W, X, acc);
    } else {
        tile_run<S, WIDE, SPLIT>(g, nrows, WS, XS, acc);
    }
}

template <class S>
__global__ __launch_bounds__(64 * TW) void f8_gateup_tile_kernel(F8Ffn a) {
    constexpr int NB = S::NB, BM = S::BM, HC = S::WR / 2;  // h columns per wavefront
    F8_TILE_LDS(S);
    __shared__ uint32_t red[S::GN][BM];
    int tile, ntile;
    if (!work_item<4>(tile_count(a.f), tile, ntile)) return;
    TileRows tr;
    if (!tile_rows<BM>(a.f, tile, tr)) return;
    const bool shared = tr.g == a.f.E;
    const int F = shared ? a.f.Fs : a.f.F, d = a.f.d, n0 = ntile * F8_BLK;
    if (n0 >= F) return;
    const int lane = lane_id(), wave = wave_index(), mh = wave / S::GN, wn = wave % S::GN, l32 = lane & 31;
    const MatRef& G = shared ? a.f.s_gate : a.f.gate;
    const MatRef& U = shared ? a.f.s_up : a.f.up;
    const size_t e = shared ? 0 : tr.g;
    F8Tile<S> g;
    g.K = d;
    g.nst = f8_blocks(d);
    // stage rows 2 HC m .. + HC - 1: gate rows n0 + HC m .., the HC rows after them: the same up rows
#pragma unroll
    for (int q = 0; q < TWC; ++q) {
        const int sr = copy_row(q * TW + wave, lane), n = min(n0 + HC * (sr / (2 * HC)) + sr % HC, F - 1);
        g.wch = copy_chunk(sr, lane);
        g.wsrc[q] = static_cast<const uint8_t*>((sr & HC) ? U.q : G.q) + (e * F + n) * d + g.wch;
    }
    auto token = [&](int r) {  // rows past the tile repeat its first; their results are not stored
        r = r < tr.nrows ? r : 0;
        if (shared) return tr.rbeg - a.f.T * a.f.k + r;
        const int f = a.f.perm_rows[tr.rbeg + r];
        return f >= 0 && f < a.f.T * a.f.k ? f / a.f.k : 0;
    };
#pragma unroll
    for (int q = 0; q < S::XQ; ++q) {
        const int sr = copy_row(q * TW + wave, lane);
        g.xch = copy_chunk(sr, lane);
        g.xsrc[q] = a.xq + (size_t)token(sr) * d + g.xch;
    }
#pragma unroll
    for (int i = 0; i < NB; ++i) g.ep[i] = a.xe + (size_t)token(32 * (mh + S::GM * i) + l32) * f8_scale_ld(d);
    const size_t srow = (e * f8_blocks(F) + ntile) * g.nst;
    g.sp[0] = reinterpret_cast<const float*>(G.scale) + srow;
    g.sp[1] = reinterpret_cast<const float*>(U.scale) + srow;
    f8_f16 acc[NB][S::GM];
    tile_go<S, false, S::GM == 1>(g, tr.nrows, WS, XS, acc);
    // h and its largest magnitude per row over the tile's 128 columns
    // (a wavefront of GM = 2 has gate and up in its two blocks, of GM = 1 in the
    // lower and upper half of one)
    constexpr int NV = HC / 2;  // h values per lane
    const int c0 = n0 + HC * wn;
    const bool in = c0 < F;  // (F is a multiple of 64)
    float h[NB][NV];
#pragma unroll
    for (int i = 0; i < NB; ++i) {
        uint32_t m = 0;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            h[i][v] = silu_f32(acc[i][0][v]) * (S::GM == 2 ? acc[i][S::GM - 1][v] : acc[i][0][(v + NV) & 15]);
            m = max(m, f8_abs_bits(h[i][v]));
        }
        m = max(m, (uint32_t)__shfl_xor((int)m, 32));
        if (lane < 32) red[wn][32 * (mh + S::GM * i) + l32] = in ? m : 0u;
    }
    __syncthreads();
    const int hi = lane >> 5;
#pragma unroll
    for (int i = 0; i < NB; ++i) {
        const int r = 32 * (mh + S::GM * i) + l32;
        uint32_t m = 0;
#pragma unroll
        for (int w = 0; w < S::GN; ++w) m = max(m, red[w][r]);
        const uint32_t byte = f8_scale_byte(m);
        const float inv = f8_inv_scale(byte);
        uint32_t c[NV / 4];
#pragma unroll
        for (int j = 0; j < NV / 4; ++j)
            c[j] = f8_pack4(h[i][4 * j], h[i][4 * j + 1], h[i][4 * j + 2], h[i][4 * j + 3], inv, byte);
        // lanes l and l + 32 hold alternate 4-column runs of a row: each takes NV adjacent columns
        uint32_t o[NV / 8];
#pragma unroll
        for (int j = 0; j < NV / 8; ++j) o[j] = (uint32_t)__shfl_xor((int)(hi ? c[j] : c[j + NV / 8]), 32);
        if (r >= tr.nrows) continue;
        const size_t hrow = (size_t)(tr.rbeg + r);
        uint8_t* dst = a.hq + hrow * a.f.ldh + c0 + NV * hi;
        if constexpr (NV == 16) {
            if (in) *reinterpret_cast<uint4*>(dst) = hi ? make_uint4(o[0], c[2], o[1], c[3]) : make_uint4(c[0], o[0], c[1], o[1]);
        } else {
            if (in) *reinterpret_cast<uint2*>(dst) = hi ? make_uint2(o[0], c[1]) : make_uint2(c[0], o[0]);
        }
        if (wn == 0 && hi == 0) a.he[hrow * f8_scale_ld(a.f.ldh) + ntile] = (uint8_t)byte;
    }
}

template <class S>
__global__ __launch_bounds__(64 * TW) void f8_down_tile_kernel(F8Ffn a) {
    constexpr int NB = S::NB, BM = S::BM;
    F8_TILE_LDS(S);
    int tile, ntile;
    if (!work_item<4>(tile_count(a.f), tile, ntile)) return;
    TileRows tr;
    if (!tile_rows<BM>(a.f, tile, tr)) return;
    const bool shared = tr.g == a.f.E;
    const int F = shared ? a.f.Fs : a.f.F, d = a.f.d, n0 = ntile * TN;
    const int lane = lane_id(), wave = wave_index(), mh = wave / S::GN, wn = wave % S::GN, l32 = lane & 31;
    const MatRef& D = shared ? a.f.s_down : a.f.down;
    const size_t e = shared ? 0 : tr.g;
    F8Tile<S> g;
    g.K = F;
    g.nst = f8_blocks(F);
#pragma unroll
    for (int q = 0; q < TWC; ++q) {
        const int sr = copy_row(q * TW + wave, lane);
        g.wch = copy_chunk(sr, lane);
        g.wsrc[q] = static_cast<const uint8_t*>(D.q) + (e * d + min(n0 + sr, d - 1)) * F + g.wch;
    }
#pragma unroll
    for (int q = 0; q < S::XQ; ++q) {
        const int sr = copy_row(q * TW + wave, lane);
        g.xch = copy_chunk(sr, lane);
        g.xsrc[q] = a.hq + (size_t)(tr.rbeg + (sr < tr.nrows ? sr : 0)) * a.f.ldh + g.xch;
    }
#pragma unroll
    for (int i = 0; i < NB; ++i) {
        const int r = 32 * (mh + S::GM * i) + l32;
        g.ep[i] = a.he + (size_t)(tr.rbeg + (r < tr.nrows ? r : 0)) * f8_scale_ld(a.f.ldh);
    }
    const int c0 = n0 + S::WR * wn;
#pragma unroll
    for (int j = 0; j < 2; ++j)  // (one block: both the same)
        g.sp[j] = reinterpret_cast<const float*>(D.scale) + (e * f8_blocks(d) + min(c0 + 32 * j % S::WR, d - 1) / F8_BLK) * g.nst;
    f8_f16 acc[NB][S::GM];
    tile_go<S, false, false>(g, tr.nrows, WS, XS, acc);
    float* out = shared ? a.f.shared_out : a.f.slot_out;
#pragma unroll
    for (int i = 0; i < NB; ++i) {
        const int r = 32 * (mh + S::GM * i) + l32;
        if (r >= tr.nrows) continue;
        int dst = tr.rbeg - a.f.T * a.f.k + r;
        float w = 1.0f;
        if (!shared) {
            dst = a.f.perm_rows[tr.rbeg + r];
            if (dst < 0 || dst >= a.f.T * a.f.k) continue;
            w = a.f.topk_w[dst];
        }
#pragma unroll
        for (int j = 0; j < S::GM; ++j)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int c = c0 + 32 * j + 8 * q + 4 * (lane >> 5);
                const f8_f16& p = acc[i][j];
                if (c < d)
                    st_stream16(out + (size_t)dst * d + c,
                                make_float4(w * p[4 * q], w * p[4 * q + 1], w * p[4 * q + 2], w * p[4 * q + 3]));
            }
    }
}

template <class S, int OF>
__global__ __launch_bounds__(64 * TW) void f8_dense_tile_kernel(BlockArgs a) {
    constexpr int NB = S::NB, BM = S::BM;
    F8_TILE_LDS(S);
    // consecutive workgroups go to the 8 XCDs in turn: give each a contiguous
    // range of the tiles, walked in groups of 4 weight tiles (gemm_dev.h)
    const int gx = gridDim.x, gy = gridDim.y, L = blockIdx.x + blockIdx.y * gx, N = gx * gy;
    const int xcd = L % N_XCD, loc = L / N_XCD, qn = N / N_XCD, rn = N % N_XCD;
    const int at = xcd < rn ? xcd * (qn + 1) + loc : rn * (qn + 1) + (xcd - rn) * qn + loc;
    const int grp = at / (gx * 4), rem = at % (gx * 4), gs = min(4, gy - grp * 4);
    const int m0 = rem / gs * BM, n0 = (grp * 4 + rem % gs) * TN, nrows = min(BM, a.m - m0);
    const int lane = lane_id(), wave = wave_index(), mh = wave / S::GN, wn = wave % S::GN, l32 = lane & 31;
    F8Tile<S> g;
    g.K = a.k;
    g.nst = f8_blocks(a.k);
#pragma unroll
    for (int q = 0; q < TWC; ++q) {
        const int sr = copy_row(q * TW + wave, lane);
        g.wch = copy_chunk(sr, lane);
        g.wsrc[q] = a.wq + (size_t)min(n0 + sr, a.n - 1) * a.k + g.wch;
    }
#pragma unroll
    for (int q = 0; q < S::XQ; ++q) {
        const int sr = copy_row(q * TW + wave, lane);
        g.xch = copy_chunk(sr, lane);
        g.xsrc[q] = a.xq + (size_t)(m0 + min(sr, nrows - 1)) * a.k + g.xch;
    }
#pragma unroll
    for (int i = 0; i < NB; ++i)
        g.ep[i] = a.xe + (size_t)(m0 + min(32 * (mh + S::GM * i) + l32, nrows - 1)) * f8_scale_ld(a.k);
    const int c0 = n0 + S::WR * wn;
#pragma unroll
    for (int j = 0; j < 2; ++j) g.sp[j] = a.ws + (size_t)(min(c0 + 32 * j % S::WR, a.n - 1) / F8_BLK) * g.nst;
    f8_f16 acc[NB][S::GM];
    tile_go<S, OF == MOE_DT_F32, false>(g, nrows, WS, XS, acc);
#pragma unroll
    for (int i = 0; i < NB; ++i) {
        const int r = 32 * (mh + S::GM * i) + l32;
        if (r >= nrows) continue;
#pragma unroll
        for (int j = 0; j < S::GM; ++j)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int c = c0 + 32 * j + 8 * q + 4 * (lane >> 5);
                if (c >= a.n) continue;
                const float v[4] = {acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]};
                f8_store4<OF>(a.out, (size_t)(m0 + r) * a.n + c, a.n - c, v, a.n % 4 == 0);
            }
    }
}

}  // namespace

hipError_t launch_f8_gateup(const F8Ffn& a, hipStream_t st, const KTime& kt) {
    const int fmax = a.f.n_shared && a.f.Fs > a.f.F ? a.f.Fs : a.f.F;
    const dim3 grid(a.f.max_tiles, f8_blocks(fmax));
    if (a.f.bm == 32) launch_kernel(f8_gateup_tile_kernel<Rows32>, grid, 64 * TW, st, kt, a);
    else if (a.f.bm == 64) launch_kernel(f8_gateup_tile_kernel<Rows64>, grid, 64 * TW, st, kt, a);
    else if (a.f.bm == 128) launch_kernel(f8_gateup_tile_kernel<Rows128>, grid, 64 * TW, st, kt, a);
    else launch_kernel(f8_gateup_tile_kernel<Rows256>, grid, 64 * TW, st, kt, a);
    return hipGetLastError();
}

hipError_t launch_f8_down(const F8Ffn& a, hipStream_t st, const KTime& kt) {
    const dim3 grid(a.f.max_tiles, (a.f.d + TN - 1) / TN);
    if (a.f.bm == 32) launch_kernel(f8_down_tile_kernel<Rows32>, grid, 64 * TW, st, kt, a);
    else if (a.f.bm == 64) launch_kernel(f8_down_tile_kernel<Rows64>, grid, 64 * TW, st, kt, a);
    else if (a.f.bm == 128) launch_kernel(f8_down_tile_kernel<Rows128>, grid, 64 * TW, st, kt, a);
    else launch_kernel(f8_down_tile_kernel<Rows256>, grid, 64 * TW, st, kt, a);
    return hipGetLastError();
}

hipError_t launch_block_matmul_tile(const BlockArgs& a, hipStream_t st) {
    const int nt = (a.n + TN - 1) / TN;
    if (a.odt == MOE_DT_F32) {
        f8_dense_tile_kernel<Rows128, MOE_DT_F32><<<dim3((a.m + 127) / 128, nt), 64 * TW, 0, st>>>(a);
    } else if ((long)((a.m + 255) / 256) * nt >= 192) {
        f8_dense_tile_kernel<Rows256, MOE_DT_BF16><<<dim3((a.m + 255) / 256, nt), 64 * TW, 0, st>>>(a);
    } else {
        f8_dense_tile_kernel<Rows128, MOE_DT_BF16><<<dim3((a.m + 127) / 128, nt), 64 * TW, 0, st>>>(a);
    }
    return hipGetLastError();
}

}  // namespace moe
