// f8_tile.hip - e4m3 products for many activation rows per weight matrix.
//
//   gate/up:  h[r, c] = silu(x_r Wg_c) (x_r Wu_c), quantised per 128 columns
//   down:     slot_out[f, :] = w_f (h_r Wd^T)
//   dense:    out[m, n] = x_m W_n
//
// A workgroup computes a tile of activation rows x weight rows (gate/up: 128
// gate and the same 128 up rows, so that a tile holds whole scale blocks of h),
// each wavefront blocks of 32 x 32 of it.  A stage is one step of 128 columns,
// the width of a scale block: 128-byte rows, copied straight from global
// memory into LDS (eight whole cache lines per copy instruction, 16-byte
// chunks swizzled by row as dma_dev.h describes), in a ring of stages behind
// one barrier per stage.  A block's sum over the stage starts from zero on the
// matrix cores and is added with the weight block's fp32 scale, uniform over
// the block (one FMA per lane's result, an SGPR operand).  The activation rows'
// e8m0 scales are applied by the 8-bit instruction itself, or (WIDE) as the rows
// are widened or after the sum.
//
// WIDE: the codes are widened to bf16 and the sums are fp32 (f8_dev.h): every
// product of the layers, and the dense one to fp32.  In 64-row tiles the weight
// bytes set the pace and it costs nothing (8 tokens: gate/up 117 us, down 63 with
// either instruction); at 128 rows per expert it costs 0.7 + 0.4 ms of 2.7.  The
// dense product to bf16 takes the 8-bit instruction, twice the rate.
//
// A tile computes only the 32-row blocks that hold rows: blocks are dealt to the
// two wavefront rows in turn, and each wavefront runs the K loop built for its
// number of live blocks.
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
// Expert tiles (256 weight rows, the two scale blocks of a 128-column h block).
// Up to 64 activation rows: two workgroups per compute unit, each with two
// stages, so that one's start and end lie under the other's loop (gate/up of
// 512 tokens, 16 rows per expert: 1.00 ms, 6.6 TB/s of weights; one workgroup
// with four stages took 1.35 ms when this took 1.06).  More: 128 rows, whose
// widened operands (64 registers of weights) fit beside the accumulators (128 rows
// per expert: gate/up 2.29 ms and down 1.34; 256-row tiles, which widen half a
// stage at a time, 2.64 and 1.62; two stages, or four of weights, in place of
// three: within 2%).
typedef Shape<1, 2, 2, 4, 2> Rows64;
typedef Shape<2, 2, 2, 4, 3> Rows128;  // also of the dense product to fp32
// Tiles of the dense product: its weights are shared by every row tile, so one
// stage ahead is enough (weights two stages ahead: 4096 x 4096 x 6144 3% longer);
// smaller ones for sizes that would leave compute units idle, and for fp32
// results (whose widened operands do not fit beside the accumulators of the largest).
typedef Shape<4, 2, 2, 4, 2> Square256;
typedef Shape<2, 2, 2, 2, 2> Square128;
typedef Shape<1, 1, 2, 2, 4> Square64;

// Sources of one tile: wave-uniform buffers and 32-bit lane offsets (64-bit lane
// pointers of the largest shape did not fit the register file, and a buffer load
// adds the step's offset without a vector instruction).
template <class S>
struct F8Tile {
    const uint8_t *wbase, *xbase, *ebase;  // weight rows (of gate or of up), activation rows, scale bytes
    uint32_t woff[S::WQ];         // the copy lane's bytes of weight copy q, at K = 0
    uint32_t xoff[S::XQ];
    uint32_t eoff[S::NB];         // scale bytes of the lane's activation row in each block
    int ch;                       // the copy lane's 16-byte chunk in a stage row, in bytes
    const float* sp[2];           // block scales of the wavefront's weight rows (gate/up: of gate, of up)
    int K, nst;
    bool once = false;            // no other tile reads these weights
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

// 32 codes of a lane's row: columns 64 h + 32 (lane / 32) .. + 31 of the stage.
struct F8Row {
    f8_u4 a, b;
};
// Byte offsets of those chunks from the first row of a block of 32 rows (the
// swizzle repeats every 16 rows, so they serve every block).
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
__device__ __forceinline__ F8Row tile_row(const uint8_t* S, const F8Lane& f, uint32_t block, int h) {
    return F8Row{*reinterpret_cast<const f8_u4*>(S + (f.o[2 * h] + block)),
                 *reinterpret_cast<const f8_u4*>(S + (f.o[2 * h + 1] + block))};
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

// The K loop of one wavefront with L live blocks and XC activation copies per
// stage; acc[i][j]: block i (activation rows) x weight row block j.
template <class S, int L, int XC, bool WIDE, bool EXPERT>
__device__ __forceinline__ void tile_loop(F8Tile<S> g, uint8_t* const (&W)[S::NST], uint8_t* const (&X)[S::NST],
                                          f8_f16 (&out)[S::NB][S::NJ]) {
    constexpr int NST = S::NST, NB = S::NB, NJ = S::NJ, TW = S::W, TWC = S::WQ;
    const int wave = wave_index(), mh = wave / S::GN, wn = wave % S::GN;
    const F8Lane fl = tile_lane(lane_id());
    constexpr int NC = TWC + XC;
    g.wbase = uniform_ptr(g.wbase);
    g.xbase = uniform_ptr(g.xbase);
    g.ebase = uniform_ptr(g.ebase);
    g.sp[0] = uniform_ptr(g.sp[0]);
    g.sp[1] = uniform_ptr(g.sp[1]);
    const int nfull = g.K / F8_BLK, last = nfull - 1;  // whole stages
    // (opaque: single registers, not parts of vectors or of 64-bit values)
#pragma unroll
    for (int q = 0; q < TWC; ++q) __asm__ volatile("" : "+v"(g.woff[q]));
#pragma unroll
    for (int q = 0; q < XC; ++q) __asm__ volatile("" : "+v"(g.xoff[q]));
#pragma unroll
    for (int i = 0; i < L; ++i) __asm__ volatile("" : "+v"(g.eoff[i]));
    const __amdgpu_buffer_rsrc_t wr = tile_buffer(g.wbase), xr = tile_buffer(g.xbase), er = tile_buffer(g.ebase);
    // (stages past the end re-read the last; not used)
    // Expert weights that no other tile reads, as g.once says, are copied
    // non-temporal (16 rows per expert: gate/up 1.08 ms, so 1.00, down 0.64 / 0.61;
    // all copies so, 64 rows per expert, many in two tiles: 1.33 / 1.55 ms; in the
    // larger tiles, 128 rows per expert, gate/up 2.56 so, 2.48 plain).
    const bool once = EXPERT && NB == 1 && __builtin_amdgcn_readfirstlane(g.once);
    auto issue_at = [&](auto ss, int kb) {
        uint8_t *w = W[decltype(ss)::value % NST], *x = X[decltype(ss)::value % NST];
        auto copies = [&](auto nt) {
#pragma unroll
            for (int q = 0; q < TWC; ++q)
                buffer_copy16<decltype(nt)::value != 0>(wr, g.woff[q], min(kb, last) * F8_BLK, w + (q * TW + wave) * 1024);
        };
        if (once) copies(ic<1>());
        else copies(ic<0>());
#pragma unroll
        for (int q = 0; q < XC; ++q) buffer_copy16(xr, g.xoff[q], min(kb, last) * F8_BLK, x + (q * TW + wave) * 1024);
    };
    // what stage n (at step kb) sends for
    auto issue = [&](auto nn, int kb) { issue_at(ic<decltype(nn)::value + NST - 1>(), kb + NST - 1); };
    uint32_t ev[NB], en[NB];
#pragma unroll
    for (int i = 0; i < L; ++i) en[i] = __builtin_amdgcn_raw_buffer_load_b32(er, (int)g.eoff[i], 0, 0);
    if (nfull > 0) {
        each<NST - 1>([&](auto ss) { issue_at(ss, decltype(ss)::value); });
    }
    // Weight scales of the WIDE loop: at the top of a round lane l holds those of
    // the round's stage l.  (Scalar loads count with the LDS reads, out of order,
    // and every partial wait for LDS data became a full one.)
    float sl[2], sn[2];
    auto scales = [&](int kb) {
#pragma unroll
        for (int j = 0; j < 2; ++j) sn[j] = g.sp[j][min(kb + lane_id(), g.nst - 1)];
    };
    if constexpr (WIDE) scales(0);
    f8_f16 acc[NB][NJ];
    each<NB * NJ>([&](auto b) { acc[decltype(b)::value / NJ][decltype(b)::value % NJ] = f8_f16{}; });
    // WIDE: the products of LDS stage B; byte SEL of ev scales the activation
    // rows, lane LN of sl the weight rows
    auto products_wide = [&](auto nn, auto ll) {
        constexpr int n = decltype(nn)::value, B = n % NST, SEL = n % 4, LN = decltype(ll)::value;
        const float s0 = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(sl[0]), LN));
        const float s1 = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(sl[1]), LN));
        // (opaque: addresses formed from them are not kept over the loop, where
        // they would take registers the accumulators need)
        uint32_t wo = S::WR * wn * F8_BLK, xo = 32 * mh * F8_BLK;
        __asm__ volatile("" : "+s"(wo), "+s"(xo));
        if constexpr (NB == 1 && NJ > 1) {
            // two workgroups per compute unit leave 128 registers: a half row at
            // a time, the activation rows read and widened for each weight block
            each<NJ>([&](auto jj) {
                constexpr int j = decltype(jj)::value;
                f8_f16 p = f8_f16{};
                each<2>([&](auto hh) {
                    constexpr int h = decltype(hh)::value;
                    const F8Row w = tile_row(W[B] + 32 * j * F8_BLK, fl, wo, h), x = tile_row(X[B], fl, xo, h);
                    p = f8_dot32(f8_widen(w.a, w.b), f8_widen(x.a, x.b), p);
                    pin();
                });
                const float a = (j > 0 ? s1 : s0);
                const f8_f16 s = f8_f16{a, a, a, a, a, a, a, a, a, a, a, a, a, a, a, a};
                acc[0][j] = __builtin_elementwise_fma(s, p * f8_scale_value((ev[0] >> (8 * SEL)) & 255u), acc[0][j]);
            });
            wait_lgkm0();
            return;
        }
        F8Row w[NJ][2];
        each<NJ>([&](auto jj) {
            constexpr int j = decltype(jj)::value;
            w[j][0] = tile_row(W[B] + 32 * j * F8_BLK, fl, wo, 0);
            w[j][1] = tile_row(W[B] + 32 * j * F8_BLK, fl, wo, 1);
        });
        F8Wide ww[NJ][2];
        each<NJ * 2>([&](auto q) {
            constexpr int j = decltype(q)::value / 2, h = decltype(q)::value % 2;
            ww[j][h] = f8_widen(w[j][h].a, w[j][h].b);
        });
        each<L>([&](auto ii) {
            constexpr int i = decltype(ii)::value;
            const F8Row x0 = tile_row(X[B] + 32 * S::GM * i * F8_BLK, fl, xo, 0);
            const F8Row x1 = tile_row(X[B] + 32 * S::GM * i * F8_BLK, fl, xo, 1);
            // The layers' row scales multiply the widened codes: exact, as those are
            // quantised finite fp32 values (but for parts below 2^-133), and one
            // operation per result less (128 rows per expert: gate/up 2.29 ms, 2.48
            // with the scale after the sum).  The dense product's scales are the
            // caller's: any scale whose product with the sum is in range is right.
            const float sx = f8_scale_value((ev[i] >> (8 * SEL)) & 255u), before = EXPERT ? sx : 1.0f;
            const F8Wide v0 = f8_widen(x0.a, x0.b, before), v1 = f8_widen(x1.a, x1.b, before);
            each<NJ>([&](auto jj) {
                constexpr int j = decltype(jj)::value;
                f8_f16 p = f8_dot32(ww[j][1], v1, f8_dot32(ww[j][0], v0, f8_f16{}));
                if constexpr (!EXPERT) p = p * sx;
                // (whole-vector operations: accumulators written element by
                // element in a loop went to scratch memory)
                const float a = j > 0 ? s1 : s0;
                const f8_f16 s = f8_f16{a, a, a, a, a, a, a, a, a, a, a, a, a, a, a, a};
                acc[i][j] = __builtin_elementwise_fma(s, p, acc[i][j]);
            });
        });
        wait_lgkm0();  // this stage's reads are done before the next barrier releases its refill
    };
    // The 8-bit products, in a fixed order: a block's products are issued before
    // the FMAs of the block before it, which then run beside the matrix unit; the
    // last block of a stage waits for the first products of the next; the copies
    // go out behind the first products.  (Left to the compiler the sums of
    // several blocks are in flight at once; in the largest shape, whose registers
    // are all taken, offsets were then reloaded from scratch memory behind the
    // copies: 4096 x 4096 x 6144 took a quarter longer.  The smaller shapes gain
    // little: 300 x 4096 x 6144 in 64 x 64 tiles 2%.)
    f8_f16 pend = f8_f16{};
    float q0 = 0.0f, q1 = 0.0f, t0 = 0.0f, t1 = 0.0f;  // scales of the block that waits, of the next stage
    if constexpr (!WIDE) {
        t0 = f8_uniform(g.sp[0], 0);
        t1 = f8_uniform(g.sp[1], 0);
    }
    auto retire = [&](auto bb, float s0, float s1) {  // block b = i NJ + j
        constexpr int i = decltype(bb)::value / NJ, j = decltype(bb)::value % NJ;
        const float a = j > 0 ? s1 : s0;
        const f8_f16 s = f8_f16{a, a, a, a, a, a, a, a, a, a, a, a, a, a, a, a};
        acc[i][j] = __builtin_elementwise_fma(s, pend, acc[i][j]);
    };
    auto products = [&](auto nn, auto more, int kb) {
        constexpr int n = decltype(nn)::value, B = n % NST, SEL = n % 4;
        constexpr bool MORE = decltype(more)::value != 0;  // a stage of the loop, which sends for a later one
        uint32_t wo = S::WR * wn * F8_BLK, xo = 32 * mh * F8_BLK;
        __asm__ volatile("" : "+s"(wo), "+s"(xo));
        F8Row w[NJ][2], x[2];
        each<2>([&](auto hh) {  // in the order of use
            constexpr int h = decltype(hh)::value;
            w[0][h] = tile_row(W[B], fl, wo, h);
            x[h] = tile_row(X[B], fl, xo, h);
        });
        each<2 * (NJ - 1)>([&](auto q) {
            constexpr int j = 1 + decltype(q)::value / 2, h = decltype(q)::value % 2;
            w[j][h] = tile_row(W[B] + 32 * j * F8_BLK, fl, wo, h);
        });
        if constexpr (MORE && SEL == 0) {
#pragma unroll
            for (int i = 0; i < L; ++i) ev[i] = en[i];
        }
        const float s0 = t0, s1 = t1;
        each<L * NJ>([&](auto b2) {
            constexpr int b = decltype(b2)::value, i = b / NJ, j = b % NJ;
            f8_f16 p = f8_mfma32<SEL>(f8_join(w[j][0].a, w[j][0].b), f8_join(x[0].a, x[0].b), f8_f16{}, ev[i]);
            p = f8_mfma32<SEL>(f8_join(w[j][1].a, w[j][1].b), f8_join(x[1].a, x[1].b), p, ev[i]);
            pin();
            if constexpr (j == NJ - 1 && i + 1 < L) {  // the next activation block's rows
                x[0] = tile_row(X[B] + 32 * S::GM * (i + 1) * F8_BLK, fl, xo, 0);
                x[1] = tile_row(X[B] + 32 * S::GM * (i + 1) * F8_BLK, fl, xo, 1);
            }
            if constexpr (b == 0) {
                if constexpr (MORE) issue(nn, kb);
                retire(ic<(L > 0 ? L * NJ - 1 : 0)>(), q0, q1);
                if constexpr (MORE) {
                    t0 = f8_uniform(g.sp[0], min(kb + 1, g.nst - 1));
                    t1 = f8_uniform(g.sp[1], min(kb + 1, g.nst - 1));
                    if constexpr (SEL == 0) {
#pragma unroll
                        for (int t = 0; t < L; ++t)
                            en[t] = __builtin_amdgcn_raw_buffer_load_b32(er, (int)g.eoff[t], kb + 4 < g.nst ? kb + 4 : 0, 0);
                    }
                }
            } else {
                retire(ic<(b > 0 ? b - 1 : 0)>(), s0, s1);
            }
            pin();
            pend = p;
        });
        q0 = s0;
        q1 = s1;
        wait_lgkm0();
    };
    auto stage = [&](auto nn, int kb) {
        constexpr int n = decltype(nn)::value, SEL = n % 4;
        // all but the copies sent after this stage's last
        wait_vm<(NST - 2) * NC>();
        barrier_nofence();
        if constexpr (!WIDE && L > 0) {
            products(nn, ic<1>(), kb);
        } else {
            issue(nn, kb);
            if constexpr (SEL == 0) {
#pragma unroll
                for (int i = 0; i < L; ++i) {
                    ev[i] = en[i];
                    en[i] = __builtin_amdgcn_raw_buffer_load_b32(er, (int)g.eoff[i], kb + 4 < g.nst ? kb + 4 : 0, 0);
                }
            }
            if constexpr (L > 0) products_wide(nn, nn);
        }
    };
    // twelve (four) stages run through every pair of LDS stage and scale byte
    constexpr int CYC = NST == 3 ? 12 : 4;
    for (int kb = 0; kb < nfull; kb += CYC) {
        if constexpr (WIDE) {
            sl[0] = sn[0];
            sl[1] = sn[1];
            scales(kb + CYC);
        }
#define F8_STAGE(n) \
    if constexpr (n < CYC) { if (kb + n < nfull) stage(ic<n>(), kb + n); }
        F8_STAGE(0) F8_STAGE(1) F8_STAGE(2) F8_STAGE(3) F8_STAGE(4) F8_STAGE(5)
        F8_STAGE(6) F8_STAGE(7) F8_STAGE(8) F8_STAGE(9) F8_STAGE(10) F8_STAGE(11)
#undef F8_STAGE
    }
    if (g.nst > nfull) {  // the step that K ends in: columns past K come from a row of zeros
        wait_vm<0>();
        barrier_nofence();  // every stage has landed and been read
        const bool in = g.ch < g.K - nfull * F8_BLK;
        const uint8_t* zero = reinterpret_cast<const uint8_t*>(f8_zeros);
        // (opaque: or the 64-bit forms of the offsets would be kept over the loop)
        auto from = [&](const uint8_t* base, uint32_t off) {
            __asm__ volatile("" : "+v"(off));
            return in ? base + nfull * F8_BLK + off : zero;
        };
#pragma unroll
        for (int q = 0; q < TWC; ++q) copy16(from(g.wbase, g.woff[q]), W[0] + (q * TW + wave) * 1024);
#pragma unroll
        for (int q = 0; q < XC; ++q) copy16(from(g.xbase, g.xoff[q]), X[0] + (q * TW + wave) * 1024);
#pragma unroll
        for (int i = 0; i < L; ++i) ev[i] = __builtin_amdgcn_raw_buffer_load_b8(er, (int)g.eoff[i], nfull, 0);
        wait_vm<0>();
        barrier_nofence();
        if constexpr (!WIDE && L > 0) {
            products(ic<0>(), ic<0>(), nfull);
        } else if constexpr (L > 0) {
            sl[0] = g.sp[0][nfull];
            sl[1] = g.sp[1][nfull];
            products_wide(ic<0>(), ic<0>());
        }
    }
    if constexpr (!WIDE && L > 0) retire(ic<(L > 0 ? L * NJ - 1 : 0)>(), q0, q1);
    wait_vm<0>();  // no copy may still be writing LDS when the workgroup ends
    each<NB * NJ>([&](auto b) {
        constexpr int i = decltype(b)::value / NJ, j = decltype(b)::value % NJ;
        out[i][j] = acc[i][j];
    });
}

// Runs the loop built for this wavefront's live blocks (rows of the tile: nrows).
template <class S, bool WIDE, bool EXPERT>
__device__ __forceinline__ void tile_run(const F8Tile<S>& g, int nrows, uint8_t* const (&W)[S::NST],
                                         uint8_t* const (&X)[S::NST], f8_f16 (&acc)[S::NB][S::NJ]) {
    const int wave = wave_index(), nblk = (nrows + 31) / 32, live = (nblk - wave / S::GN + S::GM - 1) / S::GM;
    auto run = [&](auto l, auto xc) { tile_loop<S, decltype(l)::value, decltype(xc)::value, WIDE, EXPERT>(g, W, X, acc); };
    static_assert(S::GM == 2, "two wavefronts along the activation rows");
    {  // a round of activation copies covers W / 4 blocks
        constexpr int RB = S::W / 4;
        if constexpr (S::NB == 4) {
            static_assert(RB == 2 && S::GM == 2, "eight wavefronts");
            if (nblk > 6) return live == 4 ? run(ic<4>(), ic<4>()) : run(ic<3>(), ic<4>());
            if (nblk > 4) return live == 3 ? run(ic<3>(), ic<3>()) : run(ic<2>(), ic<3>());
        }
        if constexpr (S::NB >= 2) {
            if (nblk > 2) return live == 2 ? run(ic<2>(), ic<4 / RB>()) : run(ic<1>(), ic<4 / RB>());
        }
        return live == 1 ? run(ic<1>(), ic<2 / RB>()) : run(ic<0>(), ic<2 / RB>());
    }
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

template <class S, bool WIDE, bool EXPERT>
__device__ __forceinline__ void tile_go(const F8Tile<S>& g, int nrows, uint8_t* const (&WS)[4], uint8_t* const (&XS)[4],
                                        f8_f16 (&acc)[S::NB][S::NJ]) {
    ring<S::NST>(WS, [&](auto& W) { ring<S::NST>(XS, [&](auto& X) { tile_run<S, WIDE, EXPERT>(g, nrows, W, X, acc); }); });
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

template <class S>
__global__ __launch_bounds__(64 * S::W, S::WAVES) void f8_gateup_tile_kernel(F8Ffn a) {
    constexpr int NB = S::NB, BM = S::BM, HC = S::WR / 2, TW = S::W, TWC = S::WQ;  // h columns per wavefront
    F8_TILE_LDS(S);
    // per-row maxima of the wavefronts, over the first activation stage once the K loop is done
    static_assert(S::GN * S::BM * 4 <= S::XB, "room for the maxima");
    uint32_t(*red)[BM] = reinterpret_cast<uint32_t(*)[BM]>(X0);
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
    // stage rows 2 HC m .. + HC - 1: gate rows n0 + HC m .., the HC rows after
    // them: the same up rows (a wavefront's copies are 64 rows apart: all of
    // them gate, or all up)
    static_assert(64 % (2 * HC) == 0 && TW == 8, "gate and up copies");
    g.wbase = static_cast<const uint8_t*>((8 * wave & HC) ? U.q : G.q) + (e * F + n0) * d;
#pragma unroll
    for (int q = 0; q < TWC; ++q) {
        const int r8 = 8 * (q * TW + wave), n = HC * (r8 / (2 * HC)) + r8 % HC + (lane >> 3);
        g.ch = copy_chunk(r8 + (lane >> 3), lane);
        g.woff[q] = (uint32_t)(min(n, F - 1 - n0) * d + g.ch);
    }
    auto token = [&](int r) {  // rows past the tile repeat its first; their results are not stored
        r = r < tr.nrows ? r : 0;
        if (shared) return tr.rbeg - a.f.T * a.f.k + r;
        const int f = a.f.perm_rows[tr.rbeg + r];
        return f >= 0 && f < a.f.T * a.f.k ? f / a.f.k : 0;
    };
    g.xbase = a.xq;  // (T * d is below 2^32)
    g.ebase = a.xe;
#pragma unroll
    for (int q = 0; q < S::XQ; ++q) g.xoff[q] = (uint32_t)token(copy_row(q * TW + wave, lane)) * d + g.ch;
#pragma unroll
    for (int i = 0; i < NB; ++i) g.eoff[i] = (uint32_t)token(32 * (mh + S::GM * i) + l32) * f8_scale_ld(d);
    g.once = one_tile<BM>(a.f, tr);
    const size_t srow = (e * f8_blocks(F) + ntile) * g.nst;
    g.sp[0] = reinterpret_cast<const float*>(G.scale) + srow;
    g.sp[1] = reinterpret_cast<const float*>(U.scale) + srow;
    f8_f16 acc[NB][S::NJ];
    tile_go<S, true, true>(g, tr.nrows, WS, XS, acc);
    // h and its largest magnitude per row over the tile's 128 columns
    // (a wavefront has gate and up in its two blocks)
    static_assert(S::NJ == 2 && HC == 32, "a block of gate, a block of up");
    constexpr int NV = 16;  // h values per lane
    const int c0 = n0 + HC * wn;
    const bool in = c0 < F;  // (F is a multiple of 64)
    __syncthreads();  // every wavefront has read its last stage
    each<NB>([&](auto ii) {  // h takes the place of gate in acc[i][0]
        constexpr int i = decltype(ii)::value;
        const f8_f16 ga = acc[i][0], up = acc[i][1];
        f8_f16 h = ga;
        uint32_t m = 0;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            h[v] = silu_f32(ga[v]) * up[v];
            m = max(m, f8_abs_bits(h[v]));
        }
        acc[i][0] = h;
        m = max(m, (uint32_t)__shfl_xor((int)m, 32));
        if (lane < 32) red[wn][32 * (mh + S::GM * i) + l32] = in ? m : 0u;
    });
    __syncthreads();
    const int hi = lane >> 5;
    each<NB>([&](auto ii) {
        constexpr int i = decltype(ii)::value;
        const f8_f16 h = acc[i][0];
        const int r = 32 * (mh + S::GM * i) + l32;
        uint32_t m = 0;
#pragma unroll
        for (int w = 0; w < S::GN; ++w) m = max(m, red[w][r]);
        const uint32_t byte = f8_scale_byte(m);
        const float inv = f8_inv_scale(byte);
        uint32_t c[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
            c[j] = f8_pack4(h[4 * j], h[4 * j + 1], h[4 * j + 2], h[4 * j + 3], inv, byte);
        // lanes l and l + 32 hold alternate 4-column runs of a row: each takes 16 adjacent columns
        uint32_t o[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) o[j] = (uint32_t)__shfl_xor((int)(hi ? c[j] : c[j + 2]), 32);
        if (r >= tr.nrows) return;
        const size_t hrow = (size_t)(tr.rbeg + r);
        if (in)
            *reinterpret_cast<uint4*>(a.hq + hrow * a.f.ldh + c0 + 16 * hi) =
                hi ? make_uint4(o[0], c[2], o[1], c[3]) : make_uint4(c[0], o[0], c[1], o[1]);
        if (wn == 0 && hi == 0) a.he[hrow * f8_scale_ld(a.f.ldh) + ntile] = (uint8_t)byte;
    });
}

template <class S>
__global__ __launch_bounds__(64 * S::W, S::WAVES) void f8_down_tile_kernel(F8Ffn a) {
    constexpr int NB = S::NB, BM = S::BM, TN = S::TN, TW = S::W, TWC = S::WQ;
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
        g.ch = copy_chunk(sr, lane);
        g.woff[q] = (uint32_t)(min(sr, d - 1 - n0) * F + g.ch);
    }
    g.once = one_tile<BM>(a.f, tr);
    g.wbase = static_cast<const uint8_t*>(D.q) + (e * d + n0) * F;
    g.xbase = a.hq + (size_t)tr.rbeg * a.f.ldh;
    g.ebase = a.he + (size_t)tr.rbeg * f8_scale_ld(a.f.ldh);
#pragma unroll
    for (int q = 0; q < S::XQ; ++q) {
        const int sr = copy_row(q * TW + wave, lane);
        g.xoff[q] = (uint32_t)((sr < tr.nrows ? sr : 0) * a.f.ldh + g.ch);
    }
#pragma unroll
    for (int i = 0; i < NB; ++i) {
        const int r = 32 * (mh + S::GM * i) + l32;
        g.eoff[i] = (uint32_t)((r < tr.nrows ? r : 0) * f8_scale_ld(a.f.ldh));
    }
    const int c0 = n0 + S::WR * wn;
#pragma unroll
    for (int j = 0; j < 2; ++j)  // (one block: both the same)
        g.sp[j] = reinterpret_cast<const float*>(D.scale) + (e * f8_blocks(d) + min(c0 + 32 * j % S::WR, d - 1) / F8_BLK) * g.nst;
    f8_f16 acc[NB][S::NJ];
    tile_go<S, true, true>(g, tr.nrows, WS, XS, acc);
    float* out = shared ? a.f.shared_out : a.f.slot_out;
    __syncthreads();  // every wavefront has read its last stage
    uint8_t* R = out_region<S>(WS, wave);
    int ln = lane;  // (opaque: nothing formed from it is kept over the loop)
    __asm__ volatile("" : "+v"(ln));
    auto slot = [&](int r) {  // the result row of tile row r, or -1
        if (r >= tr.nrows) return -1;
        if (shared) return tr.rbeg - a.f.T * a.f.k + r;
        const int f = a.f.perm_rows[tr.rbeg + r];
        return f >= 0 && f < a.f.T * a.f.k ? f : -1;
    };
    each<NB>([&](auto ii) {
        constexpr int i = decltype(ii)::value;
        const int r0 = 32 * (mh + S::GM * i);
        if (r0 >= tr.nrows) return;
        const int f = slot(r0 + (ln & 31));
        const float w = shared ? 1.0f : f < 0 ? 0.0f : a.f.topk_w[f];
        each<S::NJ>([&](auto jj) {
            constexpr int j = decltype(jj)::value;
            out_put_f32(R, ln, acc[i][j] * w);
            out_fence();
            const int c = c0 + 32 * j + 4 * (ln & 7);
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                const f8_f4 v = *reinterpret_cast<const f8_f4*>(R + out_chunk(8 * s + (ln >> 3), ln & 7));
                const int dst = __shfl(f, 8 * s + (ln >> 3));
                if (dst >= 0 && c < d) *reinterpret_cast<f8_f4*>(out + (size_t)dst * d + c) = v;
            }
            out_fence();
        });
    });
}

template <class S, int OF>
__global__ __launch_bounds__(64 * S::W) void f8_dense_tile_kernel(BlockArgs a) {
    constexpr int NB = S::NB, BM = S::BM, TN = S::TN, TW = S::W, TWC = S::WQ;
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
        g.ch = copy_chunk(sr, lane);
        g.woff[q] = (uint32_t)(min(sr, a.n - 1 - n0) * a.k + g.ch);
    }
    g.wbase = a.wq + (size_t)n0 * a.k;
    g.xbase = a.xq + (size_t)m0 * a.k;
    g.ebase = a.xe + (size_t)m0 * f8_scale_ld(a.k);
#pragma unroll
    for (int q = 0; q < S::XQ; ++q) g.xoff[q] = (uint32_t)(min(copy_row(q * TW + wave, lane), nrows - 1) * a.k + g.ch);
#pragma unroll
    for (int i = 0; i < NB; ++i)
        g.eoff[i] = (uint32_t)(min(32 * (mh + S::GM * i) + l32, nrows - 1) * f8_scale_ld(a.k));
    const int c0 = n0 + S::WR * wn;
#pragma unroll
    for (int j = 0; j < 2; ++j) g.sp[j] = a.ws + (size_t)(min(c0 + 32 * j % S::WR, a.n - 1) / F8_BLK) * g.nst;
    f8_f16 acc[NB][S::NJ];
    tile_go<S, OF == MOE_DT_F32, false>(g, nrows, WS, XS, acc);
    __syncthreads();  // every wavefront has read its last stage
    uint8_t* R = out_region<S>(WS, wave);
    each<NB>([&](auto ii) {
        constexpr int i = decltype(ii)::value;
        const int r0 = 32 * (mh + S::GM * i), rows = nrows - r0;
        if (rows <= 0) return;
        const size_t at = (size_t)(m0 + r0) * a.n + c0;
        if constexpr (OF == MOE_DT_BF16) {
            each<S::NJ>([&](auto jj) { out_put_bf16(R, lane, decltype(jj)::value, acc[i][decltype(jj)::value]); });
            out_fence();
            uint16_t* out = static_cast<uint16_t*>(a.out) + at;
            constexpr int BYTES = 64 * S::NJ;
            if (a.n % 8 == 0) out_rows<uint16_t, f8_u4, BYTES>(R, lane, out, a.n, rows, a.n - c0);
            else if (a.n % 4 == 0) out_rows<uint16_t, uint2, BYTES>(R, lane, out, a.n, rows, a.n - c0);
            else if (a.n % 2 == 0) out_rows<uint16_t, uint32_t, BYTES>(R, lane, out, a.n, rows, a.n - c0);
            else out_rows<uint16_t, uint16_t, BYTES>(R, lane, out, a.n, rows, a.n - c0);
            out_fence();
        } else {
            each<S::NJ>([&](auto jj) {
                constexpr int j = decltype(jj)::value;
                out_put_f32(R, lane, acc[i][j]);
                out_fence();
                float* out = static_cast<float*>(a.out) + at + 32 * j;
                if (a.n % 4 == 0) out_rows<float, f8_u4, 128>(R, lane, out, a.n, rows, a.n - c0 - 32 * j);
                else out_rows<float, uint32_t, 128>(R, lane, out, a.n, rows, a.n - c0 - 32 * j);
                out_fence();
            });
        }
    });
}

}  // namespace

hipError_t launch_f8_gateup(const F8Ffn& a, hipStream_t st, const KTime& kt) {
    const int fmax = a.f.n_shared && a.f.Fs > a.f.F ? a.f.Fs : a.f.F;
    const dim3 grid(a.f.max_tiles, f8_blocks(fmax));
    if (a.f.bm == 64) launch_kernel(f8_gateup_tile_kernel<Rows64>, grid, 64 * Rows64::W, st, kt, a);
    else launch_kernel(f8_gateup_tile_kernel<Rows128>, grid, 64 * Rows128::W, st, kt, a);
    return hipGetLastError();
}

hipError_t launch_f8_down(const F8Ffn& a, hipStream_t st, const KTime& kt) {
    static_assert(Rows64::TN == Rows128::TN, "one grid");
    const dim3 grid(a.f.max_tiles, (a.f.d + Rows64::TN - 1) / Rows64::TN);
    if (a.f.bm == 64) launch_kernel(f8_down_tile_kernel<Rows64>, grid, 64 * Rows64::W, st, kt, a);
    else launch_kernel(f8_down_tile_kernel<Rows128>, grid, 64 * Rows128::W, st, kt, a);
    return hipGetLastError();
}

template <class S, int OF>
static void dense_tile_launch(const BlockArgs& a, hipStream_t st) {
    const dim3 grid((a.m + S::BM - 1) / S::BM, (a.n + S::TN - 1) / S::TN);
    f8_dense_tile_kernel<S, OF><<<grid, 64 * S::W, 0, st>>>(a);
}
template <class S>
static void dense_tile_launch_out(const BlockArgs& a, hipStream_t st) {
    if (a.odt == MOE_DT_F32) dense_tile_launch<S, MOE_DT_F32>(a, st);
    else dense_tile_launch<S, MOE_DT_BF16>(a, st);
}

// The largest tiles that still give most compute units one (us a call, 256 x 256
// / 128 x 128 / 64 x 64 tiles, bf16 results; n x k 4096 x 6144: 300 rows 77 / 40 /
// 25, 1000 rows 77 / 44 / 55, 4096 rows 95 / 124 / 192; 4096 x 2048: 2048 rows
// 34 / 26 / 39; 700 x 1024: 4096 rows 21.5 / 12.3 / 12.2).  fp32 results double
// the matrix work: 128 x 256 tiles pay from 256 of them (2048 rows of 4096 x
// 2048 39 against 48 us for 128 x 128).
hipError_t launch_block_matmul_tile(const BlockArgs& a, hipStream_t st) {
    auto tiles = [&](int bm, int tn) { return (long)((a.m + bm - 1) / bm) * ((a.n + tn - 1) / tn); };
    if (a.odt == MOE_DT_F32 && tiles(128, 256) >= 256) dense_tile_launch<Rows128, MOE_DT_F32>(a, st);
    else if (a.odt == MOE_DT_BF16 && tiles(256, 256) >= 192) dense_tile_launch<Square256, MOE_DT_BF16>(a, st);
    else if (tiles(128, 128) >= 192) dense_tile_launch_out<Square128>(a, st);
    else dense_tile_launch_out<Square64>(a, st);
    return hipGetLastError();
}

}  // namespace moe
