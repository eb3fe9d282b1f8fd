// i8_tile.hip - int8 products for many activation rows per weight matrix.
//
//   gate/up:  h[r, c] = silu(x_r Wg_c) (x_r Wu_c), fp32
//   down:     slot_out[f, :] = w_f (h_r Wd^T), h's rows quantised
//   dense:    out[m, n] = x_m W_n
//
// A workgroup computes a tile of activation rows x weight rows (gate/up: 128
// gate and the same 128 up rows), each wavefront blocks of 32 x 32 of it.  A stage
// is 128 columns of K: 128-byte rows, copied straight from global memory into
// LDS (eight whole cache lines per copy instruction, 16-byte chunks swizzled by
// row as dma_dev.h describes), in a ring of stages behind one barrier per
// stage.  The sums stay in int32 accumulators over the whole of K; the scales of
// rows and columns are applied once, behind the loop.
//
// A tile computes only the 32-row blocks that hold rows: blocks are dealt to the
// two wavefront rows in turn, and each wavefront runs the K loop built for its
// number of live blocks.
#include "common.h"
#include "i8_dev.h"
#include "tile_dev.h"

namespace moe {
namespace {

constexpr int TK = F8_BLK;  // columns of a stage

// Expert tiles (256 weight rows) and tiles of the dense product.
typedef Shape<1, 2, 2, 4, 2> Rows64;
typedef Shape<2, 2, 2, 4, 3> Rows128;
typedef Shape<4, 2, 2, 4, 2> Square256;
typedef Shape<2, 2, 2, 2, 2> Square128;
typedef Shape<1, 1, 2, 2, 4> Square64;

// Sources of one tile: wave-uniform buffers and 32-bit lane offsets.
template <class S>
struct I8Tile {
    const uint8_t *wbase, *xbase;  // weight rows (of gate or of up), activation rows
    uint32_t woff[S::WQ];          // the copy lane's bytes of weight copy q, at K = 0
    uint32_t xoff[S::XQ];
    int ch;                        // the copy lane's 16-byte chunk in a stage row, in bytes
    int K;
    bool once = false;             // no other tile reads these weights
};

// A wavefront's sums: rows of 16 activation rows (two in a block), 16 weight
// rows.  Lane l holds weight rows 4 (l / 16) + v of activation row l % 16.
template <class S>
struct I8Sums {
    i32x4_t v[2 * S::NB][2 * S::NJ];
};

// The K loop of one wavefront with L live blocks and XC activation copies per
// stage.
template <class S, int L, int XC, bool EXPERT>
__device__ __forceinline__ void tile_loop(I8Tile<S> g, uint8_t* const (&W)[S::NST], uint8_t* const (&X)[S::NST],
                                          I8Sums<S>& out) {
    constexpr int NST = S::NST, NB = S::NB, NJ = S::NJ, TW = S::W, TWC = S::WQ, NC = TWC + XC;
    const int wave = wave_index(), mh = wave / S::GN, wn = wave % S::GN;
    const int lane = lane_id();
    uint32_t ro[2];  // this lane's 16 bytes of 16 rows of a stage, of its first and second 64 columns
#pragma unroll
    for (int h = 0; h < 2; ++h) ro[h] = (lane & 15) * TK + (((4 * h + (lane >> 4)) ^ pair_swz(lane & 15)) << 4);
    g.wbase = uniform_ptr(g.wbase);
    g.xbase = uniform_ptr(g.xbase);
    const int nfull = g.K / TK, last = nfull - 1;  // whole stages
    // (opaque: single registers, not parts of vectors or of 64-bit values)
#pragma unroll
    for (int q = 0; q < TWC; ++q) __asm__ volatile("" : "+v"(g.woff[q]));
#pragma unroll
    for (int q = 0; q < XC; ++q) __asm__ volatile("" : "+v"(g.xoff[q]));
    const __amdgpu_buffer_rsrc_t wr = tile_buffer(g.wbase), xr = tile_buffer(g.xbase);
    // expert weights that no other tile reads are copied non-temporal
    const bool once = EXPERT && NB == 1 && __builtin_amdgcn_readfirstlane(g.once);
    // (stages past the end re-read the last; not multiplied)
    auto issue_at = [&](auto ss, int kb) {
        uint8_t *w = W[decltype(ss)::value % NST], *x = X[decltype(ss)::value % NST];
        auto copies = [&](auto nt) {
#pragma unroll
            for (int q = 0; q < TWC; ++q)
                buffer_copy16<decltype(nt)::value != 0>(wr, g.woff[q], min(kb, last) * TK, w + (q * TW + wave) * 1024);
        };
        if (once) copies(ic<1>());
        else copies(ic<0>());
#pragma unroll
        for (int q = 0; q < XC; ++q) buffer_copy16(xr, g.xoff[q], min(kb, last) * TK, x + (q * TW + wave) * 1024);
    };
    I8Sums<S> acc;
    each<4 * NB * NJ>([&](auto b) { acc.v[decltype(b)::value / (2 * NJ)][decltype(b)::value % (2 * NJ)] = i32x4_t{0, 0, 0, 0}; });
    // A stage is NR reads of 16 activation rows, those of its first 64 columns
    // and those of its second; each is multiplied with the wavefront's weight
    // rows while the XR reads behind it are on their way, across the stages' ends.
    constexpr int NR = 4 * L, XR = L > 1 ? 4 : 2;
    i32x4_t w[2][2 * NJ], x[XR];
    // (opaque: addresses formed from them are not kept over the loop)
    auto at = [&](auto hh, int rows) {
        uint32_t o = rows * TK;
        __asm__ volatile("" : "+s"(o));
        return ro[decltype(hh)::value] + o;
    };
    auto read_w = [&](auto nn, auto hh) {
        constexpr int B = decltype(nn)::value % NST, h = decltype(hh)::value;
        const uint32_t o = at(hh, S::WR * wn);
        each<2 * NJ>([&](auto jj) {
            w[h][decltype(jj)::value] = *reinterpret_cast<const i32x4_t*>(W[B] + 16 * decltype(jj)::value * TK + o);
        });
    };
    auto read_x = [&](auto nn, auto rr) {  // (r >= NR: of the next stage)
        constexpr int r = decltype(rr)::value, B = (decltype(nn)::value + r / NR) % NST, h = r % NR / (2 * L), b = r % (2 * L);
        x[r % XR] = *reinterpret_cast<const i32x4_t*>(X[B] + (32 * S::GM * (b / 2) + 16 * (b % 2)) * TK + at(ic<h>(), 32 * mh));
    };
    auto multiply = [&](auto rr) {
        constexpr int r = decltype(rr)::value, h = r / (2 * L), b = r % (2 * L);
        each<2 * NJ>([&](auto jj) {
            constexpr int j = decltype(jj)::value;
            acc.v[b][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(w[h][j], x[r % XR], acc.v[b][j], 0, 0, 0);
        });
    };
    // Stage kb; the first weights and the first XR reads of it are on their way.
    auto stage = [&](auto nn, int kb) {
        constexpr int n = decltype(nn)::value;
        if constexpr (L == 0) {
            wait_vm<(NST - 2) * NC>();
            barrier_nofence();
            issue_at(nn, kb + NST);
        } else {
            each<NR>([&](auto rr) {
                constexpr int r = decltype(rr)::value;
                if constexpr (r == 0) read_w(nn, ic<1>());
                if constexpr (r + XR == NR) {
                    // everything this wavefront reads of the stage is in registers: handed over
                    wait_lgkm0();
                    wait_vm<(NST - 2) * NC>();  // stage kb + 1 has landed
                    barrier_nofence();
                    issue_at(nn, kb + NST);
                    if constexpr (NR / 2 + XR <= NR) read_w(ic<n + 1>(), ic<0>());
                }
                multiply(rr);
                read_x(nn, ic<r + XR>());
                pin();
            });
        }
    };
    if (nfull > 0) {
        each<NST>([&](auto ss) { issue_at(ss, decltype(ss)::value); });
        wait_vm<(NST - 1) * NC>();
        barrier_nofence();
        if constexpr (L > 0) {
            read_w(ic<0>(), ic<0>());
            each<XR>([&](auto rr) { read_x(ic<0>(), rr); });
        }
        for (int kb = 0; kb < nfull; kb += NST) {
            each<NST>([&](auto nn) {
                if (kb + decltype(nn)::value < nfull) stage(nn, kb + decltype(nn)::value);
            });
        }
    }
    if (g.K > nfull * TK) {  // the step that K ends in: columns past K come from a row of zeros
        wait_vm<0>();
        wait_lgkm0();
        barrier_nofence();  // every stage has landed and been read
        const bool in = g.ch < g.K - nfull * TK;
        const uint8_t* zero = reinterpret_cast<const uint8_t*>(f8_zeros);
        // (opaque: or the 64-bit forms of the offsets would be kept over the loop)
        auto from = [&](const uint8_t* base, uint32_t off) {
            __asm__ volatile("" : "+v"(off));
            return in ? base + nfull * TK + off : zero;
        };
#pragma unroll
        for (int q = 0; q < TWC; ++q) copy16(from(g.wbase, g.woff[q]), W[0] + (q * TW + wave) * 1024);
#pragma unroll
        for (int q = 0; q < XC; ++q) copy16(from(g.xbase, g.xoff[q]), X[0] + (q * TW + wave) * 1024);
        wait_vm<0>();
        barrier_nofence();
        if constexpr (L > 0) {
            read_w(ic<0>(), ic<0>());
            read_w(ic<0>(), ic<1>());
            each<NR>([&](auto rr) {
                read_x(ic<0>(), rr);
                multiply(rr);
            });
        }
    }
    wait_vm<0>();  // no copy may still be writing LDS when the workgroup ends
    out = acc;
}

// Runs the loop built for this wavefront's live blocks (rows of the tile: nrows).
template <class S, bool EXPERT>
__device__ __forceinline__ void tile_run(const I8Tile<S>& g, int nrows, uint8_t* const (&W)[S::NST],
                                         uint8_t* const (&X)[S::NST], I8Sums<S>& acc) {
    const int wave = wave_index(), nblk = (nrows + 31) / 32, live = (nblk - wave / S::GN + S::GM - 1) / S::GM;
    auto run = [&](auto l, auto xc) { tile_loop<S, decltype(l)::value, decltype(xc)::value, EXPERT>(g, W, X, acc); };
    static_assert(S::GM == 2, "two wavefronts along the activation rows");
    constexpr int RB = S::W / 4;  // a round of activation copies covers W / 4 blocks
    if constexpr (S::NB == 4) {
        static_assert(RB == 2, "eight wavefronts");
        if (nblk > 6) return live == 4 ? run(ic<4>(), ic<4>()) : run(ic<3>(), ic<4>());
        if (nblk > 4) return live == 3 ? run(ic<3>(), ic<3>()) : run(ic<2>(), ic<3>());
    }
    if constexpr (S::NB >= 2) {
        if (nblk > 2) return live == 2 ? run(ic<2>(), ic<4 / RB>()) : run(ic<1>(), ic<4 / RB>());
    }
    return live == 1 ? run(ic<1>(), ic<2 / RB>()) : run(ic<0>(), ic<2 / RB>());
}

template <class S, bool EXPERT>
__device__ __forceinline__ void tile_go(const I8Tile<S>& g, int nrows, uint8_t* const (&WS)[4], uint8_t* const (&XS)[4],
                                        I8Sums<S>& acc) {
    ring<S::NST>(WS, [&](auto& W) { ring<S::NST>(XS, [&](auto& X) { tile_run<S, EXPERT>(g, nrows, W, X, acc); }); });
}

// Sums as fp32 with the activation row's scale sx and the lane's weight rows' sw.
__device__ __forceinline__ f8_f4 scaled(const i32x4_t& p, float sx, const f8_f4& sw) {
    f8_f4 r;
#pragma unroll
    for (int v = 0; v < 4; ++v) r[v] = (float)p[v] * sx * sw[v];
    return r;
}
// Scales of weight rows c .. c + 3 of n (rows past the last repeat it).
__device__ __forceinline__ f8_f4 tile_scales(const float* s, int c, int n) {
    if (c + 4 <= n) return i8_scales4(s + c);
    f8_f4 r;
#pragma unroll
    for (int v = 0; v < 4; ++v) r[v] = s[min(c + v, n - 1)];
    return r;
}
// Results of 16 x 16 to the wavefront's region (tile_dev.h), rows 16 i .. of its
// 32, columns 16 j .. of its 32 fp32 or 64 bf16.
__device__ __forceinline__ void put_f32(uint8_t* R, int lane, int i, int j, const f8_f4& p) {
    *reinterpret_cast<f8_f4*>(R + out_chunk(16 * i + (lane & 15), 4 * j + (lane >> 4))) = p;
}
__device__ __forceinline__ void put_bf16(uint8_t* R, int lane, int i, int j, const f8_f4& p) {
    *reinterpret_cast<uint2*>(R + out_chunk(16 * i + (lane & 15), 2 * j + (lane >> 5)) + 8 * ((lane >> 4) & 1)) =
        make_uint2(f32_to_bf16(p[0]) | (uint32_t)f32_to_bf16(p[1]) << 16, f32_to_bf16(p[2]) | (uint32_t)f32_to_bf16(p[3]) << 16);
}

template <class S>
__global__ __launch_bounds__(64 * S::W, S::WAVES) void i8_gateup_tile_kernel(I8Ffn a) {
    constexpr int NB = S::NB, BM = S::BM, HC = S::WR / 2, TW = S::W, TWC = S::WQ;  // h columns per wavefront
    F8_TILE_LDS(S);
    int tile, ntile;
    if (!work_item<4>(tile_count(a.f), tile, ntile)) return;
    TileRows tr;
    if (!tile_rows<BM>(a.f, tile, tr)) return;
    const bool shared = tr.g == a.f.E;
    const int F = shared ? a.f.Fs : a.f.F, d = a.f.d, n0 = ntile * (S::TN / 2);
    if (n0 >= F) return;
    const int lane = lane_id(), wave = wave_index(), mh = wave / S::GN, wn = wave % S::GN;
    const MatRef& G = shared ? a.f.s_gate : a.f.gate;
    const MatRef& U = shared ? a.f.s_up : a.f.up;
    const size_t e = shared ? 0 : tr.g;
    I8Tile<S> g;
    g.K = d;
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
    g.xbase = reinterpret_cast<const uint8_t*>(a.xq);  // (T * d is below 2^32)
#pragma unroll
    for (int q = 0; q < S::XQ; ++q) g.xoff[q] = (uint32_t)token(copy_row(q * TW + wave, lane)) * d + g.ch;
    g.once = one_tile<BM>(a.f, tr);
    I8Sums<S> acc;
    tile_go<S, true>(g, tr.nrows, WS, XS, acc);
    static_assert(S::NJ == 2 && HC == 32, "a block of gate, a block of up");
    __syncthreads();  // every wavefront has read its last stage
    const int c0 = n0 + HC * wn;
    if (c0 >= F) return;  // (F is a multiple of 64)
    uint8_t* R = out_region<S>(WS, wave);
    f8_f4 sg[2], su[2];  // (the wavefront's first two rows of 16 are gate, the others the same rows of up)
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        sg[j] = tile_scales(reinterpret_cast<const float*>(G.scale) + e * F, c0 + 16 * j + 4 * (lane >> 4), F);
        su[j] = tile_scales(reinterpret_cast<const float*>(U.scale) + e * F, c0 + 16 * j + 4 * (lane >> 4), F);
    }
    each<NB>([&](auto ii) {
        constexpr int i = decltype(ii)::value;
        const int r0 = 32 * (mh + S::GM * i), rows = tr.nrows - r0;
        if (rows <= 0) return;
        each<2>([&](auto bb) {
            constexpr int b = decltype(bb)::value;
            const float sx = a.xs[token(r0 + 16 * b + (lane & 15))];
            each<2>([&](auto jj) {
                constexpr int j = decltype(jj)::value;
                const f8_f4 ga = scaled(acc.v[2 * i + b][j], sx, sg[j]), up = scaled(acc.v[2 * i + b][2 + j], sx, su[j]);
                f8_f4 h;
#pragma unroll
                for (int v = 0; v < 4; ++v) h[v] = silu_f32(ga[v]) * up[v];
                put_f32(R, lane, b, j, h);
            });
        });
        out_fence();
        out_rows<float, f8_u4, 128>(R, lane, a.h + (size_t)(tr.rbeg + r0) * a.f.ldh + c0, a.f.ldh, rows, HC);
        out_fence();
    });
}

template <class S>
__global__ __launch_bounds__(64 * S::W, S::WAVES) void i8_down_tile_kernel(I8Ffn a) {
    constexpr int NB = S::NB, BM = S::BM, TN = S::TN, TW = S::W, TWC = S::WQ;
    F8_TILE_LDS(S);
    int tile, ntile;
    if (!work_item<4>(tile_count(a.f), tile, ntile)) return;
    TileRows tr;
    if (!tile_rows<BM>(a.f, tile, tr)) return;
    const bool shared = tr.g == a.f.E;
    const int F = shared ? a.f.Fs : a.f.F, d = a.f.d, n0 = ntile * TN;
    const int lane = lane_id(), wave = wave_index(), mh = wave / S::GN, wn = wave % S::GN;
    const MatRef& D = shared ? a.f.s_down : a.f.down;
    const size_t e = shared ? 0 : tr.g;
    I8Tile<S> g;
    g.K = F;
#pragma unroll
    for (int q = 0; q < TWC; ++q) {
        const int sr = copy_row(q * TW + wave, lane);
        g.ch = copy_chunk(sr, lane);
        g.woff[q] = (uint32_t)(min(sr, d - 1 - n0) * F + g.ch);
    }
    g.once = one_tile<BM>(a.f, tr);
    g.wbase = static_cast<const uint8_t*>(D.q) + (e * d + n0) * F;
    g.xbase = reinterpret_cast<const uint8_t*>(a.hq) + (size_t)tr.rbeg * a.f.ldh;
#pragma unroll
    for (int q = 0; q < S::XQ; ++q) {
        const int sr = copy_row(q * TW + wave, lane);
        g.xoff[q] = (uint32_t)((sr < tr.nrows ? sr : 0) * a.f.ldh + g.ch);
    }
    I8Sums<S> acc;
    tile_go<S, true>(g, tr.nrows, WS, XS, acc);
    float* out = shared ? a.f.shared_out : a.f.slot_out;
    __syncthreads();  // every wavefront has read its last stage
    uint8_t* R = out_region<S>(WS, wave);
    int ln = lane;  // (opaque: nothing formed from it is kept over the loop)
    __asm__ volatile("" : "+v"(ln));
    const int c0 = n0 + S::WR * wn;
    if (c0 >= d) return;  // (d is a multiple of 64)
    f8_f4 sw[2 * S::NJ];
#pragma unroll
    for (int j = 0; j < 2 * S::NJ; ++j)
        sw[j] = tile_scales(reinterpret_cast<const float*>(D.scale) + e * d, c0 + 16 * j + 4 * (ln >> 4), d);
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
        float w[2], sx[2];
#pragma unroll
        for (int b = 0; b < 2; ++b) {
            const int fb = __shfl(f, 16 * b + (ln & 15));
            w[b] = shared ? 1.0f : fb < 0 ? 0.0f : a.f.topk_w[fb];
            sx[b] = a.hs[tr.rbeg + min(r0 + 16 * b + (ln & 15), tr.nrows - 1)];
        }
        each<S::NJ>([&](auto jj) {
            constexpr int j = decltype(jj)::value;
            each<4>([&](auto qq) {
                constexpr int b = decltype(qq)::value / 2, q = decltype(qq)::value % 2;
                put_f32(R, ln, b, q, scaled(acc.v[2 * i + b][2 * j + q], sx[b], sw[2 * j + q]) * w[b]);
            });
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
__global__ __launch_bounds__(64 * S::W) void i8_dense_tile_kernel(ChannelArgs a) {
    constexpr int NB = S::NB, BM = S::BM, TN = S::TN, TW = S::W, TWC = S::WQ;
    F8_TILE_LDS(S);
    // consecutive workgroups go to the 8 XCDs in turn: give each a contiguous
    // range of the tiles, walked in groups of 4 weight tiles (gemm_dev.h)
    const int gx = gridDim.x, gy = gridDim.y, L = blockIdx.x + blockIdx.y * gx, N = gx * gy;
    const int xcd = L % N_XCD, loc = L / N_XCD, qn = N / N_XCD, rn = N % N_XCD;
    const int at = xcd < rn ? xcd * (qn + 1) + loc : rn * (qn + 1) + (xcd - rn) * qn + loc;
    const int grp = at / (gx * 4), rem = at % (gx * 4), gs = min(4, gy - grp * 4);
    const int m0 = rem / gs * BM, n0 = (grp * 4 + rem % gs) * TN, nrows = min(BM, a.m - m0);
    const int lane = lane_id(), wave = wave_index(), mh = wave / S::GN, wn = wave % S::GN;
    I8Tile<S> g;
    g.K = a.k;
#pragma unroll
    for (int q = 0; q < TWC; ++q) {
        const int sr = copy_row(q * TW + wave, lane);
        g.ch = copy_chunk(sr, lane);
        g.woff[q] = (uint32_t)(min(sr, a.n - 1 - n0) * a.k + g.ch);
    }
    g.wbase = reinterpret_cast<const uint8_t*>(a.wq) + (size_t)n0 * a.k;
    g.xbase = static_cast<const uint8_t*>(a.x) + (size_t)m0 * a.k;
#pragma unroll
    for (int q = 0; q < S::XQ; ++q) g.xoff[q] = (uint32_t)(min(copy_row(q * TW + wave, lane), nrows - 1) * a.k + g.ch);
    I8Sums<S> acc;
    tile_go<S, false>(g, nrows, WS, XS, acc);
    __syncthreads();  // every wavefront has read its last stage
    uint8_t* R = out_region<S>(WS, wave);
    const int c0 = n0 + S::WR * wn;
    if (c0 >= a.n) return;
    f8_f4 sw[2 * S::NJ];
#pragma unroll
    for (int j = 0; j < 2 * S::NJ; ++j) sw[j] = tile_scales(a.ws, c0 + 16 * j + 4 * (lane >> 4), a.n);
    each<NB>([&](auto ii) {
        constexpr int i = decltype(ii)::value;
        const int r0 = 32 * (mh + S::GM * i), rows = nrows - r0;
        if (rows <= 0) return;
        float sx[2];
#pragma unroll
        for (int b = 0; b < 2; ++b) sx[b] = a.xs[m0 + r0 + min(16 * b + (lane & 15), rows - 1)];
        const size_t at = (size_t)(m0 + r0) * a.n + c0;
        if constexpr (OF == MOE_DT_BF16) {
            each<4 * S::NJ>([&](auto qq) {
                constexpr int b = decltype(qq)::value / (2 * S::NJ), j = decltype(qq)::value % (2 * S::NJ);
                put_bf16(R, lane, b, j, scaled(acc.v[2 * i + b][j], sx[b], sw[j]));
            });
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
                each<4>([&](auto qq) {
                    constexpr int b = decltype(qq)::value / 2, q = decltype(qq)::value % 2;
                    put_f32(R, lane, b, q, scaled(acc.v[2 * i + b][2 * j + q], sx[b], sw[2 * j + q]));
                });
                out_fence();
                float* out = static_cast<float*>(a.out) + at + 32 * j;
                if (a.n % 4 == 0) out_rows<float, f8_u4, 128>(R, lane, out, a.n, rows, a.n - c0 - 32 * j);
                else out_rows<float, uint32_t, 128>(R, lane, out, a.n, rows, a.n - c0 - 32 * j);
                out_fence();
            });
        }
    });
}

template <class S>
void dense_launch(const ChannelArgs& a, hipStream_t st) {
    const dim3 grid((a.m + S::BM - 1) / S::BM, (a.n + S::TN - 1) / S::TN);
    if (a.odt == MOE_DT_F32) i8_dense_tile_kernel<S, MOE_DT_F32><<<grid, 64 * S::W, 0, st>>>(a);
    else i8_dense_tile_kernel<S, MOE_DT_BF16><<<grid, 64 * S::W, 0, st>>>(a);
}

}  // namespace

hipError_t launch_i8_gateup(const I8Ffn& a, hipStream_t st, const KTime& kt) {
    const int fmax = a.f.n_shared && a.f.Fs > a.f.F ? a.f.Fs : a.f.F;
    const dim3 grid(a.f.max_tiles, (fmax + Rows64::TN / 2 - 1) / (Rows64::TN / 2));
    if (a.f.bm == 64) launch_kernel(i8_gateup_tile_kernel<Rows64>, grid, 64 * Rows64::W, st, kt, a);
    else launch_kernel(i8_gateup_tile_kernel<Rows128>, grid, 64 * Rows128::W, st, kt, a);
    return hipGetLastError();
}

hipError_t launch_i8_down(const I8Ffn& a, hipStream_t st, const KTime& kt) {
    static_assert(Rows64::TN == Rows128::TN, "one grid");
    const dim3 grid(a.f.max_tiles, (a.f.d + Rows64::TN - 1) / Rows64::TN);
    if (a.f.bm == 64) launch_kernel(i8_down_tile_kernel<Rows64>, grid, 64 * Rows64::W, st, kt, a);
    else launch_kernel(i8_down_tile_kernel<Rows128>, grid, 64 * Rows128::W, st, kt, a);
    return hipGetLastError();
}

// The largest tiles that still give most compute units one.
hipError_t launch_channel_matmul_tile(const ChannelArgs& a, hipStream_t st) {
    auto tiles = [&](int bm, int tn) { return (long)((a.m + bm - 1) / bm) * ((a.n + tn - 1) / tn); };
    if (tiles(256, 256) >= 192) dense_launch<Square256>(a, st);
    else if (tiles(128, 128) >= 192) dense_launch<Square128>(a, st);
    else dense_launch<Square64>(a, st);
    return hipGetLastError();
}

}  // namespace moe
