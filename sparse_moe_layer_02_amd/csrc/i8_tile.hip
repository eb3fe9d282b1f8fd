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
// Measured: 4096 x 4096 x 6144 83.0 us (2.5 POP/s; matrix cores); layers of d 6144, F
// 2048 and 256 experts: 512 tokens gate/up 1.09 and down 0.62 ms (weight bytes, 5.9
// and 5.2 TB/s), 4096 tokens 1.67 and 0.99.
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

// A tile's shape (tile_dev.h) with rings of NW stages of weights and NX of
// activation rows.
template <int NB_, int NJ_, int GM_, int GN_, int NW_, int NX_>
struct Rings : Shape<NB_, NJ_, GM_, GN_, 2> {
    typedef Shape<NB_, NJ_, GM_, GN_, 2> Base;
    static constexpr int NW = NW_, NX = NX_;
    static constexpr int LDS = NW * Base::WB + NX * Base::XB;
    static constexpr int WAVES = LDS <= 80 * 1024 && Base::W == 8 ? 4 : 2;  // per SIMD: two workgroups where LDS has room
    // Half of the wavefronts copy weights, half activation rows: a wavefront waits
    // for copies in the order it sent them, and the rings are of different lengths.
    static constexpr int CW = Base::W / 2;                       // copying wavefronts of a kind
    static constexpr int WQ = Base::WB / 1024 / CW, XQ = Base::XB / 1024 / CW;  // 1 KB copies of each, stage by stage
    static constexpr int Q = WQ > XQ ? WQ : XQ;
    static_assert(WQ * CW * 1024 == Base::WB && XQ * CW * 1024 == Base::XB, "whole copies");
};
// Expert tiles (256 weight rows): up to 64 rows, two workgroups per compute unit
// (16 rows per expert: gate/up 1.09 ms, 5.9 TB/s of weights); beyond, all of LDS in
// one.  The rows come through the L2 as slowly as the weights do (a tile's 786 KB of
// a 6144-column x beside 31 others' in 4 MB): gate/up of 4096 tokens, 128 rows per
// expert, stages of weights + of rows: 128-row tiles 4 + 2 2.03 ms, 3 + 3 1.70, 3 + 4
// 1.69; 256-row tiles 2 + 2 1.72, 3 + 2 1.71, 2 + 3 1.63.  (Weights straight from
// memory into registers, in the instruction's order, with rows alone in LDS: 1.65
// to 2.0 ms.  A load of 16 rows x 64 bytes moves 18 bytes a clock and compute unit
// from the L2, one of 8 rows x 128 bytes 60.)
typedef Rings<1, 2, 2, 4, 2, 2> Rows64;
typedef Rings<2, 2, 2, 4, 3, 4> Rows128;
typedef Rings<4, 2, 2, 4, 2, 3> Rows256;
// Tiles of the dense product: the largest; 128 x 128 with eight wavefronts and four
// stages, for a compute unit of its own, and with four and two, two to a unit; 64 x 64.
typedef Rings<4, 2, 2, 4, 2, 2> Square256;
typedef Rings<2, 1, 2, 4, 4, 4> Alone128;
typedef Rings<2, 2, 2, 2, 2, 2> Square128;
typedef Rings<1, 1, 2, 2, 4, 4> Square64;

// Sources of one tile: wave-uniform buffers and 32-bit lane offsets.
template <class S>
struct I8Tile {
    const uint8_t* base;     // rows of this wavefront's copies: weights (of gate or of up), or activations
    uint32_t off[S::Q];      // the copy lane's bytes of copy q, at K = 0
    int ch;                  // the copy lane's 16-byte chunk in a stage row, in bytes
    int K;
    bool once = false;       // no other tile reads these weights
};
// Whether this wavefront copies weights, and which row of a stage copy q's lane fills.
template <class S>
__device__ __forceinline__ bool copies_weights() { return wave_index() < S::CW; }
template <class S>
__device__ __forceinline__ int x_copy(int q) { return q * S::CW + wave_index() % S::CW; }
// Weights: copies c and c ^ 4 (32 rows apart: gate and up) are different wavefronts'.
template <class S>
__device__ __forceinline__ int w_copy(int q) {
    const int me = wave_index() % S::CW;
    if constexpr (S::CW != 4) return q * S::CW + me;
    const int g = 2 * q + (me & 1);
    return 8 * (g >> 2) + (g & 3) + 4 * (me >> 1);
}
template <class S>
__device__ __forceinline__ int stage_row(int q, int lane) {
    return copy_row(copies_weights<S>() ? w_copy<S>(q) : x_copy<S>(q), lane);
}

// A wavefront's sums: rows of 16 activation rows (two in a block), 16 weight
// rows.  Lane l holds weight rows 4 (l / 16) + v of activation row l % 16.
template <class S>
struct I8Sums {
    i32x4_t v[2 * S::NB][2 * S::NJ];
};

// The copies of the loop are written out: the compiler puts waits for copies it
// knows of before reads of LDS, and where paths or rounds of a ring meet it takes
// copies just sent for ones the read needs.  Here it sees none, every wait is the
// loop's own, and the rings need no names of their own for their stages.  (M0,
// where a copy finds its LDS address, is set with each.  The compiler reserves it, so
// that a clobber of it cannot be declared: nothing else in these kernels may use it,
// such as a builtin that copies to LDS; tests/test_i8_assembly.py looks.)
// 16 bytes per lane from src + off + k0 to LDS at dst (wave-uniform) + 16 lane.
template <bool NT>
__device__ __forceinline__ void send16(i32x4_t src, uint32_t off, int k0, uint32_t dst) {
    if constexpr (NT)
        __asm__ volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, %3 offen nt lds"
                         :
                         : "s"(dst), "v"(off), "s"(src), "s"(k0)
                         : "memory");
    else
        __asm__ volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds"
                         :
                         : "s"(dst), "v"(off), "s"(src), "s"(k0)
                         : "memory");
}
// The same from an address of the lane's own.
__device__ __forceinline__ void send16_from(const uint8_t* src, uint32_t dst) {
    __asm__ volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off" : : "s"(dst), "v"(src) : "memory");
}
__device__ __forceinline__ uint32_t lds_address(uint8_t* p) { return (uint32_t)reinterpret_cast<uintptr_t>((lds_void*)p); }

// The K loop of one wavefront with L live blocks and XC activation copies per
// stage; lds: the ring of weights, then the ring of activation rows.
template <class S, int L, int XC, bool EXPERT>
__device__ __forceinline__ void tile_loop(I8Tile<S> g, uint8_t* lds, I8Sums<S>& acc) {
    constexpr int NW = S::NW, NX = S::NX, NB = S::NB, NJ = S::NJ, WC = S::WQ, WB = S::WB, XB = S::XB;
    uint8_t *const W = lds, *const X = lds + NW * WB;
    const int wave = wave_index(), mh = wave / S::GN, wn = wave % S::GN, lane = lane_id();
    uint32_t ro[2];  // this lane's 16 bytes of 16 rows of a stage, of its first and second 64 columns
#pragma unroll
    for (int h = 0; h < 2; ++h) ro[h] = (lane & 15) * TK + (((4 * h + (lane >> 4)) ^ pair_swz(lane & 15)) << 4);
    const bool cw = copies_weights<S>();
    const int nfull = g.K / TK, last = nfull - 1;  // whole stages
    const uint64_t base = reinterpret_cast<uint64_t>(uniform_ptr(g.base));
    const i32x4_t src = {(int)(uint32_t)base, (int)(uint32_t)(base >> 32) & 0xFFFF, -1, 0x00020000};
    const uint32_t w0 = lds_address(W), x0 = lds_address(X);
    // expert weights that no other tile reads are copied non-temporal
    const bool once = EXPERT && NB == 1 && __builtin_amdgcn_readfirstlane(g.once);
    // (stages past the end re-read the last; not multiplied)
    auto send = [&](int kb, uint32_t ws, uint32_t xs) {  // stage kb's weights to W + ws, or its rows to X + xs
        const int k0 = min(kb, last) * TK;
        auto weights = [&](auto nt) {
#pragma unroll
            for (int q = 0; q < WC; ++q) send16<decltype(nt)::value != 0>(src, g.off[q], k0, w0 + ws + w_copy<S>(q) * 1024);
        };
        if (!cw) {
#pragma unroll
            for (int q = 0; q < XC; ++q) send16<false>(src, g.off[q], k0, x0 + xs + x_copy<S>(q) * 1024);
        } else if (once) {
            weights(ic<1>());
        } else {
            weights(ic<0>());
        }
    };
    each<4 * NB * NJ>([&](auto b) { acc.v[decltype(b)::value / (2 * NJ)][decltype(b)::value % (2 * NJ)] = i32x4_t{0, 0, 0, 0}; });
    // A stage is NR reads of 16 activation rows, those of its first 64 columns
    // and those of its second; each is multiplied with the wavefront's weight
    // rows while the XR reads behind it are on their way, across the stages' ends.
    constexpr int NR = 4 * L, XR = L > 1 ? 4 : 2;  // (L == 0: none)
    i32x4_t w[2][2 * NJ], x[XR];
    uint32_t ws = 0, xs = 0;  // the stage's places in the rings
    auto read_w = [&](auto hh) {
        constexpr int h = decltype(hh)::value;
        const uint8_t* p = W + (ro[h] + (ws + S::WR * wn * TK));
        each<2 * NJ>([&](auto jj) { w[h][decltype(jj)::value] = *reinterpret_cast<const i32x4_t*>(p + 16 * decltype(jj)::value * TK); });
    };
    auto read_x = [&](auto rr) {
        constexpr int r = decltype(rr)::value, h = r / (2 * L), b = r % (2 * L);
        x[r % XR] = *reinterpret_cast<const i32x4_t*>(X + (ro[h] + (xs + 32 * mh * TK)) + (32 * S::GM * (b / 2) + 16 * (b % 2)) * TK);
    };
    auto multiply = [&](auto rr) {
        constexpr int r = decltype(rr)::value, h = r / (2 * L), b = r % (2 * L);
        each<2 * NJ>([&](auto jj) {
            constexpr int j = decltype(jj)::value;
            acc.v[b][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(w[h][j], x[r % XR], acc.v[b][j], 0, 0, 0);
        });
    };
    // The products of a stage but the last XR, whose operands are on their way then.
    auto begin = [&] {
        each<(L > 0 ? NR - XR : 0)>([&](auto rr) {
            constexpr int r = decltype(rr)::value;
            if constexpr (r == 0) read_w(ic<1>());
            multiply(rr);
            read_x(ic<r + XR>());
            pin();
        });
    };
    auto end = [&](auto more) {
        if constexpr (L > 0) {
            if constexpr (decltype(more)::value != 0) read_w(ic<0>());
            each<XR>([&](auto rr) {
                multiply(ic<NR - XR + decltype(rr)::value>());
                if constexpr (decltype(more)::value != 0) read_x(rr);
                pin();
            });
        }
    };
    if (nfull > 0) {
        if (cw) {
#pragma unroll
            for (int s = 0; s < NW; ++s) send(s, s * WB, 0);
            wait_vm<(NW - 1) * WC>();
        } else {
#pragma unroll
            for (int s = 0; s < NX; ++s) send(s, 0, s * XB);
            wait_vm<(NX - 1) * XC>();
        }
        barrier_nofence();
        if constexpr (L > 0) {
            read_w(ic<0>());
            each<XR>([&](auto rr) { read_x(rr); });
        }
        begin();
        for (int kb = 1; kb < nfull; ++kb) {
            // From stage kb - 1 to stage kb: everything this wavefront reads of the first
            // is in registers, so its place is free; the last products of the one are
            // made while the first operands of the other are read.
            wait_lgkm0();
            if (cw) wait_vm<(NW - 2) * WC>();
            else wait_vm<(NX - 2) * XC>();
            barrier_nofence();
            send(kb - 1 + (cw ? NW : NX), ws, xs);
            ws = ws == (NW - 1) * WB ? 0 : ws + WB;
            xs = xs == (NX - 1) * XB ? 0 : xs + XB;
            end(ic<1>());
            begin();
        }
        end(ic<0>());
        wait_vm<0>();
        wait_lgkm0();
        barrier_nofence();  // every stage has landed and been read
    }
    if (g.K > nfull * TK) {  // the step that K ends in: columns past K come from a row of zeros
        ws = xs = 0;
        const bool in = g.ch < g.K - nfull * TK;
        const uint8_t* zero = reinterpret_cast<const uint8_t*>(f8_zeros);
        auto tail = [&](uint32_t to, auto count, auto copy) {
#pragma unroll
            for (int q = 0; q < decltype(count)::value; ++q) {
                uint32_t off = g.off[q];  // (opaque: or its 64-bit form would be kept over the loop)
                __asm__ volatile("" : "+v"(off));
                send16_from(in ? g.base + nfull * TK + off : zero, to + copy(q) * 1024);
            }
        };
        if (cw) tail(w0, ic<WC>(), [](int q) { return w_copy<S>(q); });
        else tail(x0, ic<XC>(), [](int q) { return x_copy<S>(q); });
        wait_vm<0>();
        barrier_nofence();
        if constexpr (L > 0) {
            read_w(ic<0>());
            read_w(ic<1>());
            each<NR>([&](auto rr) {
                read_x(rr);
                multiply(rr);
            });
        }
        wait_lgkm0();
        barrier_nofence();  // every wavefront has read its last stage: LDS is the results' now
    }
}

// Runs the loop built for this wavefront's live blocks (rows of the tile: nrows).
// No copy is on its way and no stage is read when it returns.
template <class S, bool EXPERT>
__device__ __forceinline__ void tile_go(const I8Tile<S>& g, int nrows, uint8_t* lds, I8Sums<S>& acc) {
    const int wave = wave_index(), nblk = (nrows + 31) / 32, live = (nblk - wave / S::GN + S::GM - 1) / S::GM;
    auto run = [&](auto l, auto xc) { tile_loop<S, decltype(l)::value, decltype(xc)::value, EXPERT>(g, lds, acc); };
    static_assert(S::GM == 2, "two wavefronts along the activation rows");
    constexpr int PB = 4 / S::CW;  // copies per wavefront and block of 32 rows
    static_assert(PB * S::CW == 4, "whole copies");
    if constexpr (S::NB == 4) {
        if (nblk > 6) return live == 4 ? run(ic<4>(), ic<8 * PB>()) : run(ic<3>(), ic<8 * PB>());
        if (nblk > 4) return live == 3 ? run(ic<3>(), ic<6 * PB>()) : run(ic<2>(), ic<6 * PB>());
    }
    if constexpr (S::NB >= 2) {
        if (nblk > 2) return live == 2 ? run(ic<2>(), ic<4 * PB>()) : run(ic<1>(), ic<4 * PB>());
    }
    return live == 1 ? run(ic<1>(), ic<2 * PB>()) : run(ic<0>(), ic<2 * PB>());
}

// A wavefront's region of LDS for its results (tile_dev.h).
template <class S>
__device__ __forceinline__ uint8_t* result_region(uint8_t* lds, int wave) {
    static_assert(S::W * OUT_REGION <= S::LDS, "room for every wavefront");
    return lds + wave * OUT_REGION;
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
    constexpr int NB = S::NB, BM = S::BM, HC = S::WR / 2;  // h columns per wavefront
    __shared__ __attribute__((aligned(1024))) uint8_t lds[S::LDS];
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
    static_assert(64 % (2 * HC) == 0 && HC == 32 && S::CW == 4, "gate and up copies");
    auto token = [&](int r) {  // rows past the tile repeat its first; their results are not stored
        r = r < tr.nrows ? r : 0;
        if (shared) return tr.rbeg - a.f.T * a.f.k + r;
        const int f = a.f.perm_rows[tr.rbeg + r];
        return f >= 0 && f < a.f.T * a.f.k ? f / a.f.k : 0;
    };
    // stage rows 2 HC m .. + HC - 1: gate rows n0 + HC m .., the HC rows after
    // them: the same up rows (a wavefront copies gate, or up)
    const bool cw = copies_weights<S>();
    g.base = !cw ? reinterpret_cast<const uint8_t*>(a.xq)  // (T * d is below 2^32)
                 : static_cast<const uint8_t*>(wave & 2 ? U.q : G.q) + (e * F + n0) * d;
#pragma unroll
    for (int q = 0; q < S::Q; ++q) {
        const int r = stage_row<S>(q, lane), n = HC * (r / (2 * HC)) + r % HC;
        g.ch = copy_chunk(r, lane);
        g.off[q] = (cw ? (uint32_t)(min(n, F - 1 - n0) * d) : (uint32_t)token(r) * d) + g.ch;
    }
    g.once = one_tile<BM>(a.f, tr);
    I8Sums<S> acc;
    tile_go<S, true>(g, tr.nrows, lds, acc);
    static_assert(S::NJ == 2 && HC == 32, "a block of gate, a block of up");
    const int c0 = n0 + HC * wn;
    if (c0 >= F) return;  // (F is a multiple of 64)
    uint8_t* R = result_region<S>(lds, wave);
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
    constexpr int NB = S::NB, BM = S::BM, TN = S::TN;
    __shared__ __attribute__((aligned(1024))) uint8_t lds[S::LDS];
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
    g.once = one_tile<BM>(a.f, tr);
    const bool cw = copies_weights<S>();
    g.base = cw ? static_cast<const uint8_t*>(D.q) + (e * d + n0) * F
                : reinterpret_cast<const uint8_t*>(a.hq) + (size_t)tr.rbeg * a.f.ldh;
#pragma unroll
    for (int q = 0; q < S::Q; ++q) {
        const int r = stage_row<S>(q, lane);
        g.ch = copy_chunk(r, lane);
        g.off[q] = (uint32_t)((cw ? min(r, d - 1 - n0) * F : (r < tr.nrows ? r : 0) * a.f.ldh) + g.ch);
    }
    I8Sums<S> acc;
    tile_go<S, true>(g, tr.nrows, lds, acc);
    float* out = shared ? a.f.shared_out : a.f.slot_out;
    uint8_t* R = result_region<S>(lds, wave);
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
    constexpr int NB = S::NB, BM = S::BM, TN = S::TN;
    __shared__ __attribute__((aligned(1024))) uint8_t lds[S::LDS];
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
    const bool cw = copies_weights<S>();
    g.base = cw ? reinterpret_cast<const uint8_t*>(a.wq) + (size_t)n0 * a.k : static_cast<const uint8_t*>(a.x) + (size_t)m0 * a.k;
#pragma unroll
    for (int q = 0; q < S::Q; ++q) {
        const int r = stage_row<S>(q, lane);
        g.ch = copy_chunk(r, lane);
        g.off[q] = (uint32_t)(min(r, cw ? a.n - 1 - n0 : nrows - 1) * a.k + g.ch);
    }
    I8Sums<S> acc;
    tile_go<S, false>(g, nrows, lds, acc);
    uint8_t* R = result_region<S>(lds, wave);
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
    else if (a.f.bm == 128) launch_kernel(i8_gateup_tile_kernel<Rows128>, grid, 64 * Rows128::W, st, kt, a);
    else launch_kernel(i8_gateup_tile_kernel<Rows256>, grid, 64 * Rows256::W, st, kt, a);
    return hipGetLastError();
}

hipError_t launch_i8_down(const I8Ffn& a, hipStream_t st, const KTime& kt) {
    static_assert(Rows64::TN == Rows128::TN && Rows64::TN == Rows256::TN, "one grid");
    const dim3 grid(a.f.max_tiles, (a.f.d + Rows64::TN - 1) / Rows64::TN);
    if (a.f.bm == 64) launch_kernel(i8_down_tile_kernel<Rows64>, grid, 64 * Rows64::W, st, kt, a);
    else if (a.f.bm == 128) launch_kernel(i8_down_tile_kernel<Rows128>, grid, 64 * Rows128::W, st, kt, a);
    else launch_kernel(i8_down_tile_kernel<Rows256>, grid, 64 * Rows256::W, st, kt, a);
    return hipGetLastError();
}

// By how the tiles fill 256 compute units (us a call with cold weights, bf16
// results, n x k; tiles of 256 x 256 / 128 x 256 / 128 x 128 alone / two to a unit / 64
// x 64): from 192 of the largest those (2048 rows of 6144 x 2048: 36 / 43 / 43 / 42 /
// 56; 128 of them, 2048 of 4096 x 6144: 76 / 59 / 68 / 64 / 95); from 192 of 128 x 256 and
// not over one for each unit those (the same; 1024 of 6144 x 2048: 34 / 23.5 / 27 / 24 /
// 33); 160 to 256 of 128 x 128 one to a unit (1024 of 4096 x 6144: 76 / 50 / 36 / 55 / 56;
// 512 of 6144 x 2048: 33 / 22 / 16 / 22 / 20), more of them two to a unit (2048 of 4096 x
// 512: 19 / 14 / 15 / 13.6 / 19), fewer as 64 x 64 (256 of 4096 x 6144: 79 / 50 / 35 / 55 /
// 19; 77 of 6144 x 2048: 21 / 20 / 13 / 20 / 8.5).
hipError_t launch_channel_matmul_tile(const ChannelArgs& a, hipStream_t st) {
    auto tiles = [&](int bm, int tn) { return (long)((a.m + bm - 1) / bm) * ((a.n + tn - 1) / tn); };
    const long wide = tiles(128, 256), square = tiles(128, 128);
    if (tiles(256, 256) >= 192) dense_launch<Square256>(a, st);
    else if (wide >= 192 && wide <= 256) dense_launch<Rows128>(a, st);
    else if (square > 256) dense_launch<Square128>(a, st);
    else if (square >= 160) dense_launch<Alone128>(a, st);
    else dense_launch<Square64>(a, st);
    return hipGetLastError();
}

}  // namespace moe
