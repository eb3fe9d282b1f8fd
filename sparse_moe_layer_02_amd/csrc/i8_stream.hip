// i8_stream.hip - int8 products for few activation rows.
//
//   dense:    out[m, n] = x_m W_n
//   gate/up:  h[r, c] = silu(x_r Wg_c) (x_r Wu_c), fp32
//   down:     y[t] = shared row + sum_j w_j (h_j Wd^T), with the combine
//
// Bound by the weight bytes, each read once, and at these sizes by latency.
// The weights go from memory straight into the registers of the wavefront that
// uses them, in the order the matrix instruction takes them, so neither LDS nor a
// barrier stands between HBM and the multiply.  A step is 64 columns of K: lane l
// holds columns 16 (l / 16) .. + 15 of weight row l % 16 and of activation row
// l % 16, and the 16 x 16 x 64 instruction adds their products in int32.  Sums
// are exact, so K is split as the sizes suggest; the partial sums meet in LDS.
// Rows that no expert has repeat the last one; their results are not stored.
//
// d 4096, F 2048, top-6 and the shared expert, other experts' weights in each call
// (medians): one token gate/up 25.0 us (4.7 TB/s of weights) and down 14.8 (4.0; the same
// weights again, from the memory-side cache: 23.0 and 13.7), 16 tokens with 80 experts
// 225 (6.1) and 114 (6.0).
//
// Column tails: a load past the end of K re-reads the row's last 16 columns, and
// the activation operand is zero there.
#include "common.h"
#include "dma_dev.h"
#include "gemm_dev.h"
#include "i8_dev.h"
#include "kernels.h"

namespace moe {
namespace {

constexpr int SW = 8;  // wavefronts per workgroup
constexpr int SK = 64; // columns of a step
// Steps loaded at once.  A wavefront's share of K is a multiple of them: with 8 at
// once and 12 for a wavefront the loads past its end, repeats of its last step,
// cost more than they hid (weights in the memory-side cache, 1 x 4096 x 6144: 9.7 us,
// 7.3 so; non-temporal loads 7.9; two groups ahead in place of one 8.1; 24576 x 6144: 30
// us, 5.0 TB/s.  Weights in memory, 1 x 4096 x 6144: 9.1 us).
constexpr int UU = 4;
constexpr int I8_FUSE_VALUES = 24 * 1024;  // values a workgroup quantises itself, at most (their codes lie in LDS)

__device__ __forceinline__ i32x4_t ld_codes(const int8_t* p) { return *reinterpret_cast<const i32x4_t*>(p); }
__device__ __forceinline__ i32x4_t dot16(i32x4_t w, i32x4_t x, i32x4_t c) {
    return __builtin_amdgcn_mfma_i32_16x16x64_i8(w, x, c, 0, 0, 0);
}

// The products of steps [s0, s1) of NR blocks of 16 weight rows and NT of 16
// activation rows.  wp: this lane's weight rows; x(t, c): columns c .. c + 15 of its
// activation row, from memory, or (LX) from LDS.  The first weights are sent for
// before between(), behind which x may be called.  U steps are in flight while the
// U before them are multiplied.
template <int NR, int NT, int U, bool LX>
struct Frag {
    i32x4_t w[U][NR], x[LX ? 1 : U][NT];
};
template <int NR, int NT, int U, bool LX, class X, class Between>
__device__ __forceinline__ void stream(const int8_t* const (&wp)[NR], X x, int s0, int s1, int K,
                                       i32x4_t (&acc)[NR][NT], Between between) {
    typedef Frag<NR, NT, U, LX> F;
    const int lo = 16 * (lane_id() / 16);
    auto column = [&](int s) { return min(SK * min(s, s1 - 1) + lo, K - 16); };
    auto load_w = [&](F& f, int s) {
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int r = 0; r < NR; ++r) f.w[u][r] = ld_codes(wp[r] + column(s + u));
    };
    auto load_x = [&](F& f, int s) {
        if constexpr (!LX) {
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int t = 0; t < NT; ++t) f.x[u][t] = x(t, column(s + u));
        }
        pin();
    };
    auto load = [&](F& f, int s) {
        load_w(f, s);
        load_x(f, s);
    };
    auto compute = [&](const F& f, int s) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (s + u >= s1) break;
            const int c = SK * (s + u) + lo;
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                i32x4_t v;
                if constexpr (LX) v = x(t, min(c, K - 16));
                else v = f.x[u][t];
                if (c >= K) v = i32x4_t{0, 0, 0, 0};
#pragma unroll
                for (int r = 0; r < NR; ++r) acc[r][t] = dot16(f.w[u][r], v, acc[r][t]);
            }
        }
    };
    F a, b;
    if (s0 < s1) load_w(a, s0);
    pin();
    between();
    if (s0 < s1) load_x(a, s0);
    for (int s = s0; s < s1; s += 2 * U) {
        if (s + U < s1) load(b, s + U);
        compute(a, s);
        if (s + U < s1) {
            if (s + 2 * U < s1) load(a, s + 2 * U);
            compute(b, s + U);
        }
    }
}

// Rows of fp32 or bf16 as codes in LDS by the whole workgroup (few rows: every
// workgroup doing it costs less than a launch that does it first).  The
// wavefronts share a row while there are fewer than SW.  top: a word per row.
template <int XF>
__device__ __forceinline__ void rows_to_lds(const void* x, int rows, int cols, size_t ldx, int8_t* codes, int ldq,
                                            uint32_t* top, float* scales) {
    const int lane = lane_id(), wave = wave_index();
    int wpr = SW;  // wavefronts per row
    while (wpr > 1 && wpr * rows > SW) wpr >>= 1;
    const int part = wave % wpr, first = wave / wpr, step = SW / wpr;
    constexpr int KEEP = 2;  // groups of 8 columns that stay in registers
    float v[KEEP][8];
    if ((int)threadIdx.x < rows) top[threadIdx.x] = 0u;
    __syncthreads();
    for (int r = first; r < rows; r += step) {
        uint32_t m = 0;
#pragma unroll
        for (int j = 0; j < KEEP; ++j) {
            const int c = 8 * (WAVE * (part + wpr * j) + lane);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[j][i] = 0.0f;
            if (c < cols) i8_load8<XF>(x, r * ldx + c, v[j]);
            m = max(m, i8_max8(v[j]));
        }
        for (int c = 8 * (WAVE * (part + wpr * KEEP) + lane); c < cols; c += 8 * WAVE * wpr) {
            float u[8];
            i8_load8<XF>(x, r * ldx + c, u);
            m = max(m, i8_max8(u));
        }
        m = wave_max_u32(m);
        if (lane == 0) atomicMax(&top[r], m);
    }
    __syncthreads();
    for (int r = first; r < rows; r += step) {
        const float s = i8_scale(top[r]);
        const I8Scale p = i8_scale_parts(s);
        if (part == 0 && lane == 0) scales[r] = s;
        int8_t* q = codes + r * ldq;
#pragma unroll
        for (int j = 0; j < KEEP; ++j) {
            const int c = 8 * (WAVE * (part + wpr * j) + lane);
            if (c < cols) {
                if (rows > step) i8_load8<XF>(x, r * ldx + c, v[j]);  // (the registers hold the wavefront's last row)
                *reinterpret_cast<uint2*>(q + c) = i8_codes8(v[j], p);
            }
        }
        for (int c = 8 * (WAVE * (part + wpr * KEEP) + lane); c < cols; c += 8 * WAVE * wpr) {
            float u[8];
            i8_load8<XF>(x, r * ldx + c, u);
            *reinterpret_cast<uint2*>(q + c) = i8_codes8(u, p);
        }
    }
    __syncthreads();
}

// 16 NR output columns x 16 NT rows per workgroup, K split over its wavefronts.
// XF: codes, or rows that are quantised here (all of them in one workgroup's LDS).
template <int NT, int NR, int OF, int XF>
__global__ __launch_bounds__(WAVE * SW) void i8_dense_stream_kernel(ChannelArgs a) {
    constexpr bool LX = XF != MOE_DT_I8CH;
    extern __shared__ __attribute__((aligned(16))) int8_t codes[];  // [m, k], LX
    __shared__ i32x4_t part[SW][NR][NT][WAVE];
    __shared__ uint32_t top[LX ? 16 : 1];
    __shared__ float scales[LX ? 16 : 1];
    const int lane = lane_id(), wave = wave_index();
    const int c0 = blockIdx.x * 16 * NR, m0 = blockIdx.y * 16 * NT, steps = (a.k + SK - 1) / SK;
    i32x4_t acc[NR][NT];
    const int8_t* wp[NR];
    int xr[NT];
#pragma unroll
    for (int r = 0; r < NR; ++r) {
        wp[r] = a.wq + (size_t)min(c0 + 16 * r + lane % 16, a.n - 1) * a.k;
#pragma unroll
        for (int t = 0; t < NT; ++t) acc[r][t] = i32x4_t{0, 0, 0, 0};
    }
#pragma unroll
    for (int t = 0; t < NT; ++t) xr[t] = min(m0 + 16 * t + lane % 16, a.m - 1);
    const int per = (steps + SW * UU - 1) / (SW * UU) * UU, s0 = wave * per, s1 = min(steps, s0 + per);
    if constexpr (LX) {
        stream<NR, NT, UU, true>(
            wp, [&](int t, int c) { return *reinterpret_cast<const i32x4_t*>(codes + xr[t] * a.k + c); }, s0, s1, a.k, acc,
            [&] { rows_to_lds<XF>(a.x, a.m, a.k, a.k, codes, a.k, top, scales); });
    } else {
        const int8_t* xp[NT];
#pragma unroll
        for (int t = 0; t < NT; ++t) xp[t] = static_cast<const int8_t*>(a.x) + (size_t)xr[t] * a.k;
        stream<NR, NT, UU, false>(wp, [&](int t, int c) { return ld_codes(xp[t] + c); }, s0, s1, a.k, acc, [] {});
    }
#pragma unroll
    for (int r = 0; r < NR; ++r)
#pragma unroll
        for (int t = 0; t < NT; ++t) part[wave][r][t][lane] = acc[r][t];
    __syncthreads();
    // wavefront w adds the partial sums of the (r, t) tiles w, w + SW, ...
    for (int q = wave; q < NR * NT; q += SW) {
        const int r = q / NT, t = q % NT;
        i32x4_t s = part[0][r][t][lane];
#pragma unroll
        for (int w = 1; w < SW; ++w) s += part[w][r][t][lane];
        const int c = c0 + 16 * r + 4 * (lane / 16), row = m0 + 16 * t + lane % 16;
        if (c >= a.n || row >= a.m) continue;
        const float sx = LX ? scales[row] : a.xs[row];
        float v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = (float)s[i] * sx * a.ws[min(c + i, a.n - 1)];
        f8_store4<OF>(a.out, (size_t)row * a.n + c, a.n - c, v, a.n % 4 == 0);
    }
}

template <int NT, int NR, int XF>
hipError_t dense_launch(const ChannelArgs& a, hipStream_t st) {
    const dim3 grid((a.n + 16 * NR - 1) / (16 * NR), (a.m + 16 * NT - 1) / (16 * NT));
    const size_t lds = XF == MOE_DT_I8CH ? 0 : (size_t)a.m * a.k;
    if (a.odt == MOE_DT_BF16) i8_dense_stream_kernel<NT, NR, MOE_DT_BF16, XF><<<grid, WAVE * SW, lds, st>>>(a);
    else i8_dense_stream_kernel<NT, NR, MOE_DT_F32, XF><<<grid, WAVE * SW, lds, st>>>(a);
    return hipGetLastError();
}

// ---------------------------------------------------------------------------
// Experts of few tokens.  A slot is an expert with its rows, or the shared expert
// with the tokens: a tile of the list, of which each holds up to 16 rows.
// ---------------------------------------------------------------------------

// Gate/up: 16 columns of h of one slot per workgroup, K split over its wavefronts.
__global__ __launch_bounds__(WAVE * SW) void i8_gateup_stream_kernel(I8Ffn a) {
    __shared__ i32x4_t part[SW][2][WAVE];
    const int slot = blockIdx.y, lane = lane_id(), wave = wave_index(), tid = threadIdx.x;
    const int2 tile = a.f.tiles[slot];  // (the list has room for every slot of the grid)
    if (slot >= tile_count(a.f)) return;
    const bool shared = tile.x == a.f.E;
    const int F = shared ? a.f.Fs : a.f.F, d = a.f.d, c0 = blockIdx.x * 16;
    if (c0 >= F) return;
    const MatRef& G = shared ? a.f.s_gate : a.f.gate;
    const MatRef& U = shared ? a.f.s_up : a.f.up;
    const size_t row0 = (size_t)(shared ? 0 : tile.x) * F + c0;
    const int8_t* wp[2] = {static_cast<const int8_t*>(G.q) + (row0 + lane % 16) * d,
                           static_cast<const int8_t*>(U.q) + (row0 + lane % 16) * d};
    i32x4_t acc[2][1] = {{i32x4_t{0, 0, 0, 0}}, {i32x4_t{0, 0, 0, 0}}};
    const int steps = (d + SK - 1) / SK, per = (steps + SW * UU - 1) / (SW * UU) * UU, s0 = wave * per;
    TileRows tr;
    int token = 0;
    const int8_t* xp = a.xq;
    stream<2, 1, UU, false>(
        wp, [&](int, int c) { return ld_codes(xp + c); }, s0, min(steps, s0 + per), d, acc,
        [&] {
            tile_rows<16>(a.f, slot, tr);
            const int r = min(lane % 16, tr.nrows - 1);
            token = shared ? tr.rbeg - a.f.T * a.f.k + r : a.f.perm_rows[tr.rbeg + r] / a.f.k;
            xp = a.xq + (size_t)token * d;
        });
    part[wave][0][lane] = acc[0][0];
    part[wave][1][lane] = acc[1][0];
    __syncthreads();
    if (tid >= 256) return;
    // value tid % 4 of lane tid / 4 of the sums
    const int* p = reinterpret_cast<const int*>(&part[0][0][0]) + tid;
    int g = 0, u = 0;
#pragma unroll
    for (int w = 0; w < SW; ++w) {
        g += p[w * 512];
        u += p[w * 512 + 256];
    }
    const int r = tid / 4 % 16, c = 4 * (tid / 64) + tid % 4, t = __shfl(token, r);
    if (r >= tr.nrows) return;
    const float sx = a.xs[t];
    const float ga = (float)g * sx * reinterpret_cast<const float*>(G.scale)[row0 + c];
    const float up = (float)u * sx * reinterpret_cast<const float*>(U.scale)[row0 + c];
    a.h[(size_t)(tr.rbeg + r) * a.f.ldh + c0 + c] = silu_f32(ga) * up;
}

// Down and combine: 16 columns of y per workgroup, of all tokens.  K goes in
// chunks of 512 columns, the next one's weights on their way while one is
// multiplied.  Many slots: each wavefront takes whole slots in turn, and nothing
// stands between them.  SPLIT (few slots): the chunks are dealt to the wavefronts,
// whose int32 sums are added in LDS.  A slot's sums become rows in LDS (with the
// routing weights), and at the end the rows of a token are added in the order the
// combine has.  (Quantising the rows of h here too, in every workgroup under its
// first weights, took as long as the launch that does it: a call of one token on the same inputs 51.5 /
// 50.2 us.)
constexpr int DI = 8;  // steps of a chunk
struct DownRow {  // of h
    int f;        // its result row
    float w, sx;  // routing weight, scale
    int pad;
};
struct DownLds {
    int rows, slots;  // of h; of the list
    bool split;
    __host__ __device__ size_t bytes() const { return (size_t)rows * (64 + sizeof(DownRow)) + (size_t)slots * (split ? 16 + 1024 : 16); }
};
template <int OF, bool SPLIT>
__global__ __launch_bounds__(WAVE * SW) void i8_down_stream_kernel(I8Ffn a, void* y, DownLds m) {
    extern __shared__ __attribute__((aligned(16))) uint8_t down_lds[];
    float* rows = reinterpret_cast<float*>(down_lds);
    DownRow* info = reinterpret_cast<DownRow*>(rows + m.rows * 16);
    int4* slots = reinterpret_cast<int4*>(info + m.rows);
    int* sums = reinterpret_cast<int*>(slots + m.slots);  // [slots][4 lane + v], SPLIT
    const int lane = lane_id(), wave = wave_index(), tid = threadIdx.x, lo = 16 * (lane / 16);
    const int c0 = blockIdx.x * 16, d = a.f.d, Tk = a.f.T * a.f.k;
    const int n = min(tile_count(a.f), m.slots);
    for (int i = tid; i < m.rows; i += WAVE * SW) {
        const int f = i < Tk ? a.f.perm_rows[i] : i;  // (every assignment of a selection is listed)
        info[i] = DownRow{f, i < Tk ? a.f.topk_w[f] : 1.0f, a.hs[i], 0};
    }
    for (int i = tid; i < m.slots; i += WAVE * SW) {
        const int2 t = a.f.tiles[i];
        TileRows tr = {0, 0, 0};
        if (i < n) tile_rows<16>(a.f, i, tr);
        slots[i] = make_int4(t.x, tr.rbeg, tr.nrows, 0);
    }
    if constexpr (SPLIT) {
        for (int i = tid; i < n * 256; i += WAVE * SW) sums[i] = 0;
    }
    __syncthreads();
    const int kmax = a.f.n_shared && a.f.Fs > a.f.F ? a.f.Fs : a.f.F;
    const int kx = (kmax + SK * DI - 1) / (SK * DI);  // chunks of a slot
    struct Chunk {
        i32x4_t w[DI], x[DI];
        int K, s0;
    };
    auto weights_of = [&](const int4& s) -> const MatRef& { return s.x == a.f.E ? a.f.s_down : a.f.down; };
    auto row_of = [&](const int4& s) { return (size_t)(s.x == a.f.E ? 0 : s.x) * d + c0; };  // first of the 16 weight rows
    auto load = [&](Chunk& f, const int4& s, int chunk) {
        f.K = s.x == a.f.E ? a.f.Fs : a.f.F;
        f.s0 = chunk * DI;
        const int8_t* wp = static_cast<const int8_t*>(weights_of(s).q) + (row_of(s) + lane % 16) * f.K;
        const int row = s.y + min(lane % 16, s.z - 1);
        const int8_t* xp = a.hq + (size_t)row * a.f.ldh;
#pragma unroll
        for (int u = 0; u < DI; ++u) {
            const int c = min(SK * (f.s0 + u) + lo, f.K - 16);  // (columns past the end: re-read, not used)
            f.w[u] = ld_codes(wp + c);
            f.x[u] = ld_codes(xp + c);
        }
        pin();
    };
    auto multiply = [&](const Chunk& f, i32x4_t acc) {
#pragma unroll
        for (int u = 0; u < DI; ++u) {
            const bool in = SK * (f.s0 + u) + lo < f.K;
            acc = dot16(f.w[u], in ? f.x[u] : i32x4_t{0, 0, 0, 0}, acc);
        }
        return acc;
    };
    auto result = [&](int sum, const int4& s, int r, int c, float sw) {  // row r of the slot, column c of the 16
        const DownRow q = info[s.y + r];
        const float v = (float)sum * q.sx * sw;
        rows[q.f * 16 + c] = v * q.w;
    };
    Chunk cur, next;
    if constexpr (SPLIT) {
        const int items = n * kx;  // chunks of all slots
        if (wave < items) load(cur, slots[wave / kx], wave % kx);
        for (int item = wave; item < items; item += SW) {
            if (item + SW < items) load(next, slots[(item + SW) / kx], (item + SW) % kx);
            const i32x4_t acc = multiply(cur, i32x4_t{0, 0, 0, 0});
#pragma unroll
            for (int v = 0; v < 4; ++v) atomicAdd(&sums[item / kx * 256 + 4 * lane + v], acc[v]);
            cur = next;
        }
        __syncthreads();
        for (int o = tid; o < n * 256; o += WAVE * SW) {
            const int4 s = slots[o / 256];
            const int r = o / 4 % 16, c = 4 * (o / 64 % 4) + o % 4;
            if (r < s.z) result(sums[o], s, r, c, reinterpret_cast<const float*>(weights_of(s).scale)[row_of(s) + c]);
        }
    } else {
        int slot = wave, chunk = 0;
        int4 s = slots[min(slot, n - 1)];
        if (slot < n) load(cur, s, 0);
        i32x4_t acc = {0, 0, 0, 0};
        while (slot < n) {
            const bool done = SK * DI * (chunk + 1) >= cur.K;  // the slot's last chunk
            const bool more = !done || slot + SW < n;
            const int4 after = done && more ? slots[slot + SW] : s;
            if (more) load(next, after, done ? 0 : chunk + 1);
            acc = multiply(cur, acc);
            ++chunk;
            if (done) {
                const f8_f4 sw = i8_scales4(reinterpret_cast<const float*>(weights_of(s).scale) + row_of(s) + 4 * (lane / 16));
                if (lane % 16 < s.z) {
#pragma unroll
                    for (int v = 0; v < 4; ++v) result(acc[v], s, lane % 16, 4 * (lane / 16) + v, sw[v]);
                }
                acc = i32x4_t{0, 0, 0, 0};
                slot += SW;
                chunk = 0;
                s = after;
            }
            cur = next;
        }
    }
    __syncthreads();
    if (tid < a.f.T * 16) {
        const int t = tid / 16, c = tid % 16;
        float v = a.f.n_shared ? rows[(Tk + t) * 16 + c] : 0.0f;
        for (int j = 0; j < a.f.k; ++j) v += rows[(t * a.f.k + j) * 16 + c];
        const size_t at = (size_t)t * d + c0 + c;
        if constexpr (OF == MOE_DT_BF16) static_cast<uint16_t*>(y)[at] = f32_to_bf16(v);
        else static_cast<float*>(y)[at] = v;
    }
}

}  // namespace

// Rows that are quantised by the product itself: every workgroup of 16 output
// columns does it again, so few values and few workgroups (us against a launch of its
// own first, bf16 rows, cold weights: 4096 x 6144, 1 row 10.3 / 12.8, 4 rows 12.9 / 13.7;
// 6144 x 2048, 8 rows 11.5 / 12, 12 rows 13.9 / 13.9; 24576 x 6144, 1 row 50 / 48).
bool channel_matmul_takes(int m, int n, int k) { return m <= 16 && (int64_t)m * k <= I8_FUSE_VALUES && n <= 8192; }

// The smallest tiles that leave no more than one workgroup to a compute unit, whose
// eight wavefronts share the sum (us, 16 x 16 / 32 x 16 / 32 x 32 / LDS tiles of 64 x
// 64, n x k: 64 rows of 1024 x 6144, 256 workgroups of the smallest, 8.4 / 11.6 / 13.3 /
// 16.6; 32 rows of 4096 x 6144 15.5 / 13.7 / 16.8 / 16.7; 64 rows of it 26 / 22 / 16.4 /
// 18.7; 96 rows 36 / 29 / 27 / 16.9; 512 rows of 512 x 2048 9.9 / 8.0 / 6.0 / 7.3; 48 of 6144 x
// 2048 14.2 / 12.3 / 10.3 / 8.9).
hipError_t launch_channel_matmul(const ChannelArgs& a, hipStream_t st) {
    if (a.xdt == MOE_DT_BF16) return dense_launch<1, 1, MOE_DT_BF16>(a, st);
    if (a.xdt == MOE_DT_F32) return dense_launch<1, 1, MOE_DT_F32>(a, st);
    auto groups = [&](int nt, int nr) { return (long)((a.m + 16 * nt - 1) / (16 * nt)) * ((a.n + 16 * nr - 1) / (16 * nr)); };
    if (a.m <= 16 || groups(1, 1) <= 256) return dense_launch<1, 1, MOE_DT_I8CH>(a, st);
    if (groups(2, 1) <= 256) return dense_launch<2, 1, MOE_DT_I8CH>(a, st);
    if (groups(2, 2) <= 256) return dense_launch<2, 2, MOE_DT_I8CH>(a, st);
    return launch_channel_matmul_tile(a, st);
}

// Layers of few tokens, 16 being the rows of an instruction.
bool i8_stream_takes(int T) { return T <= F8_ROUTE_MAX_T; }

hipError_t launch_i8_gateup_stream(const I8Ffn& a, hipStream_t st, const KTime& kt) {
    const int fmax = a.f.n_shared && a.f.Fs > a.f.F ? a.f.Fs : a.f.F;
    launch_kernel(i8_gateup_stream_kernel, dim3((fmax + 15) / 16, a.f.max_tiles), WAVE * SW, st, kt, a);
    return hipGetLastError();
}

// Up to this many routed rows the chunks of K are split over the wavefronts.
constexpr int DOWN_SPLIT_ROWS = 16;

hipError_t launch_i8_down_stream(const I8Ffn& a, void* y, int ydt, hipStream_t st, const KTime& kt) {
    // (up to 16 * 33 rows and 522 slots: 51 KB; split, 32 and 18: 22 KB)
    const DownLds m = {a.f.T * a.f.k + (a.f.n_shared ? a.f.T : 0), a.f.max_tiles, a.f.T * a.f.k <= DOWN_SPLIT_ROWS};
    const dim3 grid(a.f.d / 16);
    auto go = [&](auto kernel) {
        if (kt.start || kt.stop) hipExtLaunchKernelGGL(kernel, grid, WAVE * SW, m.bytes(), st, kt.start, kt.stop, 0, a, y, m);
        else kernel<<<grid, WAVE * SW, m.bytes(), st>>>(a, y, m);
    };
    auto pick = [&](auto of) {
        constexpr int OF = decltype(of)::value;
        if (m.split) go(i8_down_stream_kernel<OF, true>);
        else go(i8_down_stream_kernel<OF, false>);
    };
    if (ydt == MOE_DT_BF16) pick(ic<MOE_DT_BF16>());
    else pick(ic<MOE_DT_F32>());
    return hipGetLastError();
}

}  // namespace moe
