// balance.hip - the router's training side: how evenly the experts are loaded,
// the loss that says so, and the gradient of the logits.
//
//   p[t, e] = s[t, e] / sum_e s[t, e],   s the router's scores
//   c[q, e] = selections of expert e by sequence q's tokens, n[q] its tokens
//   f[q, e] = E c[q, e] / (k n[q]),      P[q, e] = mean of p over its tokens
//   loss[q] = sum_e f[q, e] P[q, e]      (f is a constant of the gradient)
//   dL/dl[t, e] = d_loss[q] / n[q] (f[q, e] - sum_i f[q, i] p[t, i]) d(log s)/dl p[t, e]
//               + the selected weights' part (w = scale s / sum_sel s, or scale s)
//   (softmax: d(log s)/dl is 1, and weights that are not renormalised take
//   p[t, e] sum_j d_w[t, j] w[t, j] off)
//
// Both directions read the logits once.  G lanes take a token (16 up to 256 experts,
// so that a wavefront has four and a sum over experts is four DPP steps; 64 beyond):
// lane `sub` holds four experts in a row, from 4 (sub + G j), j = 0 .. J - 1.
//
// Forward: a workgroup takes a range of tokens, sequence by sequence.  Its
// wavefronts' sums meet in LDS in a fixed order and go to the slot (range +
// sequence) of the workspace: along the tokens each step to the next range or
// the next sequence is one slot further, so no two sums share one and none has
// to be cleared first.  A second launch adds each sequence's slots in fp64 (one
// range and few sequences: the same workgroup does).  No floating-point atomics:
// the same bits every time.
#include <algorithm>
#include <type_traits>

#include "balance.h"
#include "common.h"

namespace moe {
namespace {

constexpr int BW = 8;   // wavefronts per workgroup of the forward pass

// Sequences.  q(t): the last sequence that begins at or before t (-1: none;
// n_seq: behind the last one), t the same in all lanes, which look at 64 offsets
// at once.  Offsets that do not ascend give some sequence, never an index out of
// range.
__device__ __forceinline__ int seq_of(const int32_t* off, int n_seq, int t) {
    int lo = 0, n = n_seq + 1;  // off[lo - 1] <= t < off[lo + n]
    while (n > 0) {
        const int step = (n + WAVE - 1) / WAVE, i = lo + step * (lane_id() + 1) - 1;  // the last of the lane's offsets
        const int at = min(i, lo + n - 1);
        const int below = __popcll(__ballot(lo + step * lane_id() < lo + n && off[at] <= t));
        const int end = lo + n;
        lo += step * below;
        if (lo >= end) return end - 1;
        n = step == 1 ? 0 : min(step, end - lo) - 1;
    }
    return lo - 1;
}

// 2^add e^x for x <= 0 and 0 <= add <= 32, off by less than two units where that is no
// denormal (2^r 2^f with |f| <= 1/2, f from the product's exact low part); 0 where it
// vanishes, NaN stays.
__device__ __forceinline__ float exp_neg(float x, int add) {
    constexpr float L = 1.44269502f, L_LO = 1.92596299e-8f, BIG = 12582912.0f;  // log2 e; 1.5 * 2^23
    x = x < -200.0f ? -200.0f : x;
    const float t = fmaf(x, L, BIG), r = t - BIG;
    const float p = __builtin_amdgcn_exp2f(fmaf(x, L_LO, fmaf(x, L, -r)));
    return __builtin_ldexpf(p, (int)(__float_as_uint(t) - __float_as_uint(BIG)) + add);
}

// 2^32 s and 2^32 ds/dl, s the score of a logit (softmax: up to the common factor, m the
// row's maximum, and the score itself in the derivative's place).  Scores are products
// of e^l, or e^(l / 2), and so denormal, or zero, long before a token's probabilities
// lose their meaning: with the factor all those count in full whose sum is 2^-126 and
// more, or that are not 0 as the selection's fp32 scores, and none overflows (the
// largest is 2^32 sqrt(FLT_MAX)).  The reciprocal, root and logarithm instructions are
// off by one unit each.
constexpr int UP_BITS = 32;
constexpr float UP = 0x1p32f, DOWN = 0x1p-32f;
template <int KIND, bool GRAD>
__device__ __forceinline__ float score_of(float l, float m, float& ds) {
    if constexpr (KIND == MOE_SCORE_SOFTMAX) {
        const float s = exp_neg(l - m, UP_BITS);
        if (GRAD) ds = s;
        return s;
    } else if constexpr (KIND == MOE_SCORE_SIGMOID) {
        // a = 2^32 e^-|l|: neither direction overflows, and 1 - sigmoid keeps its digits
        const float a = exp_neg(-fabsf(l), UP_BITS), h = __builtin_amdgcn_rcpf(fmaf(a, DOWN, 1.0f));
        if (GRAD) ds = a * h * h;
        return (l >= 0.0f ? UP : a) * h;
    } else {
        // below -20 softplus is e^l, off by e^-20 / 2 of itself at most, and the score e^(l / 2)
        const bool low = l < -20.0f;
        const float e = exp_neg(low ? 0.5f * l : -fabsf(l), UP_BITS), a = e * DOWN, u = 1.0f + a;
        // log(1 + a) = log u + (a - (u - 1)) / u, the difference being exact
        const float h = __builtin_amdgcn_rcpf(u), lg = fmaf(__builtin_amdgcn_logf(u), 0.693147181f, (a - (u - 1.0f)) * h);
        const float x = (l < 0.0f ? 0.0f : l) + lg, s = __builtin_amdgcn_sqrtf(x);
        if (GRAD) ds = low ? 0.5f * e : 0.5f * UP * ((l >= 0.0f ? 1.0f : a) * h) * __builtin_amdgcn_rcpf(s);
        return low ? e : s * UP;
    }
}

template <class F>
__device__ __forceinline__ void with_score(int kind, F&& f) {
    if (kind == MOE_SCORE_SOFTMAX) f(std::integral_constant<int, MOE_SCORE_SOFTMAX>());
    else if (kind == MOE_SCORE_SIGMOID) f(std::integral_constant<int, MOE_SCORE_SIGMOID>());
    else f(std::integral_constant<int, MOE_SCORE_SQRT_SOFTPLUS>());
}

// Over the G lanes of a token; each of them receives the same bits.
template <int G, class Op>
__device__ __forceinline__ float row_reduce(float v, Op op) {
    v = op(v, __uint_as_float(dpp_u32<0x128>(__float_as_uint(v))));  // row_ror 8, 4, 2, 1
    v = op(v, __uint_as_float(dpp_u32<0x124>(__float_as_uint(v))));
    v = op(v, __uint_as_float(dpp_u32<0x122>(__float_as_uint(v))));
    v = op(v, __uint_as_float(dpp_u32<0x121>(__float_as_uint(v))));
    if constexpr (G == WAVE) {
        const auto row = [&](int r) { return __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(v), 16 * r)); };
        v = op(op(row(0), row(1)), op(row(2), row(3)));
    }
    return v;
}
struct MaxF { __device__ float operator()(float a, float b) const { return fmaxf(a, b); } };
template <int G> __device__ __forceinline__ float row_sum(float v) { return row_reduce<G>(v, AddF()); }

// Whether it holds for one of a token's lanes.
template <int G>
__device__ __forceinline__ bool row_any(bool b) {
    const uint64_t m = __ballot(b);
    return G == WAVE ? m != 0 : (m >> (lane_id() & -G) & ((1ull << (G % WAVE)) - 1)) != 0;
}

// The sum of the four rows of 16 lanes, in each of them.
__device__ __forceinline__ float rows_sum(float v) {
    const uint32_t a = __float_as_uint(v);
    const auto p = __builtin_amdgcn_permlane16_swap(a, a, false, false);
    const float w = __uint_as_float(p[0]) + __uint_as_float(p[1]);
    const uint32_t b = __float_as_uint(w);
    const auto q = __builtin_amdgcn_permlane32_swap(b, b, false, false);
    return __uint_as_float(q[0]) + __uint_as_float(q[1]);
}

// Expert of a lane's value 4 j + v.
template <int G>
__device__ __forceinline__ int expert_of(int sub, int v) { return 4 * (sub + G * (v / 4)) + v % 4; }

// Element at of an array of up to 2^20 x 1024 fp32 or int32 values: its bytes are counted
// in 32 bits, which the compiler keeps in one register and adds to a scalar base.
template <class U, class T>
__device__ __forceinline__ U load_at(const T* base, uint32_t at) {
    return *reinterpret_cast<const U*>(reinterpret_cast<const char*>(base) + 4u * at);
}
// A token's row, or a sequence's; WIDE: its length and address are multiples of 16 bytes.
template <int G, int J, bool WIDE, class T4, class T>
__device__ __forceinline__ void load_row(const T* base, int row, int E, int sub, T (&l)[4 * J]) {
    const uint32_t at = (uint32_t)row * E;
    if constexpr (WIDE) {
#pragma unroll
        for (int j = 0; j < J; ++j) {
            const int e = expert_of<G>(sub, 4 * j);
            const T4 x = load_at<T4>(base, at + (e < E ? e : 0));
            l[4 * j] = x.x, l[4 * j + 1] = x.y, l[4 * j + 2] = x.z, l[4 * j + 3] = x.w;
        }
    } else {
#pragma unroll
        for (int v = 0; v < 4 * J; ++v) {
            const int e = expert_of<G>(sub, v);
            l[v] = load_at<T>(base, at + (e < E ? e : 0));
        }
    }
}

// score_of for a token's experts; inv = 1 / their sum (0 where sum s is below 2^-126).
template <int G, int J, bool GRAD>
__device__ __forceinline__ void token_scores(const float (&l)[4 * J], int E, int sub, int kind, float (&s)[4 * J],
                                             float (&ds)[4 * J], float& m, float& inv) {
    m = 0.0f;
    if (kind == MOE_SCORE_SOFTMAX) {
        m = -INFINITY;
#pragma unroll
        for (int v = 0; v < 4 * J; ++v)
            if (expert_of<G>(sub, v) < E) m = fmaxf(m, l[v]);
        m = row_reduce<G>(m, MaxF());
        if (m == -INFINITY) m = 0.0f;  // (no score, rather than NaN)
    }
    float sum = 0.0f;
    with_score(kind, [&](auto KIND) {
#pragma unroll
        for (int v = 0; v < 4 * J; ++v) {
            s[v] = score_of<KIND.value, GRAD>(l[v], m, ds[v]);
            if (expert_of<G>(sub, v) >= E) s[v] = 0.0f;
            sum += s[v];
            if (v % 4 == 3) __builtin_amdgcn_sched_barrier(0);  // four at once: all of them take too many registers
        }
    });
    sum = row_sum<G>(sum);
    inv = sum < 0x1p-126f * UP ? 0.0f : __builtin_amdgcn_rcpf(sum);
}

// A sequence's sum of the wavefronts' parts of its loss, in their order, for thread 0.
template <int W>
__device__ __forceinline__ double loss_sum(double loss, double (&parts)[W]) {
    loss = wave_sum_f64(loss);
    if (lane_id() == 0) parts[wave_index()] = loss;
    __syncthreads();
    for (int w = 1; w < W; ++w) loss += parts[w];
    return loss;
}

template <int G, int J, bool WIDE>
__global__ __launch_bounds__(BW * WAVE) void balance_kernel(BalanceArgs a) {
    constexpr int V = 4 * J, NT = WAVE / G, KI = (BALANCE_MAX_K + G - 1) / G;  // a lane's values, a wavefront's tokens, a lane's selections
    constexpr int EP = G * V;
    __shared__ __attribute__((aligned(16))) float part[BW][EP];
    __shared__ int hist[EP], alive[BW];
    __shared__ double losses[BW];
    const int tid = threadIdx.x, lane = lane_id(), wave = wave_index(), E = a.E;
    const int sub = lane % G, first = wave * NT + lane / G;
    const int t1 = min(a.T, (int)(blockIdx.x + 1) * a.chunk);
    int t0 = blockIdx.x * a.chunk;
    struct Token {
        float l[V];
        int x[KI];
        bool live;
    };
    while (t0 < t1) {
        int q = 0, e = t1;
        if (a.off) {
            q = seq_of(a.off, a.n_seq, t0);
            if (q >= a.n_seq) break;  // (the same in every wavefront)
            e = min(t1, max(a.off[q + 1], t0 + 1));
            if (q < 0) {
                t0 = e;
                continue;
            }
        }
        const auto load = [&](int t, Token& k) {
            k.live = t < e;
            t = min(t, e - 1);
            if (a.mask) k.live = k.live && a.mask[t];
            load_row<G, J, WIDE, float4>(a.logits, t, E, sub, k.l);
#pragma unroll
            for (int i = 0; i < KI; ++i) {
                const int j = sub + G * i;
                k.x[i] = j < a.k ? load_at<int>(a.idx, t * a.k + j) : -1;
            }
        };
        Token cur;
        load(t0 + first, cur);
        for (int i = tid; i < E; i += BW * WAVE) hist[i] = 0;
        __syncthreads();
        float P[V];
        int n = 0;
#pragma unroll
        for (int v = 0; v < V; ++v) P[v] = 0.0f;
        for (int t = t0; t < e; t += BW * NT) {
            float s[V], ds[V], top, inv;
            token_scores<G, J, false>(cur.l, E, sub, a.score, s, ds, top, inv);
            const bool live = cur.live;
            n += live;
#pragma unroll
            for (int i = 0; i < KI; ++i)
                if (live && cur.x[i] >= 0 && cur.x[i] < E) atomicAdd(&hist[cur.x[i]], 1);
            if (t + BW * NT < e) load(t + BW * NT + first, cur);
#pragma unroll
            for (int v = 0; v < V; ++v) P[v] = live ? fmaf(s[v], inv, P[v]) : P[v];
        }
        if constexpr (NT > 1) {
#pragma unroll
            for (int v = 0; v < V; ++v) P[v] = rows_sum(P[v]);
        }
        if (lane < G) {
#pragma unroll
            for (int j = 0; j < J; ++j)
                *reinterpret_cast<float4*>(&part[wave][expert_of<G>(sub, 4 * j)]) =
                    make_float4(P[4 * j], P[4 * j + 1], P[4 * j + 2], P[4 * j + 3]);
        }
        n = sub == 0 ? n : 0;
#pragma unroll
        for (int o = G; o < WAVE; o <<= 1) n += __shfl_xor(n, o);
        if (lane == 0) alive[wave] = n;
        __syncthreads();
        int tokens = 0;
#pragma unroll
        for (int w = 0; w < BW; ++w) tokens += alive[w];
        const size_t slot = (size_t)(blockIdx.x + q), Ep = (E + 3) / 4 * 4;
        const double rn = tokens > 0 ? 1.0 / tokens : 0.0, rf = rn * E / a.k;
        double loss = 0.0;
        for (int i = tid; i < Ep; i += BW * WAVE) {
            float s = part[0][i];
#pragma unroll
            for (int w = 1; w < BW; ++w) s += part[w][i];
            const int c = i < E ? hist[i] : 0;
            if (!a.one_launch) {
                a.sum[slot * Ep + i] = s;
                a.cnt[slot * Ep + i] = c;
            } else if (i < E) {
                a.prob[i] = (float)(s * rn);
                a.counts[i] = c;
                loss += (c * rf) * (s * rn);
            }
        }
        if (a.one_launch) {
            loss = loss_sum(loss, losses);
            if (tid == 0) a.loss[0] = (float)loss, a.tokens[0] = tokens;
            return;
        }
        if (tid == 0) a.num[slot] = tokens;
        __syncthreads();
        t0 = e;
    }
    if (a.one_launch) {  // no tokens
        for (int i = tid; i < E; i += BW * WAVE) a.prob[i] = 0.0f, a.counts[i] = 0;
        if (tid == 0) a.loss[0] = 0.0f, a.tokens[0] = 0;
        return;
    }
    if (a.blocks == 1) return;
    for (int64_t i = (int64_t)blockIdx.x * BW * WAVE + tid; i < a.n_seq; i += (int64_t)gridDim.x * BW * WAVE) a.done[i] = 0;
}

// The second launch: a sequence's experts, or a block of 64 of them, by a workgroup:
// quads of experts x ranges, then the ranges' sums in order.  The last block of a
// sequence to end adds the parts of the loss, in the blocks' order.
constexpr int JW = 16;
__global__ __launch_bounds__(JW * WAVE) void balance_join_kernel(BalanceArgs a) {
    __shared__ double sum[JW * WAVE * 4], losses[JW];
    __shared__ int cnt[JW * WAVE * 4];
    const int q = blockIdx.x / a.blocks, block = blockIdx.x % a.blocks;
    const int tid = threadIdx.x, lane = lane_id(), E = a.E, Q = (E + 3) / 4;
    const int width = a.blocks > 1 ? 16 : Q;  // quads of the block
    const int way = tid / width, quad = block * width + tid % width;
    int b = 0, e = a.T;
    if (a.off) {
        b = max(0, min(a.off[q], a.T));
        e = max(b, min(a.off[q + 1], a.T));
    }
    const int c0 = b / a.chunk, c1 = e > b ? (e - 1) / a.chunk + 1 : c0;
    const int ways = min(min(64, JW * WAVE / width), c1 - c0);
    int n = 0;
    for (int c = c0 + lane; c < c1; c += WAVE) n += a.num[c + q];
    if (way < ways && quad < Q) {
        double s[4] = {};
        int k[4] = {};
#pragma unroll 4
        for (int c = c0 + way; c < c1; c += ways) {
            const size_t at = (size_t)(c + q) * Q + quad;
            const float4 x = reinterpret_cast<const float4*>(a.sum)[at];
            const int4 y = reinterpret_cast<const int4*>(a.cnt)[at];
            s[0] += x.x, s[1] += x.y, s[2] += x.z, s[3] += x.w;
            k[0] += y.x, k[1] += y.y, k[2] += y.z, k[3] += y.w;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) sum[4 * tid + i] = s[i], cnt[4 * tid + i] = k[i];
    }
#pragma unroll
    for (int o = 1; o < WAVE; o <<= 1) n += __shfl_xor(n, o);
    __syncthreads();
    const double rn = n > 0 ? 1.0 / n : 0.0, rf = rn * E / a.k;
    double loss = 0.0;
    const int x = 4 * width * block + tid;
    if (tid < 4 * width && x < E) {
        double s = 0.0;
        int k = 0;
        for (int w = 0; w < ways; ++w) s += sum[4 * width * w + tid], k += cnt[4 * width * w + tid];
        a.prob[(size_t)q * E + x] = (float)(s * rn);
        a.counts[(size_t)q * E + x] = k;
        loss = (k * rf) * (s * rn);
    }
    loss = loss_sum(loss, losses);
    if (tid != 0) return;
    if (block == 0) a.tokens[q] = n;
    if (a.blocks > 1) {
        double* part = a.loss_part + (size_t)q * a.blocks;
        __hip_atomic_store(part + block, loss, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        if (__hip_atomic_fetch_add(a.done + q, 1, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT) != a.blocks - 1) return;
        loss = 0.0;
        for (int i = 0; i < a.blocks; ++i) loss += __hip_atomic_load(part + i, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
    a.loss[q] = (float)loss;
}

constexpr int GW = 4;  // wavefronts per workgroup of the backward pass

// What a wavefront's lanes write to LDS others of them read: in order there, kept
// in order by the compiler too.
__device__ __forceinline__ void lds_in_order() {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

template <int G, int J, bool WIDE>
__global__ __launch_bounds__(GW * WAVE, 4) void route_backward_kernel(RouteGradArgs a) {
    constexpr int V = 4 * J, NT = WAVE / G, KI = (BALANCE_MAX_K + G - 1) / G, EP = G * V;
    __shared__ __attribute__((aligned(16))) float selected[GW][NT][EP];  // the selected weights' part, 0 between tokens
    const int lane = lane_id(), sub = lane % G, grp = lane / G, E = a.E;
    const int w0 = blockIdx.x * GW + wave_index();
    float* buf = selected[wave_index()][grp];
    const bool soft = a.score == MOE_SCORE_SOFTMAX;
    if (a.d_w) {
#pragma unroll
        for (int j = 0; j < J; ++j) *reinterpret_cast<float4*>(buf + expert_of<G>(sub, 4 * j)) = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    }
    struct Token {
        float l[V], dw[KI];
        int x[KI];
        bool live;
    };
    const auto load = [&](int t, Token& k) {
        k.live = t < a.T;
        t = min(t, a.T - 1);
        if (a.mask) k.live = k.live && a.mask[t];
        if (a.d_w) {
#pragma unroll
            for (int i = 0; i < KI; ++i) {
                const int j = sub + G * i;
                const int x = j < a.k ? load_at<int>(a.idx, t * a.k + j) : -1;
                k.x[i] = x >= 0 && x < E ? x : E;
                k.dw[i] = x >= 0 && x < E ? a.scale * load_at<float>(a.d_w, t * a.k + j) : 0.0f;
            }
        }
        load_row<G, J, WIDE, float4>(a.logits, t, E, sub, k.l);
    };
    int q = 0, q_end = 0;  // the sequence of the last token, and its end
    float f[V], rate = 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v) f[v] = 0.0f;
    Token cur;
    const int b = w0 * a.chunk * NT, e = min(a.T, b + a.chunk * NT);
    for (int t_ = b; t_ < e; t_ += NT) {
        const int t = t_ + grp;
        load(t, cur);
        bool entered = false;
        while (const uint64_t need = __ballot(t >= q_end && t < a.T)) {
            const int tn = __builtin_amdgcn_readlane(t, __ffsll((unsigned long long)need) - 1);
            int qn = 0, end = a.T;
            if (a.off) {
                qn = seq_of(a.off, a.n_seq, tn);
                end = qn >= a.n_seq ? a.T : max(a.off[qn + 1], tn + 1);
                if (qn >= a.n_seq) qn = -1;
            }
            if (t >= tn && t >= q_end && t < end) {
                q = qn;
                q_end = end;
                entered = true;
            }
        }
        if (entered) {
            if (a.d_loss && q >= 0) {
                // f - 1: of the gradient's f - sum f p only differences of f count,
                // and small numbers lose less in them
                const int n = max(a.tokens[q], 1);
                const double rf = (double)E / ((double)a.k * n);
                rate = __fdiv_rn(a.d_loss[q], (float)n);
                int c[V];
                load_row<G, J, WIDE, int4>(a.counts, q, E, sub, c);
#pragma unroll
                for (int v = 0; v < V; ++v) f[v] = expert_of<G>(sub, v) < E ? (float)(c[v] * rf - 1.0) : 0.0f;
            }
        }
        float ls[KI];
        if (a.d_w) {
#pragma unroll
            for (int i = 0; i < KI; ++i)
                if (G * i < a.k) ls[i] = load_at<float>(a.logits, (uint32_t)min(t, a.T - 1) * E + (cur.x[i] < E ? cur.x[i] : 0));
        }
        float s[V], ds[V], top, inv;
        token_scores<G, J, true>(cur.l, E, sub, a.score, s, ds, top, inv);
        float off = 0.0f;
        if (a.d_loss) {
            float fp = 0.0f;
#pragma unroll
            for (int v = 0; v < V; ++v) fp = fmaf(f[v], s[v], fp);
            off = rate * (row_sum<G>(fp) * inv);
        }
        if (a.d_w) {
            // a lane's selected experts (E: none), their scores, the scores' derivatives
            // and the weights' gradients
            const float unit = soft ? inv : DOWN;
            float sel[KI], dsel[KI], add[KI], S = 0.0f;
            bool weighs = false;  // some score is not 0 as the selection's fp32 score (or NaN)
            with_score(a.score, [&](auto KIND) {
#pragma unroll
                for (int i = 0; i < KI; ++i) {
                    sel[i] = dsel[i] = 0.0f;
                    if (G * i < a.k && cur.x[i] < E) sel[i] = score_of<KIND.value, true>(ls[i], top, dsel[i]);
                    S += sel[i];
                    weighs = weighs || sel[i] * unit != 0.0f;
                }
            });
            if (a.normalise) {
                // 1 / S only ever multiplies scores and their derivatives, which are as small
                // as S: with dL/ds = (dw - dot) / S first, small scores would overflow
                S = row_sum<G>(S);
                const float rS = row_any<G>(weighs) ? __builtin_amdgcn_rcpf(S) : 0.0f;
                float dot = 0.0f;
#pragma unroll
                for (int i = 0; i < KI; ++i) dot += cur.dw[i] * (sel[i] * rS);
                dot = row_sum<G>(dot);
#pragma unroll
                for (int i = 0; i < KI; ++i) cur.dw[i] = cur.x[i] < E ? (cur.dw[i] - dot) * (dsel[i] * rS) : 0.0f;
            } else {
                float sum = 0.0f;
#pragma unroll
                for (int i = 0; i < KI; ++i) {
                    cur.dw[i] = cur.dw[i] * dsel[i] * unit;
                    sum += cur.dw[i];
                }
                if (soft) off += row_sum<G>(sum);  // (renormalised weights' add up to nothing, as the balance part does)
            }
            // an expert listed twice: one of its lanes reads the other's mark, and all
            // of them take the sum in the order of the list
            bool twice = false;
#pragma unroll
            for (int i = 0; i < KI; ++i) {
                add[i] = cur.dw[i];
                if (cur.x[i] < E) reinterpret_cast<int*>(buf)[cur.x[i]] = lane + WAVE * i;
            }
            lds_in_order();
#pragma unroll
            for (int i = 0; i < KI; ++i)
                if (cur.x[i] < E) twice |= reinterpret_cast<int*>(buf)[cur.x[i]] != lane + WAVE * i;
            if (__ballot(twice)) {
#pragma unroll
                for (int i = 0; i < KI; ++i) add[i] = 0.0f;
                for (int j = 0; j < a.k; ++j) {
                    int xj = E;
                    float dj = 0.0f;
#pragma unroll
                    for (int i = 0; i < KI; ++i) {
                        const int x = __shfl(cur.x[i], j % G, G);
                        const float d = __shfl(cur.dw[i], j % G, G);
                        if (j / G == i) xj = x, dj = d;
                    }
#pragma unroll
                    for (int i = 0; i < KI; ++i)
                        if (cur.x[i] == xj) add[i] += dj;
                }
            }
            lds_in_order();
#pragma unroll
            for (int i = 0; i < KI; ++i)
                if (cur.x[i] < E) buf[cur.x[i]] = add[i];
            lds_in_order();
        }
        const float unit = a.d_loss || soft ? inv : 1.0f;  // (1: zeros, or NaN of a NaN logit)
        float g[V];
#pragma unroll
        for (int v = 0; v < V; ++v) g[v] = fmaf(rate, f[v], -off) * ds[v] * unit;
        if (a.d_w) {
#pragma unroll
            for (int j = 0; j < J; ++j) {
                const float4 d = *reinterpret_cast<const float4*>(buf + expert_of<G>(sub, 4 * j));
                g[4 * j] += d.x, g[4 * j + 1] += d.y, g[4 * j + 2] += d.z, g[4 * j + 3] += d.w;
            }
            lds_in_order();
#pragma unroll
            for (int i = 0; i < KI; ++i)
                if (cur.x[i] < E) buf[cur.x[i]] = 0.0f;
            lds_in_order();
        }
        const bool live = cur.live && q >= 0;  // else no gradient
#pragma unroll
        for (int v = 0; v < V; ++v) g[v] = live ? g[v] : 0.0f;
        if (t < a.T) {
            float* out = a.d_logits + (size_t)t * E;
            if constexpr (WIDE) {
#pragma unroll
                for (int j = 0; j < J; ++j) {
                    const int x = expert_of<G>(sub, 4 * j);
                    if (x < E) *reinterpret_cast<float4*>(out + x) = make_float4(g[4 * j], g[4 * j + 1], g[4 * j + 2], g[4 * j + 3]);
                }
            } else {
#pragma unroll
                for (int v = 0; v < V; ++v)
                    if (expert_of<G>(sub, v) < E) out[expert_of<G>(sub, v)] = g[v];
            }
        }
    }
}

// Lanes a token, quads of experts a lane, and whether rows are read as quads.
template <class F>
void with_layout(int E, uintptr_t addresses, F&& f) {
    using std::integral_constant;
    const auto go = [&](auto G, auto J) {
        if (E % 4 == 0 && addresses % 16 == 0) f(G, J, std::true_type());
        else f(G, J, std::false_type());
    };
    const integral_constant<int, 16> g16;
    const integral_constant<int, WAVE> g64;
    if (E <= 64) go(g16, integral_constant<int, 1>());
    else if (E <= 128) go(g16, integral_constant<int, 2>());
    else if (E <= 192) go(g16, integral_constant<int, 3>());
    else if (E <= 256) go(g16, integral_constant<int, 4>());
    else if (E <= 512) go(g64, integral_constant<int, 2>());
    else go(g64, integral_constant<int, 4>());
}

}  // namespace

int balance_chunk(int T, int E, int n_seq) {
    // whole rounds of a workgroup's wavefronts; two of them stay in one workgroup, and
    // one launch (37 tokens of 192 experts: 4.9 us, two launches 6.9; four rounds of
    // 256 experts: 8.4, 7.5), where there are no more sequences to take one by one
    const int round = BW * (E <= 256 ? 4 : 1);
    if (T <= 2 * round && n_seq == 1) return 2 * round;
    const int per = (T + BALANCE_MAX_RANGES - 1) / BALANCE_MAX_RANGES;
    return (per + round - 1) / round * round;
}

hipError_t launch_balance(BalanceArgs a, hipStream_t st) {
    const int grid = (a.T + a.chunk - 1) / a.chunk;
    // 64 experts a workgroup of the second launch where a sequence has many ranges
    // (one sequence of 65536 tokens and 256 experts: 25.4 us, 28.9 with all of them; of
    // 2048 tokens: 10.9, 9.0)
    a.blocks = grid / a.n_seq >= 256 ? (a.E + 63) / 64 : 1;
    a.one_launch = grid == 1 && a.n_seq == 1;
    with_layout(a.E, reinterpret_cast<uintptr_t>(a.logits), [&](auto G, auto J, auto WIDE) {
        balance_kernel<G.value, J.value, WIDE.value><<<grid, BW * WAVE, 0, st>>>(a);
    });
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || a.one_launch) return e;
    balance_join_kernel<<<a.n_seq * a.blocks, JW * WAVE, 0, st>>>(a);
    return hipGetLastError();
}

hipError_t launch_route_backward(RouteGradArgs a, hipStream_t st) {
    const uintptr_t addresses = reinterpret_cast<uintptr_t>(a.logits) | reinterpret_cast<uintptr_t>(a.d_logits) |
                                reinterpret_cast<uintptr_t>(a.counts);
    with_layout(a.E, addresses, [&](auto G, auto J, auto WIDE) {
        const int64_t rounds = ((int64_t)a.T * G.value + WAVE - 1) / WAVE;  // a wavefront's tokens at a time
        a.chunk = (int)std::min<int64_t>(std::max<int64_t>(rounds / 4096, 1), 8);
        const int grid = (int)((rounds + GW * a.chunk - 1) / (GW * a.chunk));
        route_backward_kernel<G.value, J.value, WIDE.value><<<grid, GW * WAVE, 0, st>>>(a);
    });
    return hipGetLastError();
}

}  // namespace moe
