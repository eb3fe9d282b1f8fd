// balance.hip - the router's training side: how evenly the experts are loaded,
// the loss that says so, and the gradient of the logits.
//
//   p[t, e] = s[t, e] / sum_e s[t, e],   s the router's scores
//   c[q, e] = selections of expert e by sequence q's tokens, n[q] its tokens
//   f[q, e] = E c[q, e] / (k n[q]),      P[q, e] = mean of p over its tokens
//   loss[q] = sum_e f[q, e] P[q, e]      (f is a constant of the gradient)
//   dL/ds[t, e] = d_loss[q] / n[q] (f[q, e] - sum_i f[q, i] p[t, i]) / sum s
//               + the selected weights' part (w = scale s / sum_sel s, or scale s)
//   dL/dl[t, e] = dL/ds[t, e] s'(l), softmax: s_e (dL/ds_e - sum_i dL/ds_i s_i)
//
// Both directions read the logits once and are bound by memory.  A wavefront
// takes a token; lane l holds experts l, l + 64, ...
//
// Forward: a workgroup takes a range of tokens, sequence by sequence.  Its
// wavefronts' sums meet in LDS in a fixed order and go to the slot (range +
// sequence) of the workspace: along the tokens each step to the next range or
// the next sequence is one slot further, so no two sums share one and none has
// to be cleared first.  A second launch adds each sequence's slots in fp64.  No
// floating-point atomics: the same bits every time.
#include "balance.h"
#include "common.h"

namespace moe {
namespace {

constexpr int BW = 16;  // wavefronts per workgroup of the forward pass

// Sequences.  q(t): the last sequence that begins at or before t (-1: none).
// Offsets that do not ascend give some sequence, never an index out of range.
__device__ __forceinline__ int seq_of(const int32_t* off, int n_seq, int t) {
    int lo = 0, hi = n_seq + 1;  // off[lo - 1] <= t < off[hi]
    while (lo < hi) {
        const int mid = (lo + hi) / 2;
        if (off[mid] <= t) lo = mid + 1;
        else hi = mid;
    }
    return lo - 1;  // n_seq: behind the last sequence
}

// Scores of one token, up to a common factor (softmax), and the derivatives
// that do not need the sum.
template <int KPL>
struct Scores {
    float s[KPL], ds[KPL];  // ds: s'(l) (not softmax)
    float inv;              // 1 / sum s, 0 where the scores vanish
};

template <int KPL, bool GRAD>
__device__ __forceinline__ void token_scores(const float (&l)[KPL], int E, int kind, Scores<KPL>& r) {
    const int lane = lane_id();
    if (kind == MOE_SCORE_SOFTMAX) {
        float m = -INFINITY;
#pragma unroll
        for (int j = 0; j < KPL; ++j)
            if (lane + WAVE * j < E) m = fmaxf(m, l[j]);
#pragma unroll
        for (int o = 1; o < WAVE; o <<= 1) m = fmaxf(m, __shfl_xor(m, o));
#pragma unroll
        for (int j = 0; j < KPL; ++j) r.s[j] = m == -INFINITY ? (l[j] != l[j] ? l[j] : 0.0f) : expf(l[j] - m);
    } else {
#pragma unroll
        for (int j = 0; j < KPL; ++j) {
            // a = e^-|l|: neither direction overflows, and 1 - sigmoid keeps its digits
            const float a = expf(-fabsf(l[j])), h = __fdiv_rn(1.0f, 1.0f + a);
            const float sg = l[j] >= 0.0f ? h : a * h, one = l[j] >= 0.0f ? a * h : h;
            if (kind == MOE_SCORE_SIGMOID) {
                r.s[j] = l[j] != l[j] ? l[j] : sg;
                if (GRAD) r.ds[j] = sg * one;
            } else {
                r.s[j] = sqrtf((l[j] < 0.0f ? 0.0f : l[j]) + log1pf(a));
                if (GRAD) r.ds[j] = r.s[j] > 0.0f ? __fdiv_rn(0.5f * sg, r.s[j]) : 0.0f;
            }
        }
    }
    float sum = 0.0f;
#pragma unroll
    for (int j = 0; j < KPL; ++j) {
        if (lane + WAVE * j >= E) r.s[j] = 0.0f;
        sum += r.s[j];
    }
    sum = wave_sum(sum);
    r.inv = sum < 0x1p-126f ? 0.0f : __fdiv_rn(1.0f, sum);
}

template <int KPL>
__device__ __forceinline__ void load_row(const float* row, int E, float (&l)[KPL]) {
#pragma unroll
    for (int j = 0; j < KPL; ++j) {
        const int e = lane_id() + WAVE * j;
        l[j] = e < E ? row[e] : 0.0f;
    }
}

template <int KPL>
__global__ __launch_bounds__(BW * WAVE) void balance_kernel(BalanceArgs a) {
    __shared__ float part[BW][KPL * WAVE];
    __shared__ int hist[KPL * WAVE], alive[BW];
    const int tid = threadIdx.x, lane = lane_id(), wave = wave_index(), E = a.E;
    const int t1 = min(a.T, (int)(blockIdx.x + 1) * a.chunk);
    int t0 = blockIdx.x * a.chunk;
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
        for (int i = tid; i < E; i += BW * WAVE) hist[i] = 0;
        __syncthreads();
        float P[KPL];
        int n = 0;
#pragma unroll
        for (int j = 0; j < KPL; ++j) P[j] = 0.0f;
        for (int t = t0 + wave; t < e; t += BW) {
            if (a.mask && !a.mask[t]) continue;
            ++n;
            float l[KPL];
            Scores<KPL> r;
            load_row(a.logits + (size_t)t * E, E, l);
            for (int j = lane; j < a.k; j += WAVE) {
                const int x = a.idx[(size_t)t * a.k + j];
                if (x >= 0 && x < E) atomicAdd(&hist[x], 1);
            }
            token_scores<KPL, false>(l, E, a.score, r);
#pragma unroll
            for (int j = 0; j < KPL; ++j) P[j] += r.s[j] * r.inv;
        }
#pragma unroll
        for (int j = 0; j < KPL; ++j) part[wave][lane + WAVE * j] = P[j];
        if (lane == 0) alive[wave] = n;
        __syncthreads();
        const size_t slot = (size_t)(blockIdx.x + q);
        for (int i = tid; i < E; i += BW * WAVE) {
            float s = part[0][i];
#pragma unroll
            for (int w = 1; w < BW; ++w) s += part[w][i];
            a.sum[slot * E + i] = s;
            a.cnt[slot * E + i] = hist[i];
        }
        if (tid == 0) {
            int m = 0;
            for (int w = 0; w < BW; ++w) m += alive[w];
            a.num[slot] = m;
        }
        __syncthreads();
        t0 = e;
    }
}

// One sequence per workgroup: BW slot lanes x 64 experts at a time.
__global__ __launch_bounds__(BW * WAVE) void balance_join_kernel(BalanceArgs a) {
    __shared__ double sums[BW][WAVE];
    __shared__ int cnts[BW][WAVE];
    const int q = blockIdx.x, lane = lane_id(), wave = wave_index(), E = a.E;
    int b = 0, e = a.T;
    if (a.off) {
        b = max(0, min(a.off[q], a.T));
        e = max(b, min(a.off[q + 1], a.T));
    }
    const int c0 = b / a.chunk, c1 = e > b ? (e - 1) / a.chunk + 1 : c0;
    int n = 0;
    for (int c = c0 + lane; c < c1; c += WAVE) n += a.num[c + q];
#pragma unroll
    for (int o = 1; o < WAVE; o <<= 1) n += __shfl_xor(n, o);
    if (threadIdx.x == 0) a.tokens[q] = n;
    const double rn = n > 0 ? 1.0 / n : 0.0, rf = rn * E / a.k;
    double loss = 0.0;
    for (int i0 = 0; i0 < E; i0 += WAVE) {
        const int i = i0 + lane;
        double s = 0.0;
        int m = 0;
        if (i < E) {
            for (int c = c0 + wave; c < c1; c += BW) {
                s += (double)a.sum[(size_t)(c + q) * E + i];
                m += a.cnt[(size_t)(c + q) * E + i];
            }
        }
        sums[wave][lane] = s;
        cnts[wave][lane] = m;
        __syncthreads();
        if (wave == 0 && i < E) {
            for (int w = 1; w < BW; ++w) {
                s += sums[w][lane];
                m += cnts[w][lane];
            }
            a.prob[(size_t)q * E + i] = (float)(s * rn);
            a.counts[(size_t)q * E + i] = m;
            loss += (m * rf) * (s * rn);
        }
        __syncthreads();
    }
    if (wave == 0) {
        loss = wave_sum_f64(loss);
        if (lane == 0) a.loss[q] = (float)loss;
    }
}

constexpr int GW = 4;  // wavefronts per workgroup of the backward pass

template <int KPL>
__global__ __launch_bounds__(GW * WAVE) void route_backward_kernel(RouteGradArgs a) {
    const int lane = lane_id(), E = a.E;
    const int w0 = blockIdx.x * GW + wave_index();
    int q = -2, q_end = 0;  // the sequence of the last token, and its end
    float f[KPL], rate = 0.0f;
#pragma unroll
    for (int j = 0; j < KPL; ++j) f[j] = 0.0f;
    for (int t = w0 * a.chunk; t < min(a.T, (w0 + 1) * a.chunk); ++t) {
        float* out = a.d_logits + (size_t)t * E;
        if (q == -2 || t >= q_end) {
            q = 0;
            q_end = a.T;
            if (a.off) {
                q = seq_of(a.off, a.n_seq, t);
                q_end = q >= a.n_seq ? a.T : max(a.off[q + 1], t + 1);
                if (q >= a.n_seq) q = -1;
            }
            if (a.d_loss && q >= 0) {
                // f - 1: of the gradient's f - sum f p only differences of f count,
                // and small numbers lose less in them
                const int n = max(a.tokens[q], 1);
                const double rf = (double)E / ((double)a.k * n);
                rate = __fdiv_rn(a.d_loss[q], (float)n);
#pragma unroll
                for (int j = 0; j < KPL; ++j) {
                    const int e = lane + WAVE * j;
                    f[j] = e < E ? (float)(a.counts[(size_t)q * E + e] * rf - 1.0) : 0.0f;
                }
            }
        }
        if (q < 0 || (a.mask && !a.mask[t])) {  // no gradient
#pragma unroll
            for (int j = 0; j < KPL; ++j)
                if (lane + WAVE * j < E) out[lane + WAVE * j] = 0.0f;
            continue;
        }
        float l[KPL], g[KPL];
        Scores<KPL> r;
        load_row(a.logits + (size_t)t * E, E, l);
        token_scores<KPL, true>(l, E, a.score, r);
        const bool soft = a.score == MOE_SCORE_SOFTMAX;
        const float norm = soft ? r.inv : 1.0f;  // s as the router has it
#pragma unroll
        for (int j = 0; j < KPL; ++j) {
            r.s[j] *= norm;
            g[j] = 0.0f;
        }
        if (a.d_loss) {
            float fp = 0.0f;
            const float inv = soft ? 1.0f : r.inv;
#pragma unroll
            for (int j = 0; j < KPL; ++j) fp += f[j] * (r.s[j] * inv);
            fp = wave_sum(fp);
#pragma unroll
            for (int j = 0; j < KPL; ++j) g[j] = rate * (f[j] - fp) * inv;
        }
        if (a.d_w) {
            // lane j < k: the j-th selected expert (E: none), its score and weight's gradient
            const int x0 = lane < a.k ? a.idx[(size_t)t * a.k + lane] : E;
            const int x = x0 >= 0 && x0 < E ? x0 : E;
            float dw = x < E ? a.scale * a.d_w[(size_t)t * a.k + lane] : 0.0f, sel = 0.0f;
#pragma unroll
            for (int j = 0; j < KPL; ++j) {
                const float v = __shfl(r.s[j], x & 63);
                if (x >> 6 == j) sel = v;
            }
            if (x >= E) sel = 0.0f;
            if (a.normalise) {
                const float S = wave_sum(sel), rS = S < 0x1p-126f ? 0.0f : __fdiv_rn(1.0f, S);
                const float dot = wave_sum(dw * (sel * rS));
                dw = x < E ? (dw - dot) * rS : 0.0f;
            }
            for (int i = 0; i < a.k; ++i) {
                const int xi = __builtin_amdgcn_readlane(x, i);
                const float di = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(dw), i));
#pragma unroll
                for (int j = 0; j < KPL; ++j)
                    if (lane + WAVE * j == xi) g[j] += di;
            }
        }
        if (soft) {
            float dot = 0.0f;
#pragma unroll
            for (int j = 0; j < KPL; ++j) dot += g[j] * r.s[j];
            dot = wave_sum(dot);
#pragma unroll
            for (int j = 0; j < KPL; ++j) g[j] = r.s[j] * (g[j] - dot);
        } else {
#pragma unroll
            for (int j = 0; j < KPL; ++j) g[j] *= r.ds[j];
        }
#pragma unroll
        for (int j = 0; j < KPL; ++j)
            if (lane + WAVE * j < E) out[lane + WAVE * j] = g[j];
    }
}

}  // namespace

int balance_chunk(int T) {
    // whole rounds of a workgroup's wavefronts
    static_assert(BW == 16, "ranges of the workspace");
    const int per = (T + BALANCE_MAX_RANGES - 1) / BALANCE_MAX_RANGES;
    return (per + BW - 1) / BW * BW;
}

hipError_t launch_balance(const BalanceArgs& a, hipStream_t st) {
    const int grid = (a.T + a.chunk - 1) / a.chunk;
    if (a.E <= 256) balance_kernel<4><<<grid, BW * WAVE, 0, st>>>(a);
    else balance_kernel<16><<<grid, BW * WAVE, 0, st>>>(a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    balance_join_kernel<<<a.n_seq, BW * WAVE, 0, st>>>(a);
    return hipGetLastError();
}

hipError_t launch_route_backward(RouteGradArgs a, hipStream_t st) {
    a.chunk = a.T < 8192 ? 1 : a.T < 65536 ? 4 : 8;
    const int grid = (int)(((int64_t)a.T + GW * a.chunk - 1) / (GW * a.chunk));
    if (a.E <= 256) route_backward_kernel<4><<<grid, GW * WAVE, 0, st>>>(a);
    else route_backward_kernel<16><<<grid, GW * WAVE, 0, st>>>(a);
    return hipGetLastError();
}

}  // namespace moe
