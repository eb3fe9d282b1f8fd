// kernels.h - internal launch interface between the C-ABI host code (api.hip)
// and the kernel files.  Every launcher enqueues on the given stream and
// returns hipGetLastError().
#pragma once
#include <hip/hip_ext.h>
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "common.h"

namespace moe {

// Kernel timing of one stage: `start` receives the start timestamp of the
// stage's first kernel dispatch, `stop` the end timestamp of its last
// (hipExtLaunchKernel events, taken from the dispatch itself, so launch gaps
// before and after the stage are not counted).  Either may be null.
struct KTime {
    hipEvent_t start = nullptr, stop = nullptr;
    KTime first() const { return KTime{start, nullptr}; }
    KTime last() const { return KTime{nullptr, stop}; }
};

template <typename... KArgs, typename... Args>
inline void launch_kernel(void (*kern)(KArgs...), dim3 grid, dim3 block, hipStream_t st, const KTime& kt,
                          Args... args) {
    if (kt.start || kt.stop) hipExtLaunchKernelGGL(kern, grid, block, 0, st, kt.start, kt.stop, 0, args...);
    else kern<<<grid, block, 0, st>>>(args...);
}

struct RouteArgs {
    const void* x;
    const float* wr;
    int T, d, E, act;
    float* logits;
    bool force_gemm;  // use the tiled prefill kernel even for few tokens
};
hipError_t launch_router_logits(const RouteArgs& a, hipStream_t st, const KTime& kt = KTime());

struct SelectArgs {
    const float* logits;
    const float* bias;
    int T, E, k, score;
    float route_scale;
    int32_t* topk_idx;
    float* topk_w;
    bool generic_only;  // skip the compile-time 256-expert instantiation
};
hipError_t launch_topk(const SelectArgs& a, hipStream_t st, const KTime& kt = KTime());

// Expert groups of a selection; n_group 1 is the flat one.
struct GroupArgs {
    int n_group = 1, topk_group = 1, group_top = 1, normalise = 1;
    float inv_size = 0.0f;  // n_group / n_expert
};
hipError_t launch_group_topk(const SelectArgs& a, const GroupArgs& g, hipStream_t st, const KTime& kt = KTime());

// Rows [rows, cols] (row stride ldx elements) to codes [rows, cols] and scale
// bytes [rows, f8_scale_ld(cols)].
struct QuantArgs {
    const void* x;
    int xdt;  // MOE_DT_F32 or MOE_DT_BF16
    int rows, cols;
    int64_t ldx;
    uint8_t *q, *e;
};
hipError_t launch_quantize_rows(const QuantArgs& a, hipStream_t st, const KTime& kt = KTime());

// Dense product out[m, n] = x[m, k] w[n, k]^T of e4m3 operands.
struct BlockArgs {
    const uint8_t *xq, *xe;  // [m, k] codes, [m, f8_scale_ld(k)] scale bytes (or rows of xdt and null)
    const uint8_t* wq;       // [n, k]
    const float* ws;         // [ceil(n / 128), ceil(k / 128)]
    int m, n, k;
    void* out;               // [m, n]
    int odt;                 // MOE_DT_F32 or MOE_DT_BF16
    int xdt = MOE_DT_F8B128; // where block_matmul_takes says so, MOE_DT_F32 or MOE_DT_BF16
};
bool block_matmul_takes(int xdt, int m, int n);
hipError_t launch_block_matmul(const BlockArgs& a, hipStream_t st);
hipError_t launch_block_matmul_tile(const BlockArgs& a, hipStream_t st);  // many rows

// Rows [rows, cols] (row stride ldx elements) to int8 codes (row stride ldq) and
// one scale per row; from row rows0 on, rows have cols1 columns.
struct TokenQuantArgs {
    const void* x;
    int xdt;  // MOE_DT_F32 or MOE_DT_BF16
    int64_t rows, rows0;
    int cols, cols1;
    int64_t ldx, ldq;
    int8_t* q;
    float* s;
};
hipError_t launch_quantize_tokens(const TokenQuantArgs& a, hipStream_t st, const KTime& kt = KTime());

// Dense product out[m, n] = x[m, k] w[n, k]^T of int8 codes.
struct ChannelArgs {
    const void* x;     // [m, k] codes (or rows of xdt)
    const float* xs;   // [m]
    const int8_t* wq;  // [n, k]
    const float* ws;   // [n]
    int m, n, k;
    void* out;         // [m, n]
    int odt;           // MOE_DT_F32 or MOE_DT_BF16
    int xdt = MOE_DT_I8CH;  // where channel_matmul_takes says so, MOE_DT_F32 or MOE_DT_BF16 rows (xs unused)
};
bool channel_matmul_takes(int m, int n, int k);
hipError_t launch_channel_matmul(const ChannelArgs& a, hipStream_t st);
hipError_t launch_channel_matmul_tile(const ChannelArgs& a, hipStream_t st);  // many rows

struct PermArgs {
    const int32_t* topk_idx;
    int T, k, E;
    int n_shared;
    int32_t* offsets;    // [E+1] (read-only for launch_lists_from_offsets)
    int32_t* perm_rows;  // [T*k]
    int32_t* inv_perm;   // [T*k]
    int32_t* blk_hist;   // [n_blk, E]
    int32_t* blk_base;   // [n_blk, E]
    int32_t* meta;       // META_WORDS
    int32_t* active;     // [E] experts with rows, ascending
    int2* tiles;         // [max_tiles] (group, first row) for the grouped GEMM
    int n_blk;
    int bm;              // tile rows for the tile list
};
hipError_t launch_permute(const PermArgs& a, hipStream_t st, const KTime& kt = KTime());
// active / tile lists from existing offsets (offsets and perm_rows untouched)
hipError_t launch_lists_from_offsets(const PermArgs& a, hipStream_t st, const KTime& kt = KTime());

// One expert slot of the decode path, written by the selection kernel and read
// by the decode expert kernels in a single dependent load.  Slot 0 is the
// shared expert when there is one (e = 0, shared = 1, tokens 0..T-1, weight
// 1); the routed slots follow in ascending expert index.  Slots past the last
// active expert carry e = -1.
struct DecodeSlot {
    int32_t e;       // expert index, -1 for an unused slot
    int32_t r0;      // first row of the slot in h
    int32_t m;       // tokens routed to the slot (h rows r0 .. r0+m-1)
    int32_t shared;  // 1 for the shared expert
    int32_t tok[MOE_DECODE_MAX_TOKENS];  // token of h row r0+i
    float w[MOE_DECODE_MAX_TOKENS];      // routing weight of that row (1 for the shared expert)
};

// One set of expert weights for the FFN kernels.
struct MatRef {
    const void* q;
    const uint16_t* scale;
};

struct FfnArgs {
    const void* x;          // [T, d]
    MatRef gate, up, down;  // routed [E, F, d], [E, F, d], [E, d, F]
    MatRef s_gate, s_up, s_down;
    const int32_t* offsets;
    const int32_t* perm_rows;
    const float* topk_w;
    const int32_t* meta;    // n_active at [0], n_tiles at [1]
    const int32_t* active;  // active experts, ascending
    const int2* tiles;
    int T, d, E, k, F, Fs, n_shared, act, wdt;
    void* h;                // [T*k + T*n_shared, ldh] in the activation format
    int ldh;                // max(F, Fs)
    float* slot_out;        // [T*k, d]
    float* shared_out;      // [T, d]
    float* y;               // [T, d] (fused combine)
    int max_tiles;          // grid bound of the grouped GEMMs (tiles of bm rows)
    int bm;                 // rows per grouped-GEMM tile: 64, 128 or 256
    int shared_done;        // the shared expert's h rows were already produced (decode route kernel)
    DecodeSlot* dslots;     // decode slot table (decode path only)
    int n_dslots;           // its capacity: n_shared + min(E, T*k)
    int grid_has_shared;    // set by the launchers: the last grid slot is the shared expert
};
// gate/up GEMV over the active experts (and the shared one) -> h
hipError_t launch_gateup_gemv(const FfnArgs& a, hipStream_t st, const KTime& kt = KTime());
// gate/up GEMV of the decode path over the routed slots of the decode slot table
hipError_t launch_gateup_gemv_decode(const FfnArgs& a, hipStream_t st, const KTime& kt = KTime());
// down GEMV writing weighted slot rows and the shared rows
hipError_t launch_down_slots_gemv(const FfnArgs& a, hipStream_t st, const KTime& kt = KTime());
// grouped bf16 MFMA GEMMs (prefill)
hipError_t launch_gateup_mfma(const FfnArgs& a, hipStream_t st, const KTime& kt = KTime());
hipError_t launch_down_mfma(const FfnArgs& a, hipStream_t st, const KTime& kt = KTime());
hipError_t launch_gateup_dma(const FfnArgs& a, hipStream_t st, const KTime& kt = KTime());
// grouped MFMA GEMMs for int8 (blocks of 32 + fp16 scale) weights, 64- or 128-row tiles
hipError_t launch_gateup_mfma_q8(const FfnArgs& a, hipStream_t st, const KTime& kt = KTime());
hipError_t launch_down_mfma_q8(const FfnArgs& a, hipStream_t st, const KTime& kt = KTime());
bool q8_dma_ok(const FfnArgs& a);
hipError_t launch_gateup_q8_dma(const FfnArgs& a, hipStream_t st, const KTime& kt = KTime());
hipError_t launch_down_q8_dma(const FfnArgs& a, hipStream_t st, const KTime& kt = KTime());
hipError_t launch_down_dma(const FfnArgs& a, hipStream_t st, const KTime& kt = KTime());

// Experts with e4m3 weights: rows of x and h as codes and scale bytes.
struct F8Ffn {
    FfnArgs f;               // h unused; ldh is the row stride of hq
    uint8_t *xq, *xe;        // [T, d], [T, f8_scale_ld(d)]
    uint8_t *hq, *he;        // [T*k + T*n_shared, ldh], [.., f8_scale_ld(ldh)]
};
// Experts with int8 codes and one scale per weight row.
struct I8Ffn {
    FfnArgs f;    // h unused; ldh is the row stride of h and hq
    int8_t* xq;   // [T, d]
    float* xs;    // [T]
    float* h;     // [T*k + T*n_shared, ldh] fp32
    int8_t* hq;   // the same as codes
    float* hs;    // their rows' scales
};
hipError_t launch_i8_gateup(const I8Ffn& a, hipStream_t st, const KTime& kt = KTime());
hipError_t launch_i8_down(const I8Ffn& a, hipStream_t st, const KTime& kt = KTime());
// The same for few tokens, each at most once with an expert (a selection's): h, and
// y from h's quantised rows with the combine.
bool i8_stream_takes(int T);
hipError_t launch_i8_gateup_stream(const I8Ffn& a, hipStream_t st, const KTime& kt = KTime());
hipError_t launch_i8_down_stream(const I8Ffn& a, void* y, int ydt, hipStream_t st, const KTime& kt = KTime());
// Selection, grouping and quantisation of x (bf16) in one launch, for up to
// F8_ROUTE_MAX_T tokens.
constexpr int F8_ROUTE_MAX_T = 16;
hipError_t launch_f8_router(const RouteArgs& a, hipStream_t st, const KTime& kt = KTime());  // their logits (bf16 x)
hipError_t launch_f8_route(const SelectArgs& s, const GroupArgs& g, bool grouped, const PermArgs& p, const QuantArgs& q,
                           hipStream_t st, const KTime& kt = KTime());
hipError_t launch_i8_route(const SelectArgs& s, const GroupArgs& g, bool grouped, const PermArgs& p, const TokenQuantArgs& q,
                           hipStream_t st, const KTime& kt = KTime());
hipError_t launch_f8_gateup(const F8Ffn& a, hipStream_t st, const KTime& kt = KTime());
hipError_t launch_f8_down(const F8Ffn& a, hipStream_t st, const KTime& kt = KTime());

// The decode path (T <= MOE_DECODE_MAX_TOKENS) in four launches: router;
// selection + grouping beside the shared gate/up; routed gate/up; down +
// combine into f.y.  kt[s] times stage s (MOE_STAGES entries); the decode
// path launches nothing for the permutation and combine stages.
struct DecodeRouteArgs {
    RouteArgs r;
    SelectArgs s;
    PermArgs p;
    FfnArgs f;
    float* scores;  // [T, E] fp32 router scores (workspace)
    GroupArgs g;
    bool grouped;   // selection with groups or softmax scores, from the logits
};
hipError_t launch_decode(const DecodeRouteArgs& a, const KTime* kt, hipStream_t st);

struct CombineArgs {
    const float* slot_out;
    const float* shared_out;
    void* y;        // [T, d] of ydt
    int T, k, d;
    int ydt = MOE_DT_F32;  // or MOE_DT_BF16
};
hipError_t launch_combine(const CombineArgs& a, hipStream_t st, const KTime& kt = KTime());

}  // namespace moe
