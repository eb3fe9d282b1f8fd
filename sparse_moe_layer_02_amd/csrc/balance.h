// balance.h - internal launch interface of the balance loss and the routing's
// gradient (balance.hip).
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace moe {

struct BalanceArgs {
    const float* logits;   // [T, E]
    const int32_t* idx;    // [T, k]
    const uint8_t* mask;   // [T] or null
    const int32_t* off;    // [n_seq + 1] or null: one sequence of all tokens
    int T, E, k, score, n_seq;
    int chunk;             // tokens per workgroup (balance_chunk)
    float* sum;            // [slots, E up to a multiple of 4] workspace; slots = ceil(T / chunk) + n_seq
    int32_t* cnt;          // the same
    int32_t* num;          // [slots] tokens
    double* loss_part;     // [n_seq, blocks of 64 experts]
    int32_t* done;         // [n_seq] blocks that have ended
    int32_t* counts;       // [n_seq, E]
    int32_t* tokens;       // [n_seq]
    float* prob;           // [n_seq, E]
    float* loss;           // [n_seq]
    int blocks;            // set by the launcher
    bool one_launch;       // the same
};
constexpr int BALANCE_MAX_RANGES = 512;  // workgroups of the first launch, at most
constexpr int BALANCE_MAX_K = 32;
int balance_chunk(int T, int E, int n_seq);
hipError_t launch_balance(BalanceArgs a, hipStream_t st);

struct RouteGradArgs {
    const float* logits;
    const int32_t* idx;
    const float* d_w;       // [T, k] or null
    const uint8_t* mask;
    const int32_t* off;
    const int32_t* counts;  // with d_loss
    const int32_t* tokens;
    const float* d_loss;    // [n_seq] or null
    float* d_logits;        // [T, E]
    int T, E, k, score, n_seq, normalise;
    float scale;
    int chunk;              // rounds of a wavefront, set by the launcher
};
hipError_t launch_route_backward(RouteGradArgs a, hipStream_t st);

}  // namespace moe
