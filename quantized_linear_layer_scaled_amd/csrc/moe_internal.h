// Internal declarations of the expert operators: routing, the rows sorted by
// expert, the experts' gated products and the combination of their outputs.
// Not part of the public interface (see include/qll.h).
#pragma once

#include "ffn_internal.h"

namespace qll {

enum Score : int { SCORE_SOFTMAX = 0, SCORE_SIGMOID = 1, SCORE_COUNT };

constexpr int kMoeMaxExperts = 1024;
constexpr int kMoeMaxTopk = 64;
// Waves of a launch that has one for each token or choice (a launch holds fewer
// than 2^32 threads); more of them take another launch, or a longer loop.
constexpr int kLaunchWaves = 1 << 25;

// The rows sorted by expert, for T x k choices (entry i = token i / k).
struct SortArgs {
    const int* ids;  // [T][k]
    int* offsets;    // [E + 1]
    int* rows;       // [T * k]: token of each sorted row, -1 behind the last
    int* places;     // [T][k]: sorted row of each choice, -1 for none
    int T, E, k;
    // counts per chunk of `chunk` tokens, [chunks][E]; unused for one workgroup
    int* hist;
    int chunk, chunks;
    int per;         // chunks per workgroup of the placing launch
};

struct RouteArgs {
    const void* logits;  // [T][E]
    int bf16;
    const float* bias;   // [E] or null
    int score;
    int groups, keep, group_best;
    int renorm;
    float scale;
    int* ids;
    float* weights;
    SortArgs sort;  // offsets null: ids and weights alone
};

struct RouteBackwardArgs {
    const void* logits;
    int bf16;
    int score, renorm;
    float scale;
    const int* ids;
    const float* dweights;
    void* dlogits;  // of the logits' type
    int T, E, k;
};

// Fills in the chunks; returns the bytes of `hist` (0: one workgroup).
int64_t moe_sort_plan(SortArgs& a);
hipError_t launch_moe_route(const RouteArgs& a, hipStream_t stream);
hipError_t launch_moe_sort(const SortArgs& a, hipStream_t stream);
hipError_t launch_moe_route_backward(const RouteBackwardArgs& a, hipStream_t stream);

struct CombineArgs {
    const uint16_t* y;     // bf16 [R][K]
    const int* places;     // [T][k]
    const float* weights;  // [T][k] or null (ones)
    const void* residual;  // [T][K] of out's type, or null
    void* out;             // [T][K]
    int fp32;              // type of residual, out and dout
    const void* dout;      // backward: [T][K]
    uint16_t* dy;          // bf16 [R][K] or null
    float* dweights;       // [T][k] or null
    int T, R, K, k;
};
hipError_t launch_moe_combine(const CombineArgs& a, hipStream_t stream);
hipError_t launch_moe_combine_backward(const CombineArgs& a, hipStream_t stream);

// The experts' gated products: f as for EPI_GATED with the weights and scales
// of expert 0 (the others follow), f.R rows sorted by expert, f.rows their
// tokens of `f.tokens`.
struct GroupedArgs {
    FfnArgs f;
    const int* offsets;  // [E + 1]
    int E;
};
// Whether a launch can hold the tiles.
bool moe_gated_fits(const GroupedArgs& a);
hipError_t launch_moe_gated(const GroupedArgs& a, hipStream_t stream);

}  // namespace qll
