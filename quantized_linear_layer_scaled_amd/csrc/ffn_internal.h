// Internal declarations of the feed-forward operators: matrix products with
// bias, activation and residual, gated projections, their backward passes and
// the residual norms.  Not part of the public interface (see include/qll.h).
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace qll {

// Activation codes, as in qll_act.
enum Act : int { ACT_NONE = 0, ACT_RELU, ACT_GELU, ACT_GELU_TANH, ACT_SILU, ACT_SIGMOID, ACT_COUNT };

// What a product does with its sums.
enum FfnEpi : int {
    EPI_LINEAR = 0,  // out = act(sum * sq[r] * sp[c] + bias[c]) + res[r][c]
    EPI_GATED,       // out = act(g) * u
    EPI_DZ,          // out = dy * act'(sum + bias[c]), column sums of out to `partial`
    EPI_DGATED,      // out[r][c] = dy * u * act'(g), out[r][C + c] = dy * act(g)
    EPI_PLAIN,       // out = sum (rows from row_split on to out2)
    EPI_PARTIAL,     // Split-K: fp32 sums to `partial` [split][R][C]
    EPI_GROUPED      // EPI_GATED, the scale of row r being sq[rows[r]]
};

// out[r][c] = epilogue(sum_k Q[r][k] P[c][k]).  P holds the operand along the
// output's columns, Q the one along its rows.  An operand is K-contiguous
// ([row][k], `ld` bytes from row to row) or K-strided ([k][row], `ld` bytes
// from k to k).  With nseg = 2 the contraction runs over (P[0], Q[0]) and then
// (P[1], Q[1]), `klen` elements each.  Gated: P[0] and P[1] are the gate and
// up weights, of C rows each.
struct FfnArgs {
    const uint8_t* P[2];
    const uint8_t* Q[2];
    int64_t ldp, ldq;
    int C, R;
    int klen;      // elements of the contraction per segment
    int nseg;
    int nks;       // K stages per segment
    int splits;    // Split-K pieces (EPI_PARTIAL), `per` stages each
    int per;
    void* out;     // [R][ldo]
    void* out2;    // rows >= row_split go here (as row r - row_split)
    int row_split;
    int64_t ldo;   // elements
    int out_fp32;
    int act;
    const float* sq;        // [R]: FP8 scales of the rows
    const int* rows;        // EPI_GROUPED: [R] or null (r itself)
    int tokens;             // entries of sq there
    const float* sp[2];     // [C]: FP8 scales of the columns
    const uint16_t* bias;   // bf16 [C] or null
    const uint16_t* res;    // bf16 [R][C] or null
    const uint16_t* dy;     // bf16 [R][C]
    float* partial;
};

// Layouts of a product (the second template axis of the tile kernels).
enum FfnLayout : int {
    LAY_NT = 0,  // P and Q K-contiguous (forward products)
    LAY_NN,      // P K-strided, Q K-contiguous (gradient of the input)
    LAY_TN       // both K-strided (gradient of the weights)
};

// Rows of `partial` that EPI_DZ writes: strips of rows whose column sums it
// forms, for the tile the launch picks for (R, C).
int ffn_dz_strips(int64_t R, int64_t C);
// Split-K pieces that the launch of a bf16 input-gradient or linear product
// uses for (R, C, stages), 1 = none.
int ffn_splits(int64_t R, int64_t C, int64_t stages);

hipError_t ffn_launch(int fp8, int layout, int epi, FfnArgs a, hipStream_t stream);
// The input's (LAY_NN) and the weights' (LAY_TN) gradient in one launch,
// where ffn_pair_fits.
bool ffn_pair_fits(const FfnArgs& in, const FfnArgs& w);
hipError_t ffn_launch_pair(const FfnArgs& in, const FfnArgs& w, hipStream_t stream);
// Sum of the Split-K pieces followed by EPI_LINEAR.
hipError_t ffn_launch_reduce(const FfnArgs& a, hipStream_t stream);
// Few rows: one pass over the weights, K split over the waves of a workgroup.
// EPI_LINEAR or EPI_GATED, both operands K-contiguous; R <= 32, and
// ffn_skinny_fits says where it is the way to go.
bool ffn_skinny_fits(int epi, int64_t R, int64_t C, int64_t kbytes);
hipError_t ffn_launch_skinny(int fp8, int epi, const FfnArgs& a, hipStream_t stream);

// Column sums of bf16 x [R][C] over strips of kColsumRows rows -> fp32
// partial [strips][C], and the sum of such partials over the strips.
constexpr int kColsumRows = 64;
hipError_t launch_colsum_strips(const void* x, float* partial, int64_t R, int64_t C,
                                hipStream_t stream);
// out[p][c] = sum over strips of partial[p][strip][c]; planes with a null
// out are skipped.
struct ColsumArgs {
    const float* partial;
    int strips, C;
    float* out[3];
};
hipError_t launch_colsum_finish(const ColsumArgs& a, int planes, hipStream_t stream);

// Residual norms (see residual_norm in include/qll.h).
struct NormArgs {
    const uint16_t* y;      // bf16 [M][K] or null
    const void* r;          // [M][K] bf16 or fp32
    const uint16_t* w_post; // bf16 [K] or null
    const uint16_t* gate;   // bf16 [K] or null
    const uint16_t* w_pre;  // bf16 [K]
    void* r_out;            // [M][K], type of r (null without y)
    void* n_out;            // bf16 or e4m3 [M][K]
    float* n_scales;        // [M] (e4m3)
    // backward
    const uint16_t* dn;     // bf16 [M][K]
    const void* dr_out;     // [M][K], type of r, or null
    uint16_t* dy;           // bf16 [M][K] (null without y)
    void* dr;               // [M][K], type of r
    float* partial;         // [3][blocks][K]: dw_pre, dw_post, dgate sums
    float* stats;           // [M][4]: 1 / rms(y), 1 / rms(h), mean term (long rows)
    float alpha, beta, eps;
    int M, K;
    int r_fp32, quant;
};
constexpr int kNormMaxK = 32768;
hipError_t launch_residual_norm(const NormArgs& a, hipStream_t stream);
// Rows of each partial sum, and floats of statistics, of the backward pass.
int norm_backward_blocks(int64_t M, int64_t K);
int64_t norm_backward_stats(int64_t M, int64_t K);
hipError_t launch_residual_norm_backward(const NormArgs& a, hipStream_t stream);

}  // namespace qll
