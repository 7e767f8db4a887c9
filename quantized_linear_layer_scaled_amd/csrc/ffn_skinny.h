// Feed-forward products for few rows (R <= 64, decoding): out = epilogue of
// Q [R][K] times the weights P [C][K], bound by reading the weights once.
//
// A workgroup owns COLS output columns and its W waves split K: step s of 128
// bytes goes to wave s mod W, so the workgroup reads W * 128 consecutive bytes
// of each of its weight rows at a time.  Operands go from global memory to
// registers in the matrix cores' layout (the weights on the row side, the
// tokens on the column side), D steps in flight per wave.  The W partial sums
// are added through LDS in wave order.  The gated form puts 8 gate rows and 8
// up rows in one 16-row block; the linear form 16 rows, or 8 (the other half
// of the block repeats a row and is dropped) where 16 would leave compute
// units without a workgroup.
#pragma once

#include "ffn_epilogue.h"

namespace qll {

template <bool FP8, int EPI, int COLS, int TB, int W, int D>
__global__ __launch_bounds__(W * 64) void ffn_skinny_kernel(FfnArgs a)
{
    constexpr bool DUAL = EPI == EPI_GATED;
    static_assert(DUAL ? COLS == 8 : (COLS == 8 || COLS == 16), "columns of a workgroup");
    constexpr int THREADS = W * 64;
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int i = lane & 15, g = lane >> 4;
    const int c0 = blockIdx.x * COLS;
    const int kbytes = a.klen * (FP8 ? 1 : 2);

    // rows past the end repeat the last one: their outputs are not stored
    const int pc = min(c0 + (COLS == 8 ? (i & 7) : i), a.C - 1);
    const uint8_t* pp = (DUAL && i >= 8 ? a.P[1] : a.P[0]) + (size_t)pc * a.ldp;
    const uint8_t* qp[TB];
#pragma unroll
    for (int t = 0; t < TB; ++t)
        qp[t] = a.Q[0] + (size_t)min(16 * t + i, a.R - 1) * a.ldq;

    v4f acc[TB];
#pragma unroll
    for (int t = 0; t < TB; ++t)
        acc[t] = v4f{0, 0, 0, 0};

    auto mfma = [&](const uint4 (&p)[2], const uint4 (&q)[2], v4f c) __attribute__((always_inline)) {
        if constexpr (FP8) {
            return mfma_step<OP_FP8>(p, q, c);
        } else {
            c = mfma_step<OP_BF16>(&p[0], &q[0], c);
            return mfma_step<OP_BF16>(&p[1], &q[1], c);
        }
    };

    const int full = kbytes >> 7;
    for (int s0 = wave; s0 < full; s0 += W * D) {
        // (steps past the end load the last one again and are not multiplied)
        uint4 p[D][2], q[D][TB][2];
#pragma unroll
        for (int d = 0; d < D; ++d) {
            const int s = min(s0 + d * W, full - 1);
#pragma unroll
            for (int ks = 0; ks < 2; ++ks) {
                const int off = s * 128 + ks * 64 + g * 16;
                p[d][ks] = *(const uint4*)(pp + off);
#pragma unroll
                for (int t = 0; t < TB; ++t)
                    q[d][t][ks] = *(const uint4*)(qp[t] + off);
            }
        }
#pragma unroll
        for (int d = 0; d < D; ++d)
            if (s0 + d * W < full) {
#pragma unroll
                for (int t = 0; t < TB; ++t)
                    acc[t] = mfma(p[d], q[d][t], acc[t]);
            }
    }
    if ((kbytes & 127) && wave == full % W) {
        // the last, partial step: chunks past the end read as zeros
        uint4 p[2], q[TB][2];
#pragma unroll
        for (int ks = 0; ks < 2; ++ks) {
            const int off = full * 128 + ks * 64 + g * 16;
            const bool in = off < kbytes;
            const int at = in ? off : 0;
            const uint32_t keep = in ? 0xFFFFFFFFu : 0u;
            auto masked = [&](const uint8_t* from) __attribute__((always_inline)) {
                const uint4 v = *(const uint4*)from;
                return make_uint4(v.x & keep, v.y & keep, v.z & keep, v.w & keep);
            };
            p[ks] = masked(pp + at);
#pragma unroll
            for (int t = 0; t < TB; ++t)
                q[t][ks] = masked(qp[t] + at);
        }
#pragma unroll
        for (int t = 0; t < TB; ++t)
            acc[t] = mfma(p, q[t], acc[t]);
    }

    // partial sums [wave][token][16 block rows]
    __shared__ __attribute__((aligned(16))) float red[W][TB * 16][16];
#pragma unroll
    for (int t = 0; t < TB; ++t)
        *(float4*)&red[wave][t * 16 + i][g * 4] = make_float4(acc[t][0], acc[t][1], acc[t][2], acc[t][3]);
    __syncthreads();
#pragma unroll
    for (int e0 = 0; e0 < TB * 256; e0 += THREADS) {
        const int e = e0 + threadIdx.x;
        if (TB * 256 % THREADS != 0 && e >= TB * 256)
            break;
        const int row = e & 15, r = e >> 4;
        float v = 0.0f;
#pragma unroll
        for (int w = 0; w < W; ++w)
            v += red[w][r][row];
        const int c = c0 + row;
        if constexpr (DUAL) {
            const float u = __shfl_xor(v, 8, 64);  // (e and its lane share the low bits)
            if (row < 8 && c < a.C && r < a.R) {
                float gs = v, us = u;
                if (a.sq) {
                    gs = gs * a.sq[r] * a.sp[0][c];
                    us = us * a.sq[r] * a.sp[1][c];
                }
                with_act(a.act, [&](auto A) { gs = act_value<decltype(A)::value>(gs); });
                store_value(a, gs * us, r, c);
            }
        } else {
            if (row < COLS && c < a.C && r < a.R)
                store_value(a, linear_value(a, v, r, c), r, c);
        }
    }
}

}  // namespace qll
