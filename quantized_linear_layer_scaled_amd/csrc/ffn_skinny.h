// Feed-forward products for few rows (R <= 32, decoding): out = epilogue of
// Q [R][K] times the weights P [C][K], bound by reading the weights once.
//
// A workgroup owns COLS output columns and its W waves split K: step s of 128
// bytes goes to wave s mod W, so the workgroup reads W * 128 consecutive bytes
// of each of its weight rows at a time.  Operands go from global memory to
// registers in the matrix cores' layout (the weights on the row side, the
// tokens on the column side).  The W partial sums are added through LDS in
// wave order.  Past 16 rows a second block of tokens (TB = 2) meets the same
// weight registers.  Measured and not kept (M = 1 to 16, N = 2048 to 12288): two
// or four steps in flight per wave, 4 or 16 waves, two or four blocks of columns
// per workgroup; each wins up to 8% on some size and loses as much or more on
// others (N = 2048, K = 6144, M = 4, bf16: 8.9 us, the others 8.8 to 21; gated
// N = 12288, K = 4096, M = 1: 38.8 us = 5.2 TB/s, the others 35.8 to 62).  The
// gated form puts 8 gate rows and 8 up rows in one 16-row block; the linear
// form 16 rows, or 8 (the other half of the block stays zero) where 16 would
// leave compute units without a workgroup.
#pragma once

#include "ffn_epilogue.h"

namespace qll {

template <bool FP8, int EPI, int COLS, int TB, int W>
__global__ __launch_bounds__(W * 64) void ffn_skinny_kernel(FfnArgs a)
{
    constexpr bool DUAL = EPI == EPI_GATED;
    static_assert(DUAL ? COLS == 8 : (COLS == 8 || COLS == 16), "columns of a block");
    static_assert(W >= 4 * TB, "a thread per sum");
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int i = lane & 15, g = lane >> 4;
    const int c0 = blockIdx.x * COLS;
    const int kbytes = a.klen * (FP8 ? 1 : 2);

    // A lane's row of each operand, as a byte offset of its 16-byte chunk g; a
    // lane without one reads zeros (an offset out of range).  The gated form's
    // weights are two matrices, so its lanes keep addresses instead, and those
    // past the end repeat the last row (their sums are not stored).
    const __amdgpu_buffer_rsrc_t rp = __builtin_amdgcn_make_buffer_rsrc(
        (void*)(a.P[0] + (size_t)c0 * a.ldp), (short)0,
        (int)(min(a.C - c0, COLS) * (int)a.ldp), 0x00020000);
    const __amdgpu_buffer_rsrc_t rq =
        __builtin_amdgcn_make_buffer_rsrc((void*)a.Q[0], (short)0, a.R * (int)a.ldq, 0x00020000);
    const int row = COLS == 8 ? (i & 7) : i;
    const uint8_t* pp = (i >= 8 ? a.P[1] : a.P[0]) + (size_t)min(c0 + row, a.C - 1) * a.ldp + g * 16;
    const uint32_t vp = i < COLS ? (uint32_t)row * (uint32_t)a.ldp + g * 16 : kOutOfRange;
    uint32_t vq[TB];
    v4f acc[TB];
#pragma unroll
    for (int t = 0; t < TB; ++t) {
        const int r = 16 * t + i;
        vq[t] = r < a.R ? (uint32_t)r * (uint32_t)a.ldq + g * 16 : kOutOfRange;
        acc[t] = v4f{0, 0, 0, 0};
    }
    const int steps = (kbytes + 127) >> 7;
    for (int s = wave; s < steps; s += W) {
        uint4 p[2], q[TB][2];
#pragma unroll
        for (int ks = 0; ks < 2; ++ks) {
            const int off = s * 128 + ks * 64;
            const bool in = off + g * 16 < kbytes;  // else past the row's end: zeros
            if constexpr (DUAL) {
                const uint32_t keep = in ? 0xFFFFFFFFu : 0u;
                const uint4 v = *(const uint4*)(pp + (in ? off : -16 * g));
                p[ks] = make_uint4(v.x & keep, v.y & keep, v.z & keep, v.w & keep);
            } else {
                p[ks] = __builtin_bit_cast(uint4, __builtin_amdgcn_raw_buffer_load_b128(
                                                      rp, (int)(in ? vp + off : kOutOfRange), 0, 0));
            }
#pragma unroll
            for (int t = 0; t < TB; ++t)
                q[t][ks] = __builtin_bit_cast(
                    uint4, __builtin_amdgcn_raw_buffer_load_b128(
                               rq, (int)(in ? vq[t] + off : kOutOfRange), 0, 0));
        }
#pragma unroll
        for (int t = 0; t < TB; ++t) {
            if constexpr (FP8) {
                acc[t] = mfma_step<OP_FP8>(p, q[t], acc[t]);
            } else {
                acc[t] = mfma_step<OP_BF16>(&p[0], &q[t][0], acc[t]);
                acc[t] = mfma_step<OP_BF16>(&p[1], &q[t][1], acc[t]);
            }
        }
    }

    // partial sums [wave][token][block row]
    __shared__ __attribute__((aligned(16))) float red[W][TB * 16][16];
#pragma unroll
    for (int t = 0; t < TB; ++t)
        *(float4*)&red[wave][16 * t + i][g * 4] =
            make_float4(acc[t][0], acc[t][1], acc[t][2], acc[t][3]);
    __syncthreads();
    if (threadIdx.x < TB * 256) {
        const int br = threadIdx.x & 15, r = threadIdx.x >> 4;
        float v = 0.0f;
#pragma unroll
        for (int w = 0; w < W; ++w)
            v += red[w][r][br];
        const int c = c0 + br;
        if constexpr (DUAL) {
            const float u = __shfl_xor(v, 8, 64);
            if (br < 8 && c < a.C && r < a.R) {
                float gs = v, us = u;
                if (a.sq) {
                    gs = gs * a.sq[r] * a.sp[0][c];
                    us = us * a.sq[r] * a.sp[1][c];
                }
                with_act(a.act, [&](auto A) { gs = act_value<decltype(A)::value>(gs); });
                store_value(a, gs * us, r, c);
            }
        } else {
            if (br < COLS && c < a.C && r < a.R)
                store_value(a, linear_value(a, v, r, c), r, c);
        }
    }
}

}  // namespace qll
