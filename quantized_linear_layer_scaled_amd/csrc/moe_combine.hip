// Combination of the experts' outputs for gfx950:
//
//   out[t] = residual[t] + sum_j w[t][j] y[places[t][j]]
//   backward: dy[places[t][j]] = w[t][j] dout[t],  dw[t][j] = <dout[t], y[places[t][j]]>
//
// Bound by HBM.  A choice without a row (place -1) adds nothing and gets a
// zero gradient.
#include "ffn_epilogue.h"
#include "moe_internal.h"

namespace qll {

namespace {

template <bool F32>
__device__ __forceinline__ void load8(const void* p, size_t at, float* f)
{
    if constexpr (F32) {
        const float4 a = *(const float4*)((const float*)p + at), b = *(const float4*)((const float*)p + at + 4);
        f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
        f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
    } else {
        load_bf16<8>((const uint16_t*)p + at, f);
    }
}

// A thread per 8 columns of a token.
template <bool F32>
__global__ __launch_bounds__(256) void moe_combine_kernel(CombineArgs a)
{
    const int vectors = a.K / 8;
    const int64_t total = (int64_t)a.T * vectors;
    for (int64_t at = (int64_t)blockIdx.x * 256 + threadIdx.x; at < total; at += (int64_t)gridDim.x * 256) {
    const int64_t t = at / vectors;
    const int c = (int)(at - t * vectors) * 8;
    float sum[8];
    if (a.residual) {
        load8<F32>(a.residual, (size_t)t * a.K + c, sum);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            sum[e] = 0.0f;
    }
    for (int j = 0; j < a.k; ++j) {
        const int r = a.places[t * a.k + j];
        if ((unsigned)r >= (unsigned)a.R)
            continue;
        const float w = a.weights ? a.weights[t * a.k + j] : 1.0f;
        float y[8];
        load_bf16<8>(a.y + (size_t)r * a.K + c, y);
#pragma unroll
        for (int e = 0; e < 8; ++e)
            sum[e] += w * y[e];
    }
    if constexpr (F32)
        store_f32<8>((float*)a.out + (size_t)t * a.K + c, sum);
    else
        store_bf16<8>((uint16_t*)a.out + (size_t)t * a.K + c, sum);
    }
}

// A wave per choice; the choices of a token share a workgroup's L1.
template <bool F32>
__global__ __launch_bounds__(256) void moe_combine_backward_kernel(CombineArgs a)
{
    const int lane = threadIdx.x & 63;
    const int64_t i = (int64_t)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    if (i >= (int64_t)a.T * a.k)
        return;
    const int64_t t = i / a.k;
    const int r = a.places[i];
    float dot = 0.0f;
    if ((unsigned)r < (unsigned)a.R) {
        const float w = a.weights ? a.weights[i] : 1.0f;
        for (int c = lane * 8; c < a.K; c += 512) {
            float d[8], y[8];
            load8<F32>(a.dout, (size_t)t * a.K + c, d);
            if (a.dweights) {
                load_bf16<8>(a.y + (size_t)r * a.K + c, y);
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    dot += d[e] * y[e];
            }
            if (a.dy) {
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    d[e] *= w;
                store_bf16<8>(a.dy + (size_t)r * a.K + c, d);
            }
        }
    }
    if (a.dweights) {
#pragma unroll
        for (int s = 1; s < 64; s <<= 1)
            dot += __shfl_xor(dot, s, 64);
        if (lane == 0)
            a.dweights[i] = dot;
    }
}

}  // namespace

hipError_t launch_moe_combine(const CombineArgs& a, hipStream_t stream)
{
    // (a launch holds fewer than 2^32 threads)
    const int64_t all = ((int64_t)a.T * (a.K / 8) + 255) / 256;
    const int64_t blocks = all < (1 << 23) ? all : 1 << 23;
    if (a.fp32)
        moe_combine_kernel<true><<<(unsigned)blocks, 256, 0, stream>>>(a);
    else
        moe_combine_kernel<false><<<(unsigned)blocks, 256, 0, stream>>>(a);
    return hipGetLastError();
}

hipError_t launch_moe_combine_backward(const CombineArgs& a, hipStream_t stream)
{
    const int64_t blocks = ((int64_t)a.T * a.k + 3) / 4;
    if (a.fp32)
        moe_combine_backward_kernel<true><<<(unsigned)blocks, 256, 0, stream>>>(a);
    else
        moe_combine_backward_kernel<false><<<(unsigned)blocks, 256, 0, stream>>>(a);
    return hipGetLastError();
}

}  // namespace qll
