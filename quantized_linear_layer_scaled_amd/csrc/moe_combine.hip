// Combination of the experts' outputs for gfx950:
//
//   out[t] = residual[t] + sum_j w[t][j] y[places[t][j]]
//   backward: dy[places[t][j]] = w[t][j] dout[t],  dw[t][j] = <dout[t], y[places[t][j]]>
//
// Bound by HBM.  A choice without a row (place -1) adds nothing and gets a
// zero gradient.
#include "ffn_epilogue.h"
#include "moe_internal.h"
#include "quant_encode.h"

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

// A thread per 8 columns of a token; the rows of FOUR choices are under way at a
// time.  ALIGNED: topk is a multiple of four, so places and weights come as
// vectors.  (One choice at a time, each behind its place: T = 4093, top-8,
// K = 4104 70 us; this way 65, 5.2 TB/s.)
template <bool F32, bool ALIGNED>
__global__ __launch_bounds__(256) void moe_combine_kernel(CombineArgs a)
{
    constexpr int FOUR = 4;
    const int vectors = a.K / 8;
    const int64_t total = (int64_t)a.T * vectors;
    for (int64_t at = (int64_t)blockIdx.x * 256 + threadIdx.x; at < total;
         at += (int64_t)gridDim.x * 256) {
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
        for (int j = 0; j < a.k; j += FOUR) {
            int r[FOUR];
            float w[FOUR];
            const int* places = a.places + t * a.k + j;
            const float* weights = a.weights + t * a.k + j;
            if constexpr (ALIGNED) {
                const int4 p = *(const int4*)places;
                r[0] = p.x; r[1] = p.y; r[2] = p.z; r[3] = p.w;
                const float4 f = a.weights ? *(const float4*)weights : make_float4(1.0f, 1.0f, 1.0f, 1.0f);
                w[0] = f.x; w[1] = f.y; w[2] = f.z; w[3] = f.w;
            } else {
#pragma unroll
                for (int i = 0; i < FOUR; ++i) {
                    const int to = min(i, a.k - 1 - j);
                    r[i] = j + i < a.k ? places[to] : -1;
                    w[i] = a.weights ? weights[to] : 1.0f;
                }
            }
            uint4 y[FOUR];
#pragma unroll
            for (int i = 0; i < FOUR; ++i)
                if ((unsigned)r[i] < (unsigned)a.R)
                    y[i] = *(const uint4*)(a.y + (size_t)r[i] * a.K + c);
#pragma unroll
            for (int i = 0; i < FOUR; ++i)
                if ((unsigned)r[i] < (unsigned)a.R) {
                    float f[8];
                    unpack8(y[i], f);
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        sum[e] += w[i] * f[e];
                }
        }
        if constexpr (F32)
            store_f32<8>((float*)a.out + (size_t)t * a.K + c, sum);
        else
            store_bf16<8>((uint16_t*)a.out + (size_t)t * a.K + c, sum);
    }
}

// A wave per choice, U vectors of its row under way; the choices of a token share
// a workgroup's L1.  dy is stored past L2 where it does not fit (T = 4096, top-8,
// K = 2048: one vector at a time 65 us; several 61.5; and past L2 58.2, 4.9 TB/s).
constexpr int64_t kL2Elements = (int64_t)16 << 20;  // eight of 4 MiB, bf16
template <bool F32>
__global__ __launch_bounds__(256) void moe_combine_backward_kernel(CombineArgs a)
{
    const bool past_l2 = (int64_t)a.T * a.k * a.K > kL2Elements;
    const int lane = threadIdx.x & 63;
    const int64_t i = (int64_t)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    if (i >= (int64_t)a.T * a.k)
        return;
    const int64_t t = i / a.k;
    const int r = a.places[i];
    float dot = 0.0f;
    if ((unsigned)r < (unsigned)a.R) {
        const float w = a.weights ? a.weights[i] : 1.0f;
        constexpr int U = F32 ? 2 : 4;  // vectors under way
        for (int c0 = lane * 8; c0 < a.K; c0 += U * 512) {
            float d[U][8];
            uint4 y[U];
#pragma unroll
            for (int i = 0; i < U; ++i) {
                const int c = c0 + i * 512;
                if (c < a.K) {
                    load8<F32>(a.dout, (size_t)t * a.K + c, d[i]);
                    if (a.dweights)
                        y[i] = *(const uint4*)(a.y + (size_t)r * a.K + c);
                }
            }
#pragma unroll
            for (int i = 0; i < U; ++i) {
                const int c = c0 + i * 512;
                if (c >= a.K)
                    break;
                if (a.dweights) {
                    float f[8];
                    unpack8(y[i], f);
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        dot += d[i][e] * f[e];
                }
                if (a.dy) {
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        d[i][e] *= w;
                    if (past_l2)
                        store_bf16<8, true>(a.dy + (size_t)r * a.K + c, d[i]);
                    else
                        store_bf16<8>(a.dy + (size_t)r * a.K + c, d[i]);
                }
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
    // (tensors may start at any 4 bytes)
    const bool aligned = a.k % 4 == 0 && (((uintptr_t)a.places | (uintptr_t)a.weights) & 15) == 0;
    const auto kernel = a.fp32 ? (aligned ? moe_combine_kernel<true, true> : moe_combine_kernel<true, false>)
                               : (aligned ? moe_combine_kernel<false, true> : moe_combine_kernel<false, false>);
    kernel<<<(unsigned)blocks, 256, 0, stream>>>(a);
    return hipGetLastError();
}

hipError_t launch_moe_combine_backward(const CombineArgs& a, hipStream_t stream)
{
    const int most = kLaunchWaves / a.k;  // tokens of a launch
    const auto kernel = a.fp32 ? moe_combine_backward_kernel<true> : moe_combine_backward_kernel<false>;
    hipError_t rc = hipSuccess;
    for (int t = 0; t < a.T && rc == hipSuccess; t += most) {
        CombineArgs b = a;
        const size_t choice = (size_t)t * a.k;
        b.places = a.places + choice;
        b.weights = a.weights ? a.weights + choice : nullptr;
        b.dweights = a.dweights ? a.dweights + choice : nullptr;
        b.dout = (const char*)a.dout + (size_t)t * a.K * (a.fp32 ? 4 : 2);
        b.T = a.T - t < most ? a.T - t : most;
        kernel<<<(unsigned)(((int64_t)b.T * a.k + 3) / 4), 256, 0, stream>>>(b);
        rc = hipGetLastError();
    }
    return rc;
}

}  // namespace qll
