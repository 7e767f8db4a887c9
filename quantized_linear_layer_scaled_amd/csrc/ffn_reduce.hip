// Second launches of the feed-forward products: the sum of Split-K pieces
// with the linear epilogue, and column sums (bias gradients, and the vector
// gradients of the norms).  All sums run in a fixed order.
#include "ffn_epilogue.h"

namespace qll {

// One thread per 4 columns of a row (C % 4 == 0), or per element.
template <bool VEC>
__global__ __launch_bounds__(256) void ffn_reduce_kernel(FfnArgs a)
{
    constexpr int W = VEC ? 4 : 1;
    const size_t plane = (size_t)a.R * a.C;
    const size_t at = ((size_t)blockIdx.x * 256 + threadIdx.x) * W;
    if (at >= plane)
        return;
    const int r = (int)(at / a.C), c = (int)(at % a.C);
    if constexpr (VEC) {
        float v[4] = {0, 0, 0, 0};
        for (int s = 0; s < a.splits; ++s) {
            const float4 p = *(const float4*)(a.partial + s * plane + at);
            v[0] += p.x;
            v[1] += p.y;
            v[2] += p.z;
            v[3] += p.w;
        }
        ColumnVector<4> cv;
        load_columns<EPI_LINEAR, 4>(a, c, cv);
        with_act(a.act, [&](auto A) {
            ffn_store_act<EPI_LINEAR, 4, decltype(A)::value>(a, v, nullptr, r, c, cv, nullptr);
        });
    } else {
        float v = 0.0f;
        for (int s = 0; s < a.splits; ++s)
            v += a.partial[s * plane + at];
        store_value(a, linear_value(a, v, r, c), r, c);
    }
}

hipError_t ffn_launch_reduce(const FfnArgs& a, hipStream_t stream)
{
    const size_t n = (size_t)a.R * a.C;
    if (a.C % 4 == 0)
        ffn_reduce_kernel<true><<<(unsigned)((n / 4 + 255) / 256), 256, 0, stream>>>(a);
    else
        ffn_reduce_kernel<false><<<(unsigned)((n + 255) / 256), 256, 0, stream>>>(a);
    return hipGetLastError();
}

// partial[strip][c] = sum of x[r][c] over the strip's rows; 8 columns per
// thread, C % 8 == 0
__global__ __launch_bounds__(256) void colsum_strips_kernel(const uint16_t* x, float* partial, int R,
                                                            int C)
{
    const int c = (blockIdx.y * 256 + threadIdx.x) * 8;
    if (c >= C)
        return;
    const int r0 = blockIdx.x * kColsumRows, r1 = min(R, r0 + kColsumRows);
    float s[8] = {0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll 8
    for (int r = r0; r < r1; ++r) {
        float v[8];
        load_bf16<8>(x + (size_t)r * C + c, v);
#pragma unroll
        for (int e = 0; e < 8; ++e)
            s[e] += v[e];
    }
    store_f32<8>(partial + (size_t)blockIdx.x * C + c, s);
}

hipError_t launch_colsum_strips(const void* x, float* partial, int64_t R, int64_t C,
                                hipStream_t stream)
{
    const dim3 grid((unsigned)((R + kColsumRows - 1) / kColsumRows), (unsigned)((C / 8 + 255) / 256));
    colsum_strips_kernel<<<grid, 256, 0, stream>>>((const uint16_t*)x, partial, (int)R, (int)C);
    return hipGetLastError();
}

// 64 columns per workgroup; its 16 waves take every sixteenth strip each and
// are added in order.
__global__ __launch_bounds__(1024) void colsum_finish_kernel(ColsumArgs a)
{
    __shared__ float red[16][64];
    float* out = a.out[blockIdx.y];
    if (!out)
        return;
    const float* partial = a.partial + (size_t)blockIdx.y * a.strips * a.C;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int c = blockIdx.x * 64 + lane;
    float v = 0.0f;
    if (c < a.C) {
#pragma unroll 4
        for (int s = wave; s < a.strips; s += 16)
            v += partial[(size_t)s * a.C + c];
    }
    red[wave][lane] = v;
    __syncthreads();
    if (wave == 0 && c < a.C) {
        v = red[0][lane];
#pragma unroll
        for (int w = 1; w < 16; ++w)
            v += red[w][lane];
        out[c] = v;
    }
}

hipError_t launch_colsum_finish(const ColsumArgs& a, int planes, hipStream_t stream)
{
    colsum_finish_kernel<<<dim3((unsigned)((a.C + 63) / 64), (unsigned)planes), 1024, 0, stream>>>(a);
    return hipGetLastError();
}

}  // namespace qll
