// Residual norms for gfx950, forward and backward, one row per workgroup
// slice and everything of a row in registers:
//
//   p = y / rms(y) * w_post        (or y)      rms(v) = sqrt(mean(v^2) + eps)
//   h = alpha r + beta gate p                  the new residual stream
//   n = h / rms(h) * w_pre                     bf16, or e4m3 with a row scale
//
// Bound by HBM: y and r are read once, h and n written once.  All sums are
// fp32; h is used unrounded for n, and rounded only where it is stored.
//
// Backward, with iy = 1 / rms(y), ih = 1 / rms(h), given dn and dr':
//   u  = dn w_pre                 dw_pre  = sum_m dn h ih
//   d  = dr' + ih (u - h ih^2 mean(u h))        dr = alpha d
//   dt = beta d                   dgate   = sum_m dt p
//   v  = dt gate w_post           dw_post = sum_m dt gate y iy
//   dy = iy (v - y iy^2 mean(v y))              (no post-norm: dy = dt gate)
// h, p and the rms are computed again from y and r, so nothing is kept from
// the forward pass.  The sums over rows stay in registers per column over the
// rows of a workgroup (a thread owns its columns), and the workgroups' sums
// are added in order by a second launch: no atomics.
#include "ffn_epilogue.h"
#include "quant_encode.h"

namespace qll {

namespace {

// Sum (or maximum) over the T threads of a row, in every thread.  `red`: one
// float per wave, not reused before the next barrier of the caller's rows.
template <int T, bool MAX>
__device__ __forceinline__ float row_reduce(float v, float* red)
{
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const float o = __shfl_xor(v, d, 64);
        v = MAX ? fmaxf(v, o) : v + o;
    }
    if constexpr (T > 64) {
        constexpr int WV = T / 64;
        const int wave = threadIdx.x >> 6;
        if ((threadIdx.x & 63) == 0)
            red[wave] = v;
        __syncthreads();
        v = red[0];
#pragma unroll
        for (int w = 1; w < WV; ++w)
            v = MAX ? fmaxf(v, red[w]) : v + red[w];
    }
    return v;
}

template <bool F32>
__device__ __forceinline__ void load_stream(const void* p, size_t at, float* f)
{
    if constexpr (F32) {
        const float4 x = *(const float4*)((const float*)p + at);
        const float4 y = *(const float4*)((const float*)p + at + 4);
        f[0] = x.x; f[1] = x.y; f[2] = x.z; f[3] = x.w;
        f[4] = y.x; f[5] = y.y; f[6] = y.z; f[7] = y.w;
    } else {
        load_bf16<8>((const uint16_t*)p + at, f);
    }
}

template <bool F32>
__device__ __forceinline__ void store_stream(void* p, size_t at, const float* f)
{
    if constexpr (F32)
        store_f32<8>((float*)p + at, f);
    else
        store_bf16<8>((uint16_t*)p + at, f);
}

__device__ __forceinline__ float inv_rms(float sum, int K, float eps)
{
    return 1.0f / sqrtf(sum / (float)K + eps);
}

}  // namespace

// T threads per row, CH runs of 8 columns per thread; rows of up to 64
// threads share a workgroup of 256.
template <int T, int CH, bool HAS_Y, bool F32, bool QUANT>
__global__ __launch_bounds__(T < 256 ? 256 : T) void residual_norm_kernel(NormArgs a)
{
    constexpr int TB = T < 256 ? 256 : T;
    static_assert(T == 64 || T >= 256, "threads of a row");
    __shared__ float red[3][TB / 64];
    const int t = threadIdx.x % T;
    const int m = blockIdx.x * (TB / T) + threadIdx.x / T;
    if (T < 256 && m >= a.M)
        return;  // (whole waves; rows of 64 threads meet no barrier)
    const int K = a.K;
    const size_t row = (size_t)m * K;

    float h[CH][8];
    float y[HAS_Y ? CH : 1][8];
    float sy = 0.0f;
#pragma unroll
    for (int j = 0; j < CH; ++j) {
        const int c = (t + j * T) * 8;
#pragma unroll
        for (int e = 0; e < 8; ++e)
            h[j][e] = 0.0f;
        if (c < K)
            load_stream<F32>(a.r, row + c, h[j]);
        if constexpr (HAS_Y) {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                y[j][e] = 0.0f;
            if (c < K)
                load_bf16<8>(a.y + row + c, y[j]);
#pragma unroll
            for (int e = 0; e < 8; ++e)
                sy += y[j][e] * y[j][e];
        }
    }
    float sh = 0.0f;
    if constexpr (HAS_Y) {
        float iy = 1.0f;
        if (a.w_post)
            iy = inv_rms(row_reduce<T, false>(sy, red[0]), K, a.eps);
#pragma unroll
        for (int j = 0; j < CH; ++j) {
            const int c = (t + j * T) * 8;
            if (c < K) {
                float w[8];
                if (a.w_post) {
                    load_bf16<8>(a.w_post + c, w);
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        y[j][e] = y[j][e] * iy * w[e];
                }
                if (a.gate) {
                    load_bf16<8>(a.gate + c, w);
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        y[j][e] *= w[e];
                }
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    h[j][e] = a.alpha * h[j][e] + a.beta * y[j][e];
                store_stream<F32>(a.r_out, row + c, h[j]);
            }
        }
    }
#pragma unroll
    for (int j = 0; j < CH; ++j)
#pragma unroll
        for (int e = 0; e < 8; ++e)
            sh += h[j][e] * h[j][e];
    const float ih = inv_rms(row_reduce<T, false>(sh, red[1]), K, a.eps);
    float amax = 0.0f;
#pragma unroll
    for (int j = 0; j < CH; ++j) {
        const int c = (t + j * T) * 8;
        if (c < K) {
            float w[8];
            load_bf16<8>(a.w_pre + c, w);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                h[j][e] = h[j][e] * ih * w[e];
                amax = fmaxf(amax, fabsf(h[j][e]));
            }
            if constexpr (!QUANT)
                store_bf16<8>((uint16_t*)a.n_out + row + c, h[j]);
        }
    }
    if constexpr (QUANT) {
        // the rule of quantize_per_token_fp8, on the fp32 values
        amax = row_reduce<T, true>(amax, red[2]);
        const Quot q(amax / 448.0f);
        if (t == 0)
            a.n_scales[m] = q.s;
#pragma unroll
        for (int j = 0; j < CH; ++j) {
            const int c = (t + j * T) * 8;
            if (c < K) {
                float f[8];
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    f[e] = q.s == 0.0f ? 0.0f
                                       : clamp448(q.fast ? q.by_reciprocal(h[j][e]) : h[j][e] / q.s);
                int w0 = __builtin_amdgcn_cvt_pk_fp8_f32(f[0], f[1], 0, false);
                w0 = __builtin_amdgcn_cvt_pk_fp8_f32(f[2], f[3], w0, true);
                int w1 = __builtin_amdgcn_cvt_pk_fp8_f32(f[4], f[5], 0, false);
                w1 = __builtin_amdgcn_cvt_pk_fp8_f32(f[6], f[7], w1, true);
                *(uint2*)((uint8_t*)a.n_out + row + c) = make_uint2((uint32_t)w0, (uint32_t)w1);
            }
        }
    }
}

// One row at a time per workgroup of T threads, rows blockIdx.x, + gridDim.x,
// ...; the vector gradients' sums stay in registers.
template <int T, int CH, bool HAS_Y, bool F32>
__global__ __launch_bounds__(T) void residual_norm_backward_kernel(NormArgs a)
{
    __shared__ float red[2][4][T / 64];
    const int t = threadIdx.x;
    const int K = a.K;
    const float invk = 1.0f / (float)K;
    float s_pre[CH][8], s_post[HAS_Y ? CH : 1][8], s_gate[HAS_Y ? CH : 1][8];
#pragma unroll
    for (int j = 0; j < CH; ++j)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            s_pre[j][e] = 0.0f;
            if constexpr (HAS_Y)
                s_post[j][e] = s_gate[j][e] = 0.0f;
        }
    int par = 0;
    for (int m = blockIdx.x; m < a.M; m += gridDim.x, par ^= 1) {
        const size_t row = (size_t)m * K;
        float h[CH][8], u[CH][8], d[CH][8], y[HAS_Y ? CH : 1][8];
        float sy = 0.0f;
#pragma unroll
        for (int j = 0; j < CH; ++j) {
            const int c = (t + j * T) * 8;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                h[j][e] = u[j][e] = d[j][e] = 0.0f;
                if constexpr (HAS_Y)
                    y[j][e] = 0.0f;
            }
            if (c < K) {
                load_stream<F32>(a.r, row + c, h[j]);
                load_bf16<8>(a.dn + row + c, u[j]);
                if (a.dr_out)
                    load_stream<F32>(a.dr_out, row + c, d[j]);
                if constexpr (HAS_Y)
                    load_bf16<8>(a.y + row + c, y[j]);
            }
            if constexpr (HAS_Y) {
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    sy += y[j][e] * y[j][e];
            }
        }
        float iy = 1.0f;
        if constexpr (HAS_Y) {
            if (a.w_post)
                iy = inv_rms(row_reduce<T, false>(sy, red[par][0]), K, a.eps);
        }
        float sh = 0.0f, suh = 0.0f;
#pragma unroll
        for (int j = 0; j < CH; ++j) {
            const int c = (t + j * T) * 8;
            if (c < K) {
                float w[8];
                if constexpr (HAS_Y) {
                    float p[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        p[e] = y[j][e];
                    if (a.w_post) {
                        load_bf16<8>(a.w_post + c, w);
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            p[e] = y[j][e] * iy * w[e];
                    }
                    if (a.gate) {
                        load_bf16<8>(a.gate + c, w);
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            p[e] *= w[e];
                    }
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        h[j][e] = a.alpha * h[j][e] + a.beta * p[e];
                }
                load_bf16<8>(a.w_pre + c, w);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    sh += h[j][e] * h[j][e];
                    suh += u[j][e] * w[e] * h[j][e];
                }
            }
        }
        sh = row_reduce<T, false>(sh, red[par][1]);
        suh = row_reduce<T, false>(suh, red[par][2]);
        const float ih = inv_rms(sh, K, a.eps);
        const float mh = suh * invk * ih * ih;
        float svy = 0.0f;
#pragma unroll
        for (int j = 0; j < CH; ++j) {
            const int c = (t + j * T) * 8;
            if (c < K) {
                float w[8], o[8];
                load_bf16<8>(a.w_pre + c, w);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    s_pre[j][e] += u[j][e] * h[j][e] * ih;
                    d[j][e] += ih * (u[j][e] * w[e] - h[j][e] * mh);
                    o[e] = a.alpha * d[j][e];
                }
                store_stream<F32>(a.dr, row + c, o);
                if constexpr (HAS_Y) {
                    float w1[8], g[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        w1[e] = g[e] = 1.0f;
                        d[j][e] *= a.beta;
                    }
                    if (a.w_post)
                        load_bf16<8>(a.w_post + c, w1);
                    if (a.gate)
                        load_bf16<8>(a.gate + c, g);
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const float yn = y[j][e] * iy;
                        s_gate[j][e] += d[j][e] * yn * w1[e];
                        d[j][e] *= g[e];
                        s_post[j][e] += d[j][e] * yn;
                        d[j][e] *= w1[e];
                        svy += d[j][e] * y[j][e];
                    }
                }
            }
        }
        if constexpr (HAS_Y) {
            float my = 0.0f;
            if (a.w_post)
                my = row_reduce<T, false>(svy, red[par][3]) * invk * iy * iy;
#pragma unroll
            for (int j = 0; j < CH; ++j) {
                const int c = (t + j * T) * 8;
                if (c < K) {
                    float o[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        o[e] = iy * (d[j][e] - y[j][e] * my);
                    store_bf16<8>(a.dy + row + c, o);
                }
            }
        }
    }
    const size_t plane = (size_t)gridDim.x * K;
    float* part = a.partial + (size_t)blockIdx.x * K;
#pragma unroll
    for (int j = 0; j < CH; ++j) {
        const int c = (t + j * T) * 8;
        if (c < K) {
            store_f32<8>(part + c, s_pre[j]);
            if constexpr (HAS_Y) {
                if (a.w_post)
                    store_f32<8>(part + plane + c, s_post[j]);
                if (a.gate)
                    store_f32<8>(part + 2 * plane + c, s_gate[j]);
            }
        }
    }
}

namespace {

template <int T, int CH>
hipError_t forward(const NormArgs& a, hipStream_t s)
{
    constexpr int TB = T < 256 ? 256 : T;
    const unsigned grid = (unsigned)((a.M + TB / T - 1) / (TB / T));
    auto go = [&](auto HY, auto F, auto Q) {
        residual_norm_kernel<T, CH, decltype(HY)::value, decltype(F)::value, decltype(Q)::value>
            <<<grid, TB, 0, s>>>(a);
    };
    using Y = std::true_type;
    using N = std::false_type;
    switch ((a.y ? 4 : 0) + (a.r_fp32 ? 2 : 0) + (a.quant ? 1 : 0)) {
    case 0: go(N{}, N{}, N{}); break;
    case 1: go(N{}, N{}, Y{}); break;
    case 2: go(N{}, Y{}, N{}); break;
    case 3: go(N{}, Y{}, Y{}); break;
    case 4: go(Y{}, N{}, N{}); break;
    case 5: go(Y{}, N{}, Y{}); break;
    case 6: go(Y{}, Y{}, N{}); break;
    default: go(Y{}, Y{}, Y{}); break;
    }
    return hipGetLastError();
}

template <int T, int CH>
hipError_t backward(const NormArgs& a, hipStream_t s)
{
    const unsigned grid = (unsigned)norm_backward_blocks(a.M, a.K);
    if (a.y) {
        if (a.r_fp32)
            residual_norm_backward_kernel<T, CH, true, true><<<grid, T, 0, s>>>(a);
        else
            residual_norm_backward_kernel<T, CH, true, false><<<grid, T, 0, s>>>(a);
    } else {
        if (a.r_fp32)
            residual_norm_backward_kernel<T, CH, false, true><<<grid, T, 0, s>>>(a);
        else
            residual_norm_backward_kernel<T, CH, false, false><<<grid, T, 0, s>>>(a);
    }
    return hipGetLastError();
}

}  // namespace

hipError_t launch_residual_norm(const NormArgs& a, hipStream_t s)
{
    const int runs = a.K / 8;
    if (runs <= 64)
        return forward<64, 1>(a, s);
    if (runs <= 256)
        return a.M >= 1024 ? forward<64, 4>(a, s) : forward<256, 1>(a, s);
    if (runs <= 512)
        return a.M >= 1024 ? forward<256, 2>(a, s) : forward<512, 1>(a, s);
    if (runs <= 1024)
        return a.M >= 1024 ? forward<256, 4>(a, s) : forward<1024, 1>(a, s);
    if (runs <= 2048)
        return forward<1024, 2>(a, s);
    return forward<1024, 4>(a, s);
}

int norm_backward_blocks(int64_t M, int64_t K)
{
    const int64_t runs = K / 8;
    const int64_t most = runs <= 256 ? 1024 : 512;
    if (M <= most)
        return (int)M;
    return (int)most;
}

hipError_t launch_residual_norm_backward(const NormArgs& a, hipStream_t s)
{
    const int runs = a.K / 8;
    if (runs <= 64)
        return backward<64, 1>(a, s);
    if (runs <= 128)
        return backward<128, 1>(a, s);
    if (runs <= 256)
        return backward<256, 1>(a, s);
    if (runs <= 512)
        return backward<512, 1>(a, s);
    if (runs <= 1024)
        return backward<1024, 1>(a, s);
    if (runs <= 2048)
        return backward<1024, 2>(a, s);
    return backward<1024, 4>(a, s);
}

}  // namespace qll
