// Activations, their slopes and the epilogues of the feed-forward products.
// Everything is computed in fp32 from the fp32 sums and rounded once, to
// nearest even, where it is stored.
#pragma once

#include "ffn_internal.h"
#include "gemm_pipe.h"

namespace qll {

__device__ __forceinline__ float bf16_value(uint16_t h) { return __uint_as_float((uint32_t)h << 16); }

// 1 / (1 + e^-z); the reciprocal and the exponential are the hardware's
// (about 1 ulp each), far below the rounding of a bf16 result.
__device__ __forceinline__ float sigmoid_f(float z)
{
    return __builtin_amdgcn_rcpf(1.0f + __expf(-z));
}

constexpr float kGeluA = 0.7978845608028654f;   // sqrt(2 / pi)
constexpr float kGeluB = 0.044715f;
constexpr float kInvSqrt2 = 0.7071067811865476f;
constexpr float kInvSqrt2Pi = 0.3989422804014327f;

template <int ACT>
__device__ __forceinline__ float act_value(float z)
{
    if constexpr (ACT == ACT_RELU) {
        return z < 0.0f ? 0.0f : z;  // (a NaN stays one)
    } else if constexpr (ACT == ACT_GELU) {
        return 0.5f * z * (1.0f + erff(z * kInvSqrt2));
    } else if constexpr (ACT == ACT_GELU_TANH) {
        // (1 + tanh v) / 2 = sigmoid(2 v)
        return z * sigmoid_f(2.0f * kGeluA * (z + kGeluB * z * z * z));
    } else if constexpr (ACT == ACT_SILU) {
        return z * sigmoid_f(z);
    } else if constexpr (ACT == ACT_SIGMOID) {
        return sigmoid_f(z);
    } else {
        return z;
    }
}

// f = act(z), d = act'(z)
template <int ACT>
__device__ __forceinline__ void act_slope(float z, float& f, float& d)
{
    if constexpr (ACT == ACT_RELU) {
        f = z < 0.0f ? 0.0f : z;
        d = z > 0.0f ? 1.0f : 0.0f;
    } else if constexpr (ACT == ACT_GELU) {
        const float cdf = 0.5f * (1.0f + erff(z * kInvSqrt2));
        f = z * cdf;
        d = cdf + z * (kInvSqrt2Pi * __expf(-0.5f * z * z));
    } else if constexpr (ACT == ACT_GELU_TANH) {
        // past +-16 the sigmoid is 0 or 1 in fp32, and z^3 cannot overflow
        const float zc = fminf(fmaxf(z, -16.0f), 16.0f);
        const float q = sigmoid_f(2.0f * kGeluA * (zc + kGeluB * zc * zc * zc));
        f = z * q;
        d = q + zc * q * (1.0f - q) * (2.0f * kGeluA) * (1.0f + 3.0f * kGeluB * zc * zc);
    } else if constexpr (ACT == ACT_SILU) {
        const float q = sigmoid_f(z);
        f = z * q;
        d = q * (1.0f + z * (1.0f - q));
    } else if constexpr (ACT == ACT_SIGMOID) {
        f = sigmoid_f(z);
        d = f * (1.0f - f);
    } else {
        f = z;
        d = 1.0f;
    }
}

// f(integral_constant<ACT>) for the activation code act (uniform)
template <typename F>
__device__ __forceinline__ void with_act(int act, F&& f)
{
    switch (act) {
    case ACT_RELU: f(std::integral_constant<int, ACT_RELU>{}); break;
    case ACT_GELU: f(std::integral_constant<int, ACT_GELU>{}); break;
    case ACT_GELU_TANH: f(std::integral_constant<int, ACT_GELU_TANH>{}); break;
    case ACT_SILU: f(std::integral_constant<int, ACT_SILU>{}); break;
    case ACT_SIGMOID: f(std::integral_constant<int, ACT_SIGMOID>{}); break;
    default: f(std::integral_constant<int, ACT_NONE>{}); break;
    }
}

// W consecutive bf16 values (W = 4 or 8, aligned to their size) <-> floats
template <int W>
__device__ __forceinline__ void load_bf16(const uint16_t* p, float* f)
{
    static_assert(W == 4 || W == 8, "vector width");
    uint32_t w[W / 2];
    if constexpr (W == 8) {
        const uint4 v = *(const uint4*)p;
        w[0] = v.x; w[1] = v.y; w[2] = v.z; w[3] = v.w;
    } else {
        const uint2 v = *(const uint2*)p;
        w[0] = v.x; w[1] = v.y;
    }
#pragma unroll
    for (int i = 0; i < W / 2; ++i) {
        f[2 * i] = __uint_as_float(w[i] << 16);
        f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
}
// NT: a non-temporal store, for outputs that all compute units write at the
// same time at the end of their tiles: plain ones wait, dirty, in L2 and slow
// the next tile's first copies (forward products at M = 8192, N = 12288,
// K = 4096: 1-7% less with NT).
template <int W, bool NT = false>
__device__ __forceinline__ void store_bf16(uint16_t* p, const float* f)
{
    static_assert(W == 4 || W == 8, "vector width");
    if constexpr (W == 8 && NT)
        store16_stream(p, bf16x2_rne(f[0], f[1]), bf16x2_rne(f[2], f[3]), bf16x2_rne(f[4], f[5]),
                       bf16x2_rne(f[6], f[7]));
    else if constexpr (W == 8)
        *(uint4*)p = make_uint4(bf16x2_rne(f[0], f[1]), bf16x2_rne(f[2], f[3]),
                                bf16x2_rne(f[4], f[5]), bf16x2_rne(f[6], f[7]));
    else
        *(uint2*)p = make_uint2(bf16x2_rne(f[0], f[1]), bf16x2_rne(f[2], f[3]));
}
template <int W>
__device__ __forceinline__ void store_f32(float* p, const float* f)
{
#pragma unroll
    for (int i = 0; i < W; i += 4)
        *(float4*)(p + i) = make_float4(f[i], f[i + 1], f[i + 2], f[i + 3]);
}

// bf16_rne of one value, a NaN kept (bf16_rne is for finite values and
// infinities).
__device__ __forceinline__ uint16_t bf16_one(float f) { return (uint16_t)bf16x2_rne(f, f); }

// One output element of EPI_LINEAR.
__device__ __forceinline__ float linear_value(const FfnArgs& a, float v, int r, int c)
{
    if (a.sq)
        v = v * a.sq[r] * a.sp[0][c];
    if (a.bias)
        v += bf16_value(a.bias[c]);
    with_act(a.act, [&](auto A) { v = act_value<decltype(A)::value>(v); });
    if (a.res)
        v += bf16_value(a.res[(size_t)r * a.C + c]);
    return v;
}

__device__ __forceinline__ void store_value(const FfnArgs& a, float v, int r, int64_t c)
{
    char* base = (char*)(r < a.row_split ? a.out : a.out2);
    const size_t i = (size_t)(r < a.row_split ? r : r - a.row_split) * a.ldo + c;
    if (a.out_fp32)
        ((float*)base)[i] = v;
    else
        ((uint16_t*)base)[i] = bf16_one(v);
}

// The same columns where rows are not whole vectors (C % W != 0): element by
// element.  EPI_DZ, EPI_DGATED and EPI_PLAIN take whole vectors only.
template <int EPI, int W>
__device__ __forceinline__ void ffn_store_ragged(const FfnArgs& a, const float* v, const float* u,
                                                 int r, int c)
{
    if (r >= a.R)
        return;
#pragma unroll
    for (int i = 0; i < W; ++i) {
        const int ci = c + i;
        if (ci >= a.C)
            continue;
        if constexpr (EPI == EPI_PARTIAL) {
            a.partial[((size_t)blockIdx.y * a.R + r) * a.C + ci] = v[i];
        } else if constexpr (EPI == EPI_LINEAR) {
            store_value(a, linear_value(a, v[i], r, ci), r, ci);
        } else if constexpr (EPI == EPI_GATED) {
            float g = v[i], up = u[i];
            if (a.sq) {
                g = g * a.sq[r] * a.sp[0][ci];
                up = up * a.sq[r] * a.sp[1][ci];
            }
            with_act(a.act, [&](auto A) { g = act_value<decltype(A)::value>(g); });
            store_value(a, g * up, r, ci);
        }
    }
}

// The W output columns c .. c + W - 1 of row r, whose fp32 sums are v (gated:
// the gate's, u the up projection's); rows are whole vectors (C % W == 0), so
// the vector is in range as a whole and aligned.  EPI_DZ adds its outputs to
// cs.
template <int EPI, int W, int ACT>
__device__ __forceinline__ void ffn_store_act(const FfnArgs& a, float* v, const float* u, int r,
                                              int c, float* cs)
{
    if (r >= a.R)
        return;
    if (c >= a.C)
        return;
    if constexpr (EPI == EPI_PARTIAL) {
        store_f32<W>(a.partial + ((size_t)blockIdx.y * a.R + r) * a.C + c, v);
    } else if constexpr (EPI == EPI_PLAIN) {
        uint16_t* base = (uint16_t*)(r < a.row_split ? a.out : a.out2);
        store_bf16<W>(base + (size_t)(r < a.row_split ? r : r - a.row_split) * a.ldo + c, v);
    } else if constexpr (EPI == EPI_LINEAR) {
        if (a.sq) {
            const float s = a.sq[r];
#pragma unroll
            for (int i = 0; i < W; ++i)
                v[i] = v[i] * s * a.sp[0][c + i];
        }
        if (a.bias) {
            float b[W];
            load_bf16<W>(a.bias + c, b);
#pragma unroll
            for (int i = 0; i < W; ++i)
                v[i] += b[i];
        }
#pragma unroll
        for (int i = 0; i < W; ++i)
            v[i] = act_value<ACT>(v[i]);
        if (a.res) {
            float b[W];
            load_bf16<W>(a.res + (size_t)r * a.C + c, b);
#pragma unroll
            for (int i = 0; i < W; ++i)
                v[i] += b[i];
        }
        char* base = (char*)(r < a.row_split ? a.out : a.out2);
        const size_t at = (size_t)(r < a.row_split ? r : r - a.row_split) * a.ldo + c;
        if (a.out_fp32)
            store_f32<W>((float*)base + at, v);
        else
            store_bf16<W, true>((uint16_t*)base + at, v);
    } else if constexpr (EPI == EPI_GATED) {
        float o[W];
        const float s = a.sq ? a.sq[r] : 1.0f;
#pragma unroll
        for (int i = 0; i < W; ++i) {
            float g = v[i], up = u[i];
            if (a.sq) {
                g = g * s * a.sp[0][c + i];
                up = up * s * a.sp[1][c + i];
            }
            o[i] = act_value<ACT>(g) * up;
        }
        if (a.out_fp32)
            store_f32<W>((float*)a.out + (size_t)r * a.ldo + c, o);
        else
            store_bf16<W, true>((uint16_t*)a.out + (size_t)r * a.ldo + c, o);
    } else if constexpr (EPI == EPI_DZ) {
        float b[W], d[W];
        load_bf16<W>(a.dy + (size_t)r * a.C + c, d);
        if (a.bias)
            load_bf16<W>(a.bias + c, b);
#pragma unroll
        for (int i = 0; i < W; ++i) {
            float f, sl;
            act_slope<ACT>(a.bias ? v[i] + b[i] : v[i], f, sl);
            d[i] *= sl;
            cs[i] += d[i];
        }
        // the gradient products take bf16: one rounding here, one at theirs
        store_bf16<W>((uint16_t*)a.out + (size_t)r * a.ldo + c, d);
    } else if constexpr (EPI == EPI_DGATED) {
        float d[W], dg[W], du[W];
        load_bf16<W>(a.dy + (size_t)r * a.C + c, d);
#pragma unroll
        for (int i = 0; i < W; ++i) {
            float f, sl;
            act_slope<ACT>(v[i], f, sl);
            dg[i] = d[i] * u[i] * sl;
            du[i] = d[i] * f;
        }
        uint16_t* o = (uint16_t*)a.out + (size_t)r * a.ldo + c;
        store_bf16<W>(o, dg);
        store_bf16<W>(o + a.C, du);
    }
}

}  // namespace qll
