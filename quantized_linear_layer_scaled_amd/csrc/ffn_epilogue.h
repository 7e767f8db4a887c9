// Activations, their slopes and the epilogues of the feed-forward products.
// Everything is computed in fp32 from the fp32 sums and rounded once, to
// nearest even, where it is stored.
#pragma once

#include "ffn_internal.h"
#include "gemm_pipe.h"

namespace qll {

__device__ __forceinline__ float bf16_value(uint16_t h) { return __uint_as_float((uint32_t)h << 16); }

// 1 / (1 + e^-z); the reciprocal and the exponential of two are the hardware's
// (about 1 ulp each), and the exponent's rounding moves e^-z by |z| 2^-24 of
// itself: far below the rounding of a bf16 result.
__device__ __forceinline__ float sigmoid_f(float z)
{
    return __builtin_amdgcn_rcpf(1.0f + __expf(-z));
}

constexpr float kGeluA = 0.7978845608028654f;   // sqrt(2 / pi)
constexpr float kGeluB = 0.044715f;
constexpr float kInvSqrt2Pi = 0.3989422804014327f;

// Phi(z), the normal distribution function, and e = exp(-z^2 / 2).  Below zero
// Phi(-a) = e g(a), so nothing cancels and the tail keeps its accuracy relative
// to itself; above, 1 - e g.  g(a) = exp(a^2 / 2) erfc(a / sqrt 2) / 2 falls
// from 1/2 like 1 / a: a polynomial t Q(t) in t = 1 / (1 + 0.305 a), of least
// maximum relative error on 0 <= a <= 14 (9.4e-8), past which e is 0.  The
// exponent's own roundings are the largest error: in all at most
// (1.25 z^2 + 16) 2^-24 of Phi.  Its exponential is the density's too.  (The
// library's erff costs four times as much: a tile of gelu slopes 25 us of
// vector instructions.)
__device__ __forceinline__ float normal_cdf(float z, float& e)
{
    constexpr float kHalfLog2e = 0.72134752f;
    const float t = __builtin_amdgcn_rcpf(1.0f + 0.305f * fabsf(z));
    e = __builtin_amdgcn_exp2f(-kHalfLog2e * (z * z));
    float q = 0.0367022827f;
    q = q * t - 0.153001919f;
    q = q * t + 0.185741723f;
    q = q * t - 0.0380010158f;
    q = q * t + 0.121035233f;
    q = q * t + 0.103416525f;
    q = q * t + 0.122467548f;
    q = q * t + 0.121639684f;
    const float tail = q * t * e;
    return z < 0.0f ? tail : 1.0f - tail;
}

template <int ACT>
__device__ __forceinline__ float act_value(float z)
{
    if constexpr (ACT == ACT_RELU) {
        return z < 0.0f ? 0.0f : z;  // (a NaN stays one)
    } else if constexpr (ACT == ACT_GELU) {
        float e;
        return z * normal_cdf(z, e);
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
        float e;
        const float cdf = normal_cdf(z, e);
        f = z * cdf;
        d = cdf + z * (kInvSqrt2Pi * e);
    } else if constexpr (ACT == ACT_GELU_TANH) {
        // past +-16 the sigmoid is 0 or 1 in fp32, and z^3 cannot overflow
        // (comparisons, which keep a NaN; fminf and fmaxf drop it)
        const float zc = z > 16.0f ? 16.0f : (z < -16.0f ? -16.0f : z);
        const float q = sigmoid_f(2.0f * kGeluA * (zc + kGeluB * zc * zc * zc));
        f = z * q;
        d = q + zc * q * (1.0f - q) * (2.0f * kGeluA) * (1.0f + 3.0f * kGeluB * zc * zc);
    } else if constexpr (ACT == ACT_SILU) {
        const float q = sigmoid_f(z);
        f = z * q;
        d = q * (1.0f + z * (1.0f - q));
    } else if constexpr (ACT == ACT_SIGMOID) {
        // f (1 - f) from e^-|z|: 1 - f would cancel where f is next to 1
        const float e = __expf(-fabsf(z));
        const float r = __builtin_amdgcn_rcpf(1.0f + e);
        f = z < 0.0f ? e * r : r;
        d = e * r * r;
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

// Vectors of 32-bit words at any 2-byte address: rows of an odd number of
// columns start anywhere, and the memory takes such accesses as they are.
typedef uint32_t u32x4_any __attribute__((ext_vector_type(4), aligned(2)));
typedef uint32_t u32x2_any __attribute__((ext_vector_type(2), aligned(2)));

// W consecutive bf16 values (W = 4 or 8) <-> floats
template <int W>
__device__ __forceinline__ void load_bf16(const uint16_t* p, float* f)
{
    static_assert(W == 4 || W == 8, "vector width");
    uint32_t w[W / 2];
    if constexpr (W == 8) {
        const u32x4_any v = *(const u32x4_any*)p;
        w[0] = v.x; w[1] = v.y; w[2] = v.z; w[3] = v.w;
    } else {
        const u32x2_any v = *(const u32x2_any*)p;
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
// K = 4096: 1-7% less with NT; 8-byte vectors and outputs that the next
// product reads: 2-3% more).
template <int W, bool NT = false>
__device__ __forceinline__ void store_bf16(uint16_t* p, const float* f)
{
    static_assert(W == 4 || W == 8, "vector width");
    if constexpr (W == 8) {
        const u32x4_any v = {bf16x2_rne(f[0], f[1]), bf16x2_rne(f[2], f[3]),
                             bf16x2_rne(f[4], f[5]), bf16x2_rne(f[6], f[7])};
        if constexpr (NT)
            __builtin_nontemporal_store(v, (u32x4_any*)p);
        else
            *(u32x4_any*)p = v;
    } else {
        *(u32x2_any*)p = u32x2_any{bf16x2_rne(f[0], f[1]), bf16x2_rne(f[2], f[3])};
    }
}
template <int W>
__device__ __forceinline__ void store_f32(float* p, const float* f)
{
    typedef float f32x4_any __attribute__((ext_vector_type(4), aligned(4)));
#pragma unroll
    for (int i = 0; i < W; i += 4)
        *(f32x4_any*)(p + i) = f32x4_any{f[i], f[i + 1], f[i + 2], f[i + 3]};
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

// What the columns of one vector share: their scales and biases, read once
// (columns past the end stay 0).
template <int W>
struct ColumnVector {
    float s0[W], s1[W], b[W];
};
template <int EPI, int W>
__device__ __forceinline__ void load_columns(const FfnArgs& a, int c, ColumnVector<W>& v)
{
    if constexpr (EPI == EPI_LINEAR || EPI == EPI_GATED || EPI == EPI_DZ) {
#pragma unroll
        for (int i = 0; i < W; ++i) {
            v.s0[i] = v.s1[i] = v.b[i] = 0.0f;
            if (c + i >= a.C)
                continue;
            if (EPI != EPI_DZ && a.sq) {
                v.s0[i] = a.sp[0][c + i];
                if (EPI == EPI_GATED)
                    v.s1[i] = a.sp[1][c + i];
            }
            if (EPI != EPI_GATED && a.bias)
                v.b[i] = bf16_value(a.bias[c + i]);
        }
    }
}

// The W output columns c .. c + W - 1 of row r, whose fp32 sums are v (gated:
// the gate's, u the up projection's).  A vector that reaches past the last
// column is stored element by element.  EPI_DZ adds its outputs to cs.
// (EPI_DZ, EPI_DGATED and EPI_PLAIN have C % 8 == 0.)
template <int EPI, int W, int ACT>
__device__ __forceinline__ void ffn_store_act(const FfnArgs& a, float* v, const float* u, int r,
                                              int c, const ColumnVector<W>& cv, float* cs)
{
    if (r >= a.R || c >= a.C)
        return;
    const bool whole = c + W <= a.C;
    if constexpr (EPI == EPI_PARTIAL) {
        float* o = a.partial + ((size_t)blockIdx.y * a.R + r) * a.C + c;
        if (whole) {
            store_f32<W>(o, v);
        } else {
#pragma unroll
            for (int i = 0; i < W; ++i)
                if (c + i < a.C)
                    o[i] = v[i];
        }
    } else if constexpr (EPI == EPI_PLAIN) {
        uint16_t* base = (uint16_t*)(r < a.row_split ? a.out : a.out2);
        store_bf16<W>(base + (size_t)(r < a.row_split ? r : r - a.row_split) * a.ldo + c, v);
    } else if constexpr (EPI == EPI_LINEAR || EPI == EPI_GATED) {
        const float s = a.sq ? a.sq[r] : 1.0f;
#pragma unroll
        for (int i = 0; i < W; ++i) {
            float z = v[i];
            if (a.sq)
                z = z * s * cv.s0[i];
            if constexpr (EPI == EPI_LINEAR) {
                v[i] = act_value<ACT>(a.bias ? z + cv.b[i] : z);
            } else {
                float up = u[i];
                if (a.sq)
                    up = up * s * cv.s1[i];
                v[i] = act_value<ACT>(z) * up;
            }
        }
        if (EPI == EPI_LINEAR && a.res) {
            const uint16_t* from = a.res + (size_t)r * a.C + c;
            if (whole) {
                float b[W];
                load_bf16<W>(from, b);
#pragma unroll
                for (int i = 0; i < W; ++i)
                    v[i] += b[i];
            } else {
#pragma unroll
                for (int i = 0; i < W; ++i)
                    if (c + i < a.C)
                        v[i] += bf16_value(from[i]);
            }
        }
        char* base = (char*)(r < a.row_split ? a.out : a.out2);
        const size_t at = (size_t)(r < a.row_split ? r : r - a.row_split) * a.ldo + c;
        if (whole) {
            if (a.out_fp32)
                store_f32<W>((float*)base + at, v);
            else
                store_bf16<W, true>((uint16_t*)base + at, v);
        } else {
#pragma unroll
            for (int i = 0; i < W; ++i)
                if (c + i < a.C)
                    store_value(a, v[i], r, c + i);
        }
    } else if constexpr (EPI == EPI_DZ) {
        float d[W];
        load_bf16<W>(a.dy + (size_t)r * a.C + c, d);
#pragma unroll
        for (int i = 0; i < W; ++i) {
            float f, sl;
            act_slope<ACT>(a.bias ? v[i] + cv.b[i] : v[i], f, sl);
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
