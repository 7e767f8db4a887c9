// Residual norms for gfx950, forward and backward, one row per workgroup
// slice and everything of a row in registers:
//
//   p = y / rms(y) * w_post        (or y)      rms(v) = sqrt(mean(v^2) + eps)
//   h = alpha r + beta gate p                  the new residual stream
//   n = h / rms(h) * w_pre                     bf16, or e4m3 with a row scale
//
// Bound by HBM: y and r are read once, h and n written once (M = 4096,
// K = 4096, e4m3 out: 26.3 us = 4.5 TB/s of the 5.2 that a copy reaches;
// M = 8192, K = 8192: 93 us).  All sums are fp32; h is used unrounded for n,
// and rounded only where it is stored.
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
// are added in order by a second launch: no atomics.  M = 8192, K = 4096: 87
// us = 4.6 TB/s.
#include "ffn_epilogue.h"
#include "quant_encode.h"

namespace qll {

namespace {

// The larger of two magnitudes, a NaN if either is one: the order of their
// bits, in which a NaN is above infinity (fmaxf drops it).
__device__ __forceinline__ float magnitude_max(float a, float b)
{
    return __uint_as_float(max(__float_as_uint(a), __float_as_uint(b)));
}

// Sum (or maximum, of magnitudes) over the T threads of a row, in every
// thread.  `red`: one float per wave, not reused before the next barrier of
// the caller's rows.
template <int T, bool MAX>
__device__ __forceinline__ float row_reduce(float v, float* red)
{
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const float o = __shfl_xor(v, d, 64);
        v = MAX ? magnitude_max(v, o) : v + o;
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
            v = MAX ? magnitude_max(v, red[w]) : v + red[w];
    }
    return v;
}

// Eight values of the stream as they lie in memory, and as floats.
template <bool F32>
struct StreamRun {
    uint4 w[F32 ? 2 : 1];
    __device__ __forceinline__ void clear()
    {
#pragma unroll
        for (int p = 0; p < (F32 ? 2 : 1); ++p)
            w[p] = make_uint4(0, 0, 0, 0);
    }
    __device__ __forceinline__ void load(const void* base, size_t at)
    {
#pragma unroll
        for (int p = 0; p < (F32 ? 2 : 1); ++p)
            w[p] = *(const uint4*)((const char*)base + (F32 ? (at + 4 * p) * 4 : at * 2));
    }
    __device__ __forceinline__ void widen(float* f) const
    {
        if constexpr (F32) {
            const uint32_t v[8] = {w[0].x, w[0].y, w[0].z, w[0].w, w[1].x, w[1].y, w[1].z, w[1].w};
#pragma unroll
            for (int e = 0; e < 8; ++e)
                f[e] = __uint_as_float(v[e]);
        } else {
            unpack8(w[0], f);
        }
    }
};

template <bool F32>
__device__ __forceinline__ void store_stream(void* p, size_t at, const float* f)
{
    if constexpr (F32)
        store_f32<8>((float*)p + at, f);
    else
        store_bf16<8>((uint16_t*)p + at, f);
}

// A thread's runs of the three channel vectors (missing ones read as 1), kept
// in registers over the rows where there is one run per thread, else read
// again for each row.
template <int T, int CH>
struct Vectors {
    static constexpr bool KEEP = CH == 1;
    const NormArgs& a;
    int t;
    uint4 kept[3];
    __device__ __forceinline__ Vectors(const NormArgs& args, int tid) : a(args), t(tid)
    {
        if constexpr (KEEP) {
#pragma unroll
            for (int v = 0; v < 3; ++v)
                kept[v] = fetch(v, 0);
        }
    }
    __device__ __forceinline__ uint4 fetch(int v, int j) const
    {
        const uint16_t* p = v == 0 ? a.w_post : (v == 1 ? a.gate : a.w_pre);
        const int c = (t + j * T) * 8;
        return p && c < a.K ? *(const uint4*)(p + c)
                            : make_uint4(0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u);
    }
    __device__ __forceinline__ void get(int v, int j, float* f) const
    {
        unpack8(KEEP ? kept[v] : fetch(v, j), f);
    }
};

__device__ __forceinline__ float inv_rms(float sum, int K, float eps)
{
    return 1.0f / sqrtf(sum / (float)K + eps);
}

}  // namespace

// One row at a time per workgroup of T threads, CH runs of 8 columns per
// thread, rows blockIdx.x, + gridDim.x, ...  The next row's words are loaded
// before this row's sums are formed (one run per thread; longer rows have no
// registers for it).
template <int T, int CH, bool HAS_Y, bool F32, bool QUANT>
__global__ __launch_bounds__(T) void residual_norm_kernel(NormArgs a)
{
    __shared__ float red[2][3][T / 64];
    constexpr bool AHEAD = CH == 1;
    const int t = threadIdx.x;
    const int K = a.K;
    const Vectors<T, CH> vec(a, t);
    struct Row {
        uint4 y[CH];
        StreamRun<F32> r[CH];
    } next;
    auto fetch = [&](int m) __attribute__((always_inline)) {
        const size_t row = (size_t)m * K;
#pragma unroll
        for (int j = 0; j < CH; ++j) {
            const int c = (t + j * T) * 8;
            next.y[j] = make_uint4(0, 0, 0, 0);
            next.r[j].clear();
            if (m < a.M && c < K) {
                next.r[j].load(a.r, row + c);
                if constexpr (HAS_Y)
                    next.y[j] = *(const uint4*)(a.y + row + c);
            }
        }
    };
    if constexpr (AHEAD)
        fetch(blockIdx.x);
    int par = 0;
    for (int m = blockIdx.x; m < a.M; m += gridDim.x, par ^= 1) {
        const size_t row = (size_t)m * K;
        if constexpr (!AHEAD)
            fetch(m);
        float h[CH][8], y[HAS_Y ? CH : 1][8];
        float sy = 0.0f, sh = 0.0f;
#pragma unroll
        for (int j = 0; j < CH; ++j) {
            next.r[j].widen(h[j]);
            if constexpr (HAS_Y) {
                unpack8(next.y[j], y[j]);
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    sy += y[j][e] * y[j][e];
            }
        }
        if constexpr (AHEAD)
            fetch(m + gridDim.x);
        if constexpr (HAS_Y) {
            float iy = 1.0f;
            if (a.w_post)
                iy = inv_rms(row_reduce<T, false>(sy, red[par][0]), K, a.eps);
#pragma unroll
            for (int j = 0; j < CH; ++j) {
                const int c = (t + j * T) * 8;
                float w1[8], g[8];
                vec.get(0, j, w1);
                vec.get(1, j, g);
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    h[j][e] = a.alpha * h[j][e] + a.beta * (y[j][e] * iy * w1[e] * g[e]);
                if (c < K)
                    store_stream<F32>(a.r_out, row + c, h[j]);
            }
        }
#pragma unroll
        for (int j = 0; j < CH; ++j)
#pragma unroll
            for (int e = 0; e < 8; ++e)
                sh += h[j][e] * h[j][e];
        const float ih = inv_rms(row_reduce<T, false>(sh, red[par][1]), K, a.eps);
        float amax = 0.0f;
#pragma unroll
        for (int j = 0; j < CH; ++j) {
            const int c = (t + j * T) * 8;
            float w2[8];
            vec.get(2, j, w2);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                h[j][e] = h[j][e] * ih * w2[e];
                amax = magnitude_max(amax, fabsf(h[j][e]));
            }
            if constexpr (!QUANT) {
                if (c < K)
                    store_bf16<8>((uint16_t*)a.n_out + row + c, h[j]);
            }
        }
        if constexpr (QUANT) {
            // The rule of quantize_per_token_fp8, on the fp32 values.  A row
            // whose maximum is a NaN or infinite has that scale and takes the
            // division, whose NaN the clamp below keeps (clamp448 does not):
            // no codes make such a row look like a finite one.
            amax = row_reduce<T, true>(amax, red[par][2]);
            const Quot q(amax / 448.0f);
            if (t == 0)
                a.n_scales[m] = q.s;
#pragma unroll
            for (int j = 0; j < CH; ++j) {
                const int c = (t + j * T) * 8;
                float f[8];
                if (q.fast) {
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        f[e] = clamp448(q.by_reciprocal(h[j][e]));
                } else {
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const float v = q.s == 0.0f ? 0.0f : h[j][e] / q.s;
                        f[e] = v > 448.0f ? 448.0f : (v < -448.0f ? -448.0f : v);
                    }
                }
                int w0 = __builtin_amdgcn_cvt_pk_fp8_f32(f[0], f[1], 0, false);
                w0 = __builtin_amdgcn_cvt_pk_fp8_f32(f[2], f[3], w0, true);
                int w1 = __builtin_amdgcn_cvt_pk_fp8_f32(f[4], f[5], 0, false);
                w1 = __builtin_amdgcn_cvt_pk_fp8_f32(f[6], f[7], w1, true);
                if (c < K)
                    *(uint2*)((uint8_t*)a.n_out + row + c) = make_uint2((uint32_t)w0, (uint32_t)w1);
            }
        }
    }
}

// Rows as above; the vector gradients' sums stay in registers.  The rows are
// kept as they lie in memory and widened in each of the three passes over
// them, which leaves the registers for the sums.
//
// SUMS false (rows of more than 8192 columns, whose sums do not fit in the
// registers: with them K = 16384, M = 4096 spills and takes 415 us and more,
// against 156 us of memory traffic): the rows' statistics go to a.stats, and
// residual_norm_vectors_kernel forms the vector gradients from them.
template <int T, int CH, bool HAS_Y, bool F32, bool SUMS>
__global__ __launch_bounds__(T) void residual_norm_backward_kernel(NormArgs a)
{
    __shared__ float red[2][4][T / 64];
    constexpr bool AHEAD = SUMS && CH <= 2;
    const int t = threadIdx.x;
    const int K = a.K;
    const float invk = 1.0f / (float)K;
    const Vectors<T, CH> vec(a, t);
    constexpr int SCH = SUMS ? CH : 1;
    float s_pre[SCH][8], s_post[SCH][8], s_gate[SCH][8];
#pragma unroll
    for (int j = 0; j < SCH; ++j)
#pragma unroll
        for (int e = 0; e < 8; ++e)
            s_pre[j][e] = s_post[j][e] = s_gate[j][e] = 0.0f;
    struct Row {
        uint4 y[HAS_Y ? CH : 1], u[CH];
        StreamRun<F32> r[CH], d[CH];
    } next;
    auto fetch = [&](int m) __attribute__((always_inline)) {
        const size_t row = (size_t)m * K;
#pragma unroll
        for (int j = 0; j < CH; ++j) {
            const int c = (t + j * T) * 8;
            next.u[j] = make_uint4(0, 0, 0, 0);
            if constexpr (HAS_Y)
                next.y[j] = make_uint4(0, 0, 0, 0);
            next.r[j].clear();
            next.d[j].clear();
            if (m < a.M && c < K) {
                next.u[j] = *(const uint4*)(a.dn + row + c);
                if constexpr (HAS_Y)
                    next.y[j] = *(const uint4*)(a.y + row + c);
                next.r[j].load(a.r, row + c);
                if (a.dr_out)
                    next.d[j].load(a.dr_out, row + c);
            }
        }
    };
    if constexpr (AHEAD)
        fetch(blockIdx.x);
    int par = 0;
    for (int m = blockIdx.x; m < a.M; m += gridDim.x, par ^= 1) {
        const size_t row = (size_t)m * K;
        if constexpr (!AHEAD)
            fetch(m);
        const Row now = next;
        if constexpr (AHEAD)
            fetch(m + gridDim.x);
        float iy = 1.0f;
        if constexpr (HAS_Y) {
            if (a.w_post) {
                float sy = 0.0f;
#pragma unroll
                for (int j = 0; j < CH; ++j) {
                    float y[8];
                    unpack8(now.y[j], y);
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        sy += y[e] * y[e];
                }
                iy = inv_rms(row_reduce<T, false>(sy, red[par][0]), K, a.eps);
            }
        }
        // h of run j, and the normed y times w_post (p) where there is a y
        auto stream = [&](int j, float* h, float* p) __attribute__((always_inline)) {
            now.r[j].widen(h);
            if constexpr (HAS_Y) {
                float w1[8], g[8];
                unpack8(now.y[j], p);
                vec.get(0, j, w1);
                vec.get(1, j, g);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    p[e] = p[e] * iy * w1[e];
                    h[e] = a.alpha * h[e] + a.beta * (p[e] * g[e]);
                }
            }
        };
        float sh = 0.0f, suh = 0.0f;
#pragma unroll
        for (int j = 0; j < CH; ++j) {
            float h[8], p[8], u[8], w2[8];
            stream(j, h, p);
            unpack8(now.u[j], u);
            vec.get(2, j, w2);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                sh += h[e] * h[e];
                suh += u[e] * w2[e] * h[e];
            }
        }
        sh = row_reduce<T, false>(sh, red[par][1]);
        suh = row_reduce<T, false>(suh, red[par][2]);
        const float ih = inv_rms(sh, K, a.eps);
        const float mh = suh * invk * ih * ih;
        if (!SUMS && t == 0)
            *(float4*)(a.stats + 4 * (size_t)m) = make_float4(iy, ih, mh, 0.0f);
        float svy = 0.0f;
        float v[HAS_Y ? CH : 1][8];  // dy before the post-norm's own term
#pragma unroll
        for (int j = 0; j < CH; ++j) {
            const int c = (t + j * T) * 8;
            float h[8], p[8], u[8], w2[8], d[8], o[8];
            stream(j, h, p);
            unpack8(now.u[j], u);
            vec.get(2, j, w2);
            now.d[j].widen(d);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                if constexpr (SUMS)
                    s_pre[j][e] += u[e] * h[e] * ih;
                d[e] += ih * (u[e] * w2[e] - h[e] * mh);
                o[e] = a.alpha * d[e];
            }
            if (c < K)
                store_stream<F32>(a.dr, row + c, o);
            if constexpr (HAS_Y) {
                float w1[8], g[8], y[8];
                vec.get(0, j, w1);
                vec.get(1, j, g);
                unpack8(now.y[j], y);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float dt = a.beta * d[e];
                    const float dp = dt * g[e];
                    if constexpr (SUMS) {
                        s_gate[j][e] += dt * p[e];
                        s_post[j][e] += dp * (y[e] * iy);
                    }
                    v[j][e] = dp * w1[e];
                    svy += v[j][e] * y[e];
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
                float y[8], o[8];
                unpack8(now.y[j], y);
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    o[e] = iy * (v[j][e] - y[e] * my);
                if (c < K)
                    store_bf16<8>(a.dy + row + c, o);
            }
        }
    }
    if constexpr (SUMS) {
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
}

// The vector gradients' partial sums over rows blockIdx.x, + gridDim.x, ...
// for 8 columns per thread, from the rows' statistics.
template <bool HAS_Y, bool F32>
__global__ __launch_bounds__(256) void residual_norm_vectors_kernel(NormArgs a)
{
    const int K = a.K;
    const int c = (blockIdx.y * 256 + threadIdx.x) * 8;
    if (c >= K)
        return;
    const Vectors<256, 1> vec(a, c / 8);
    float w1[8], g[8], w2[8];
    vec.get(0, 0, w1);
    vec.get(1, 0, g);
    vec.get(2, 0, w2);
    float s_pre[8], s_post[8], s_gate[8];
#pragma unroll
    for (int e = 0; e < 8; ++e)
        s_pre[e] = s_post[e] = s_gate[e] = 0.0f;
#pragma unroll 2
    for (int m = blockIdx.x; m < a.M; m += gridDim.x) {
        const size_t at = (size_t)m * K + c;
        const float4 st = *(const float4*)(a.stats + 4 * (size_t)m);
        const float iy = st.x, ih = st.y, mh = st.z;
        StreamRun<F32> r, dr;
        r.load(a.r, at);
        dr.clear();
        if (a.dr_out)
            dr.load(a.dr_out, at);
        float h[8], u[8], d[8], y[8];
        r.widen(h);
        dr.widen(d);
        unpack8(*(const uint4*)(a.dn + at), u);
        if constexpr (HAS_Y)
            unpack8(*(const uint4*)(a.y + at), y);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            float p = 0.0f;
            if constexpr (HAS_Y) {
                p = y[e] * iy * w1[e];
                h[e] = a.alpha * h[e] + a.beta * (p * g[e]);
            }
            s_pre[e] += u[e] * h[e] * ih;
            if constexpr (HAS_Y) {
                const float dt = a.beta * (d[e] + ih * (u[e] * w2[e] - h[e] * mh));
                s_gate[e] += dt * p;
                s_post[e] += dt * g[e] * (y[e] * iy);
            }
        }
    }
    const size_t plane = (size_t)gridDim.x * K;
    float* part = a.partial + (size_t)blockIdx.x * K + c;
    store_f32<8>(part, s_pre);
    if constexpr (HAS_Y) {
        if (a.w_post)
            store_f32<8>(part + plane, s_post);
        if (a.gate)
            store_f32<8>(part + 2 * plane, s_gate);
    }
}

namespace {

// a launch holds less than 2^32 threads
constexpr int kMostRows = 1 << 21;

template <int T, int CH>
hipError_t forward(const NormArgs& a, hipStream_t s)
{
    // as many workgroups as the compute units hold threads for; rows of
    // several runs per thread gain nothing from a loop
    constexpr int most = CH > 1 ? kMostRows : 256 * (2048 / T);
    const unsigned grid = (unsigned)(a.M < most ? a.M : most);
    auto go = [&](auto HY, auto F, auto Q) {
        residual_norm_kernel<T, CH, decltype(HY)::value, decltype(F)::value, decltype(Q)::value>
            <<<grid, T, 0, s>>>(a);
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

template <int T, int CH, bool SUMS>
hipError_t backward(const NormArgs& a, hipStream_t s)
{
    const unsigned blocks = (unsigned)norm_backward_blocks(a.M, a.K);
    const unsigned grid = SUMS ? blocks : (unsigned)(a.M < kMostRows ? a.M : kMostRows);
    const dim3 strips(blocks, (unsigned)((a.K / 8 + 255) / 256));
    auto go = [&](auto HY, auto F) {
        residual_norm_backward_kernel<T, CH, decltype(HY)::value, decltype(F)::value, SUMS>
            <<<grid, T, 0, s>>>(a);
        if constexpr (!SUMS)
            residual_norm_vectors_kernel<decltype(HY)::value, decltype(F)::value>
                <<<strips, 256, 0, s>>>(a);
    };
    using Y = std::true_type;
    using N = std::false_type;
    switch ((a.y ? 2 : 0) + (a.r_fp32 ? 1 : 0)) {
    case 0: go(N{}, N{}); break;
    case 1: go(N{}, Y{}); break;
    case 2: go(Y{}, N{}); break;
    default: go(Y{}, Y{}); break;
    }
    return hipGetLastError();
}

}  // namespace

hipError_t launch_residual_norm(const NormArgs& a, hipStream_t s)
{
    const int runs = a.K / 8;
    if (runs <= 64)
        return forward<64, 1>(a, s);
    if (runs <= 128)
        return forward<128, 1>(a, s);
    if (runs <= 256)
        return forward<256, 1>(a, s);
    if (runs <= 512)
        return forward<512, 1>(a, s);
    if (runs <= 1024)
        return forward<512, 2>(a, s);
    if (runs <= 2048)
        return forward<1024, 2>(a, s);
    return forward<1024, 4>(a, s);
}

// Rows of partial sums: workgroups of the backward kernel, what one wave of
// workgroups with 200-odd registers fills.  More of them cost more partial
// sums than they hide (M = 1024, K = 4096: 256 workgroups 21.8 us, 512 27.5,
// 1024 35.8; M = 8192, K = 2048: 512 48.9, 1024 57.3).  Past 8192 columns,
// strips of the vectors' kernel.
int norm_backward_blocks(int64_t M, int64_t K)
{
    const int64_t runs = K / 8;
    const int64_t most = runs <= 128 ? 1024 : (runs <= 256 ? 512 : (runs <= 1024 ? 256 : 128));
    return (int)(M < most ? M : most);
}

int64_t norm_backward_stats(int64_t M, int64_t K) { return K > 8192 ? 4 * M : 0; }

hipError_t launch_residual_norm_backward(const NormArgs& a, hipStream_t s)
{
    const int runs = a.K / 8;
    if (runs <= 64)
        return backward<64, 1, true>(a, s);
    if (runs <= 128)
        return backward<128, 1, true>(a, s);
    if (runs <= 256)
        return backward<256, 1, true>(a, s);
    if (runs <= 512)
        return backward<512, 1, true>(a, s);
    if (runs <= 1024)
        return backward<512, 2, true>(a, s);
    if (runs <= 2048)
        return backward<1024, 2, false>(a, s);
    return backward<1024, 4, false>(a, s);
}

}  // namespace qll
