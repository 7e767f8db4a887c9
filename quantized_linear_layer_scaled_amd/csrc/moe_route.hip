// Routing to experts for gfx950: scores, the choice of experts, their weights,
// and the rows sorted by expert.
//
//   p = softmax(x) or 1 / (1 + e^-x);  c = p + bias, or x itself without one
//   of the `keep` groups with the largest sums of their best values, the k
//   experts with the largest c, ties to the lower index
//   w = scale p, or scale p / (sum of p over the chosen)
//
// A wave routes a token: lane l holds the VPL experts l VPL .. of it in
// registers.  A choice is right or wrong, so values next to each other have to
// be told apart: sums with a bias are formed in 64 bits (the vector units do
// them at the rate of 32 bits), and without one the logits themselves are
// compared.  The values become unsigned keys of the same order, 0 for none;
// the k largest come out one by one, each a maximum over the wave's upper key
// halves and, where several lanes share it, over the lower ones.
//
// The sort by expert is stable and without atomics whose order would show:
// every workgroup counts its chunk of tokens, and a second launch adds the
// counts before its own chunk and places the choices 64 at a time, equal
// experts of a wave being found by comparing the bits of their numbers over
// the lanes.  Up to kOneGroup choices a single workgroup does everything.
#include "ffn_epilogue.h"
#include "moe_internal.h"

namespace qll {

namespace {

constexpr int kOneGroup = 1024;  // choices that one workgroup sorts
constexpr float kNan = __builtin_nanf("");
constexpr float kInf = __builtin_inff();

// ---- wave reductions (lane 63 collects, every lane gets the result) ----

template <int CTRL, int ROWS, typename T>
__device__ __forceinline__ T dpp_or(T none, T v)
{
    if constexpr (sizeof(T) == 8) {
        const uint64_t n = __builtin_bit_cast(uint64_t, none), u = __builtin_bit_cast(uint64_t, v);
        const uint32_t lo = __builtin_amdgcn_update_dpp((int)(uint32_t)n, (int)(uint32_t)u, CTRL, ROWS, 0xF, false);
        const uint32_t hi = __builtin_amdgcn_update_dpp((int)(n >> 32), (int)(u >> 32), CTRL, ROWS, 0xF, false);
        return __builtin_bit_cast(T, ((uint64_t)hi << 32) | lo);
    } else {
        const int n = __builtin_bit_cast(int, none), u = __builtin_bit_cast(int, v);
        return __builtin_bit_cast(T, __builtin_amdgcn_update_dpp(n, u, CTRL, ROWS, 0xF, false));
    }
}
template <typename T>
__device__ __forceinline__ T last_lane(T v)
{
    if constexpr (sizeof(T) == 8) {
        const uint64_t u = __builtin_bit_cast(uint64_t, v);
        const uint32_t lo = __builtin_amdgcn_readlane((int)(uint32_t)u, 63);
        const uint32_t hi = __builtin_amdgcn_readlane((int)(u >> 32), 63);
        return __builtin_bit_cast(T, ((uint64_t)hi << 32) | lo);
    } else {
        return __builtin_bit_cast(T, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), 63));
    }
}
template <typename T, typename F>
__device__ __forceinline__ T wave_reduce(T v, T none, F&& f)
{
    v = f(v, dpp_or<0x111, 0xF>(none, v));  // row_shr 1, 2, 4, 8
    v = f(v, dpp_or<0x112, 0xF>(none, v));
    v = f(v, dpp_or<0x114, 0xF>(none, v));
    v = f(v, dpp_or<0x118, 0xF>(none, v));
    v = f(v, dpp_or<0x142, 0xA>(none, v));  // row_bcast 15, 31
    v = f(v, dpp_or<0x143, 0xC>(none, v));
    return last_lane(v);
}
__device__ __forceinline__ uint32_t wave_max(uint32_t v)
{
    return wave_reduce(v, 0u, [](uint32_t a, uint32_t b) { return a > b ? a : b; });
}
__device__ __forceinline__ float wave_max(float v)
{
    return wave_reduce(v, -kInf, [](float a, float b) { return fmaxf(a, b); });
}
template <typename T>
__device__ __forceinline__ T wave_sum(T v)
{
    return wave_reduce(v, (T)0, [](T a, T b) { return a + b; });
}

// ---- keys: unsigned numbers in the order of the values, NaN as -inf; > 0 ----

__device__ __forceinline__ uint32_t order_key(float v)
{
    v = v != v ? -kInf : v + 0.0f;  // (-0 is 0)
    const uint32_t b = __float_as_uint(v);
    return b ^ ((uint32_t)((int)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ uint64_t order_key(double v)
{
    v = v != v ? (double)-kInf : v + 0.0;
    const uint64_t b = __builtin_bit_cast(uint64_t, v);
    return b ^ ((uint64_t)((int64_t)b >> 63) | 0x8000000000000000ull);
}

__device__ __forceinline__ float logit(const void* x, int bf16, size_t at)
{
    return bf16 ? bf16_value(((const uint16_t*)x)[at]) : ((const float*)x)[at];
}

// The k largest keys, ties to the lower expert; lane j gets the j-th expert.
template <int VPL, typename KEY>
__device__ __forceinline__ int choose(KEY (&key)[VPL], int k, int lane)
{
    int mine = 0;
    for (int j = 0; j < k; ++j) {
        KEY best = key[0];
        int at = 0;
#pragma unroll
        for (int v = 1; v < VPL; ++v)
            if (key[v] > best) {
                best = key[v];
                at = v;
            }
        uint32_t hi;
        if constexpr (sizeof(KEY) == 8)
            hi = (uint32_t)(best >> 32);
        else
            hi = best;
        uint64_t who = __ballot(hi == wave_max(hi));
        if constexpr (sizeof(KEY) == 8) {
            if (who & (who - 1)) {
                const uint32_t lo = (who >> lane) & 1 ? (uint32_t)best : 0u;
                who &= __ballot(lo == wave_max(lo));
            }
        }
        const int from = __ffsll((long long)who) - 1;
        const int e = __builtin_amdgcn_readlane(lane * VPL + at, from);
        if (lane == j)
            mine = e;
#pragma unroll
        for (int v = 0; v < VPL; ++v)
            if (lane * VPL + v == e)
                key[v] = 0;
    }
    return mine;
}

// ---- the sort by expert ----

template <int WAVES>
struct SortShared {
    int base[kMoeMaxExperts];   // next row of an expert
    int total[kMoeMaxExperts];  // its choices (of a batch, or of all)
    uint16_t count[WAVES][kMoeMaxExperts];
    int wave_total[WAVES];
};

// base[e] += the choices of the experts before e (of total[]); offsets to
// memory from one workgroup.  Returns the choices of all experts.
template <int WAVES>
__device__ int scan_experts(SortShared<WAVES>& s, int E, int* offsets, bool write)
{
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    int before = 0;
    for (int e0 = 0; e0 < E; e0 += WAVES * 64) {
        const int e = e0 + (int)threadIdx.x;
        const int mine = e < E ? s.total[e] : 0;
        int sum = mine;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const int o = __shfl_up(sum, d, 64);
            if (lane >= d)
                sum += o;
        }
        if (lane == 63)
            s.wave_total[wave] = sum;
        __syncthreads();
        int lower = before;
#pragma unroll
        for (int w = 0; w < WAVES; ++w) {
            lower += w < wave ? s.wave_total[w] : 0;
            before += s.wave_total[w];
        }
        if (e < E) {
            s.base[e] += lower + sum - mine;
            if (write)
                offsets[e] = lower + sum - mine;
        }
        __syncthreads();
    }
    if (write && threadIdx.x == 0)
        offsets[E] = before;
    return before;
}

// Places the choices first .. last - 1 in order, a batch of WAVES * 64 at a
// time; id(i) is choice i's expert.
template <int WAVES, typename ID>
__device__ void place_choices(SortShared<WAVES>& s, const SortArgs& a, int first, int last, ID&& id)
{
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int bits = 32 - __clz((a.E - 1) | 1);
    for (int i0 = first; i0 < last; i0 += WAVES * 64) {
        for (int x = threadIdx.x; x < a.E; x += WAVES * 64)
#pragma unroll
            for (int w = 0; w < WAVES; ++w)
                s.count[w][x] = 0;
        __syncthreads();
        const int i = i0 + (int)threadIdx.x;
        const int e = i < last ? id(i) : -1;
        const bool live = (unsigned)e < (unsigned)a.E;
        uint64_t same = __ballot(live);
        for (int b = 0; b < bits; ++b) {
            const uint64_t set = __ballot((e >> b) & 1);
            same &= (e >> b) & 1 ? set : ~set;
        }
        const int rank = __popcll(same & ((1ull << lane) - 1));
        if (live && rank == 0)
            s.count[wave][e] = (uint16_t)__popcll(same);
        __syncthreads();
        for (int x = threadIdx.x; x < a.E; x += WAVES * 64) {
            int sum = 0;
#pragma unroll
            for (int w = 0; w < WAVES; ++w) {
                const int c = s.count[w][x];
                s.count[w][x] = (uint16_t)sum;
                sum += c;
            }
            s.total[x] = sum;
        }
        __syncthreads();
        if (i < last) {
            const int at = live ? s.base[e] + s.count[wave][e] + rank : -1;
            a.places[i] = at;
            if (live)
                a.rows[at] = i / a.k;
        }
        __syncthreads();
        for (int x = threadIdx.x; x < a.E; x += WAVES * 64)
            s.base[x] += s.total[x];
    }
}

// All choices by one workgroup.
template <int WAVES, typename ID>
__device__ void sort_choices(SortShared<WAVES>& s, const SortArgs& a, ID&& id)
{
    const int n = a.T * a.k;
    for (int e = threadIdx.x; e < a.E; e += WAVES * 64)
        s.base[e] = s.total[e] = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += WAVES * 64) {
        const int e = id(i);
        if ((unsigned)e < (unsigned)a.E)
            atomicAdd(&s.total[e], 1);
    }
    __syncthreads();
    const int placed = scan_experts(s, a.E, a.offsets, true);
    for (int i = placed + (int)threadIdx.x; i < n; i += WAVES * 64)
        a.rows[i] = -1;
    place_choices(s, a, 0, n, id);
}

// ---- kernels ----

enum Plan : int { PLAN_NONE = 0, PLAN_COUNT, PLAN_ALL };

// Tokens blockIdx.x * chunk ..; PLAN_COUNT: and the chunk's counts; PLAN_ALL:
// one workgroup, all tokens, and the sort.
template <int VPL, int WAVES, int PLAN>
__global__ __launch_bounds__(WAVES * 64) void moe_route_kernel(RouteArgs a)
{
    const SortArgs& s = a.sort;
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int E = s.E, k = s.k;
    __shared__ double group_value[WAVES][64 * VPL];
    __shared__ int counts[PLAN == PLAN_COUNT ? 64 * VPL : 1];
    __shared__ int chosen[PLAN == PLAN_ALL ? kOneGroup : 1];
    if constexpr (PLAN == PLAN_COUNT) {
        for (int e = threadIdx.x; e < E; e += WAVES * 64)
            counts[e] = 0;
        __syncthreads();
    }
    const bool grouped = a.keep < a.groups;
    const int size = E / a.groups;
    float bias[VPL];
    int group[VPL];
#pragma unroll
    for (int v = 0; v < VPL; ++v) {
        const int e = lane * VPL + v;
        bias[v] = a.bias && e < E ? a.bias[e] : 0.0f;
        group[v] = min(e / size, 63);
    }

    const int t0 = blockIdx.x * s.chunk, t1 = min(s.T, t0 + s.chunk);
    for (int t = t0 + wave; t < t1; t += WAVES) {
        const size_t row = (size_t)t * E;
        float x[VPL];
        float m = -kInf;
        bool bad = false;  // a row whose softmax is not a number
#pragma unroll
        for (int v = 0; v < VPL; ++v) {
            const int e = lane * VPL + v;
            x[v] = e < E ? logit(a.logits, a.bf16, row + e) : -kInf;
            m = fmaxf(m, x[v]);
            bad |= !(x[v] < kInf);
        }
        float z = 0.0f;
        if (a.score == SCORE_SOFTMAX) {
            m = wave_max(m);
            bad = __any(bad);
            if (!a.renorm) {
#pragma unroll
                for (int v = 0; v < VPL; ++v)
                    z += m > -kInf ? expf(x[v] - m) : 0.0f;
                z = wave_sum(z);
            }
        }
        double c[VPL];  // what groups, and choices with a bias, go by
        if (grouped || a.bias) {
            if (a.score == SCORE_SOFTMAX) {
                double sum = 0.0;
#pragma unroll
                for (int v = 0; v < VPL; ++v) {
                    c[v] = m > -kInf ? exp((double)x[v] - (double)m) : 0.0;
                    sum += c[v];
                }
                sum = wave_sum(sum);
#pragma unroll
                for (int v = 0; v < VPL; ++v)
                    c[v] = sum > 0.0 ? c[v] / sum : c[v];
            } else {
#pragma unroll
                for (int v = 0; v < VPL; ++v)
                    c[v] = 1.0 / (1.0 + exp(-(double)x[v]));
            }
#pragma unroll
            for (int v = 0; v < VPL; ++v)
                c[v] += (double)bias[v];
        }
        uint64_t open = ~0ull;  // groups to choose from
        if (grouped) {
            double* mine = group_value[wave];
#pragma unroll
            for (int v = 0; v < VPL; ++v)
                mine[lane * VPL + v] = c[v] == c[v] ? c[v] : (double)-kInf;
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            double first = -kInf, second = -kInf;
            if (lane < a.groups)
                for (int i = 0; i < size; ++i) {
                    const double v = mine[lane * size + i];
                    second = fmax(second, fmin(first, v));
                    first = fmax(first, v);
                }
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            if (a.group_best > 1 && size > 1)
                first += second;
            uint64_t key[1] = {lane < a.groups ? order_key(first) : 0};
            const int g = choose<1>(key, a.keep, lane);
            open = 0;
            for (int j = 0; j < a.keep; ++j)
                open |= 1ull << __builtin_amdgcn_readlane(g, j);
        }
        auto pickable = [&](int v) {
            return lane * VPL + v < E && ((open >> group[v]) & 1);
        };
        int id;
        if (a.bias) {
            uint64_t key[VPL];
#pragma unroll
            for (int v = 0; v < VPL; ++v)
                key[v] = pickable(v) ? order_key(c[v]) : 0;
            id = choose(key, k, lane);
        } else {
            uint32_t key[VPL];
#pragma unroll
            for (int v = 0; v < VPL; ++v)
                key[v] = pickable(v) ? order_key(x[v]) : 0;
            id = choose(key, k, lane);
        }
        float w = 0.0f;
        if (lane < k) {
            const float l = logit(a.logits, a.bf16, row + id);
            if (a.score == SCORE_SIGMOID)
                w = 1.0f / (1.0f + expf(-l));
            else
                w = bad ? kNan : (m > -kInf ? expf(l - m) : 0.0f);
        }
        if (a.renorm)
            z = wave_sum(w);
        if (a.renorm || a.score == SCORE_SOFTMAX)
            w = w == 0.0f && z == 0.0f ? 0.0f : w / z;
        if (lane < k) {
            a.ids[(size_t)t * k + lane] = id;
            a.weights[(size_t)t * k + lane] = a.scale * w;
            if constexpr (PLAN == PLAN_COUNT)
                atomicAdd(&counts[id], 1);
            if constexpr (PLAN == PLAN_ALL)
                chosen[t * k + lane] = id;
        }
    }
    if constexpr (PLAN == PLAN_COUNT) {
        __syncthreads();
        for (int e = threadIdx.x; e < E; e += WAVES * 64)
            s.hist[(size_t)blockIdx.x * E + e] = counts[e];
    }
    if constexpr (PLAN == PLAN_ALL) {
        __shared__ SortShared<WAVES> shared;
        __syncthreads();
        sort_choices(shared, s, [&](int i) { return chosen[i]; });
    }
}

// One workgroup, choices from memory.
__global__ __launch_bounds__(1024) void moe_sort_kernel(SortArgs a)
{
    __shared__ SortShared<16> shared;
    sort_choices(shared, a, [&](int i) { return a.ids[i]; });
}

__global__ __launch_bounds__(256) void moe_count_kernel(SortArgs a)
{
    __shared__ int counts[kMoeMaxExperts];
    for (int e = threadIdx.x; e < a.E; e += 256)
        counts[e] = 0;
    __syncthreads();
    const int i0 = blockIdx.x * a.chunk * a.k;
    const int i1 = min(a.T, ((int)blockIdx.x + 1) * a.chunk) * a.k;
    for (int i = i0 + (int)threadIdx.x; i < i1; i += 256) {
        const int e = a.ids[i];
        if ((unsigned)e < (unsigned)a.E)
            atomicAdd(&counts[e], 1);
    }
    __syncthreads();
    for (int e = threadIdx.x; e < a.E; e += 256)
        a.hist[(size_t)blockIdx.x * a.E + e] = counts[e];
}

// Places the choices of `per` chunks.
__global__ __launch_bounds__(512) void moe_place_kernel(SortArgs a)
{
    __shared__ SortShared<8> s;
    const int c0 = blockIdx.x * a.per, c1 = min(a.chunks, c0 + a.per);
    for (int e = threadIdx.x; e < a.E; e += 512)
        s.base[e] = s.total[e] = 0;
    __syncthreads();
    // the counts of all chunks, and of those before c0: the threads share the
    // chunks of an expert
    const int parts = max(512 / a.E, 1);
    for (int x = threadIdx.x; x < parts * a.E; x += 512) {
        const int e = x % a.E, p = x / a.E;
        int sum = 0, before = 0;
#pragma unroll 8
        for (int c = p; c < a.chunks; c += parts) {
            const int n = a.hist[(size_t)c * a.E + e];
            sum += n;
            before += c < c0 ? n : 0;
        }
        atomicAdd(&s.total[e], sum);
        atomicAdd(&s.base[e], before);
    }
    __syncthreads();
    const int placed = scan_experts(s, a.E, a.offsets, blockIdx.x == 0);
    const int n = a.T * a.k;
    for (int i = placed + blockIdx.x * 512 + (int)threadIdx.x; i < n; i += gridDim.x * 512)
        a.rows[i] = -1;
    place_choices(s, a, c0 * a.chunk * a.k, min(a.T, c1 * a.chunk) * a.k,
                  [&](int i) { return a.ids[i]; });
}

// dx of w = scale p[ids] (or renormalised), a wave per token:
//   softmax      dx = p (dp - <dp, p>), dp = scale dw at the chosen
//   renormalised the same over the chosen alone
//   sigmoid      dx = dp p (1 - p), renormalised dp = (dw - <dw, r>) / sum p
template <int VPL>
__global__ __launch_bounds__(256) void moe_route_backward_kernel(RouteBackwardArgs a)
{
    const int lane = threadIdx.x & 63;
    const int t = blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    if (t >= a.T)
        return;
    const size_t row = (size_t)t * a.E;
    const int id = lane < a.k ? a.ids[(size_t)t * a.k + lane] : -1;
    const bool live = (unsigned)id < (unsigned)a.E;
    const float dw = live ? a.scale * a.dweights[(size_t)t * a.k + lane] : 0.0f;
    const float xc = live ? logit(a.logits, a.bf16, row + id) : -kInf;
    float g;      // the gradient that reaches logit `id`
    float x[VPL], p[VPL];
    float dot = 0.0f;
    const bool dense = a.score == SCORE_SOFTMAX && !a.renorm;
    if (dense) {
        float m = -kInf, z = 0.0f;
#pragma unroll
        for (int v = 0; v < VPL; ++v) {
            const int e = lane * VPL + v;
            x[v] = e < a.E ? logit(a.logits, a.bf16, row + e) : -kInf;
            m = fmaxf(m, x[v]);
        }
        m = wave_max(m);
#pragma unroll
        for (int v = 0; v < VPL; ++v) {
            p[v] = m > -kInf || x[v] != x[v] ? expf(x[v] - m) : 0.0f;
            z += p[v];
        }
        z = wave_sum(z);
        const float iz = z == 0.0f ? 0.0f : 1.0f / z;
#pragma unroll
        for (int v = 0; v < VPL; ++v)
            p[v] *= iz;
        g = live && (m > -kInf || xc != xc) ? dw * (expf(xc - m) * iz) : 0.0f;
        dot = wave_sum(g);
    } else if (a.score == SCORE_SOFTMAX) {
        const float m = wave_max(xc);
        const float e = live && (m > -kInf || xc != xc) ? expf(xc - m) : 0.0f;
        const float z = wave_sum(e);
        const float r = z == 0.0f ? 0.0f : e / z;
        g = r * (dw - wave_sum(dw * r));
    } else {
        // p and p (1 - p) from e^-|x|: 1 - p would cancel where p is next to 1
        const float e = expf(-fabsf(xc));
        const float i = 1.0f / (1.0f + e);
        const float s = live ? (xc < 0.0f ? e * i : i) : 0.0f;
        g = dw;
        if (a.renorm) {
            const float z = wave_sum(s);
            const float iz = z == 0.0f ? 0.0f : 1.0f / z;
            g = (dw - wave_sum(dw * (s * iz))) * iz;
        }
        g = live ? g * (e * i * i) : 0.0f;
    }
    float d[VPL];
#pragma unroll
    for (int v = 0; v < VPL; ++v)
        d[v] = dense ? -p[v] * dot : 0.0f;
    for (int j = 0; j < a.k; ++j) {
        const int e = __builtin_amdgcn_readlane(id, j);
        const float gj = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, g), j));
#pragma unroll
        for (int v = 0; v < VPL; ++v)
            d[v] += lane * VPL + v == e ? gj : 0.0f;
    }
#pragma unroll
    for (int v = 0; v < VPL; ++v) {
        const int e = lane * VPL + v;
        if (e < a.E) {
            if (a.bf16)
                ((uint16_t*)a.dlogits)[row + e] = bf16_one(d[v]);
            else
                ((float*)a.dlogits)[row + e] = d[v];
        }
    }
}

// f(integral_constant<experts per lane>)
template <typename F>
hipError_t with_vpl(int E, F&& f)
{
    if (E <= 64)
        return f(std::integral_constant<int, 1>{});
    if (E <= 128)
        return f(std::integral_constant<int, 2>{});
    if (E <= 256)
        return f(std::integral_constant<int, 4>{});
    if (E <= 512)
        return f(std::integral_constant<int, 8>{});
    return f(std::integral_constant<int, 16>{});
}

}  // namespace

int64_t moe_sort_plan(SortArgs& a)
{
    const int64_t n = (int64_t)a.T * a.k;
    if (n <= kOneGroup) {
        a.chunk = a.T;
        a.chunks = a.per = 1;
        return 0;
    }
    // at most 512 chunks, and 256 workgroups that place about 1024 choices or
    // more each
    const int64_t chunk = ((int64_t)a.T + 511) / 512;
    a.chunk = (int)(chunk < 32 ? 32 : (chunk + 31) / 32 * 32);
    a.chunks = (a.T + a.chunk - 1) / a.chunk;
    const int64_t want = n / 1024 < 1 ? 1 : (n / 1024 > 256 ? 256 : n / 1024);
    a.per = (int)((a.chunks + want - 1) / want);
    return (int64_t)a.chunks * a.E * 4;
}

hipError_t launch_moe_route(const RouteArgs& a, hipStream_t stream)
{
    const SortArgs& s = a.sort;
    hipError_t rc = with_vpl(s.E, [&](auto V) {
        constexpr int VPL = decltype(V)::value;
        if (!s.offsets) {
            RouteArgs b = a;
            b.sort.chunk = 4;
            moe_route_kernel<VPL, 4, PLAN_NONE><<<(s.T + 3) / 4, 256, 0, stream>>>(b);
        } else if (!s.hist) {
            // (the groups' values of 16 waves would not fit in LDS)
            constexpr int WAVES = VPL >= 16 ? 8 : 16;
            moe_route_kernel<VPL, WAVES, PLAN_ALL><<<1, WAVES * 64, 0, stream>>>(a);
        } else {
            moe_route_kernel<VPL, 8, PLAN_COUNT><<<s.chunks, 512, 0, stream>>>(a);
        }
        return hipGetLastError();
    });
    if (rc != hipSuccess || !s.hist)
        return rc;
    moe_place_kernel<<<(s.chunks + s.per - 1) / s.per, 512, 0, stream>>>(s);
    return hipGetLastError();
}

hipError_t launch_moe_sort(const SortArgs& a, hipStream_t stream)
{
    if (!a.hist) {
        moe_sort_kernel<<<1, 1024, 0, stream>>>(a);
        return hipGetLastError();
    }
    moe_count_kernel<<<a.chunks, 256, 0, stream>>>(a);
    const hipError_t rc = hipGetLastError();
    if (rc != hipSuccess)
        return rc;
    moe_place_kernel<<<(a.chunks + a.per - 1) / a.per, 512, 0, stream>>>(a);
    return hipGetLastError();
}

hipError_t launch_moe_route_backward(const RouteBackwardArgs& a, hipStream_t stream)
{
    return with_vpl(a.E, [&](auto V) {
        moe_route_backward_kernel<decltype(V)::value><<<(a.T + 3) / 4, 256, 0, stream>>>(a);
        return hipGetLastError();
    });
}

}  // namespace qll
