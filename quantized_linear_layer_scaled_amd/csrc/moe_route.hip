// Routing to experts for gfx950: scores, the choice of experts, their weights,
// and the rows sorted by expert.
//
//   p = softmax(x) or 1 / (1 + e^-x);  c = p + bias, or x itself without one
//   of the `keep` groups with the largest sums of their best values, the k
//   experts with the largest c, ties to the lower index
//   w = scale p, or scale p / (sum of p over the chosen)
//
// A wave routes a token: lane l holds the VPL experts l VPL .. of it in
// registers.  Values become unsigned keys of the same order, 0 for none, and
// the k largest come out one by one, each a maximum over the wave.  Bound by
// the chain of these maxima (six DPP steps, a ballot and two lane reads, each
// behind the one before), not by the logits: 8191 tokens, 256 experts, top-8,
// fp32: softmax 11 us, 7.2 of it with top-1; sigmoid with a bias 13.5, and with
// 4 of 8 groups 17.5, where vector instructions take 45% of the SIMDs' cycles.
// Few experts leave lanes idle (8192 tokens of 8, top-2: 6 us).  512 experts with
// a plan have 16 waves of 128 registers and spill 15 to 27 more: 20 us with top-8,
// against 16 without a plan, in 4 waves of 164.
//
// A choice is right or wrong, so values next to each other have to be told
// apart.  Without a bias the logits themselves are compared.  With one the sums
// are formed in 32 bits first, with a bound on their error; where two picks, the
// last one and the next, or the last open group and the next are closer than
// that (one token in 400 at these sizes), the few in question, or else the
// whole token, are formed again in 64 bits.  (All of it in 64 bits: 20 us
// more; a wave that redoes its token takes about 3 us, and the launch waits for
// it.)
//
// The sort by expert is stable and without atomics whose order would show:
// every workgroup counts its chunk of tokens, and a second launch adds the
// counts before its own chunks and places the choices 64 at a time, equal
// experts of a wave being found by comparing the bits of their numbers over
// the lanes (65528 choices of 256 experts: 8.5 us, by 64 workgroups that each read
// all counts; counting them in a launch of its own 2.9).  Up to kOneGroup choices
// a single workgroup does everything (one token, 64 experts, top-8: 5.3 us).
#include "ffn_epilogue.h"
#include "moe_internal.h"

namespace qll {

namespace {

// Counts of a chunk in memory: whole 16-byte vectors.
__host__ __device__ constexpr int hist_stride(int E) { return (E + 3) / 4 * 4; }

constexpr int kOneGroup = 1024;  // choices that one workgroup sorts
constexpr float kNan = __builtin_nanf("");
constexpr float kInf = __builtin_inff();
// Sigmoids whose sum is below kDeep are e^x to 2^-50 and lose bits below
// 2^-126; with the largest logit at kNothing or below they count as 0.
constexpr float kDeep = 0x1p-56f, kNothing = -700.0f;

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
__device__ __forceinline__ T from_lane(T v, int lane)
{
    if constexpr (sizeof(T) == 8) {
        const uint64_t u = __builtin_bit_cast(uint64_t, v);
        const uint32_t lo = __builtin_amdgcn_readlane((int)(uint32_t)u, lane);
        const uint32_t hi = __builtin_amdgcn_readlane((int)(u >> 32), lane);
        return __builtin_bit_cast(T, ((uint64_t)hi << 32) | lo);
    } else {
        return __builtin_bit_cast(T, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), lane));
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
    return from_lane(v, 63);
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

// e^z, the exponent's rounding and the hardware's 2^y (1 ulp) apart
__device__ __forceinline__ float exp_f(float z)
{
    return __builtin_amdgcn_exp2f(z * 1.442695041f);
}

// 2^y for |y| <= 1000, to 2^-51 of itself, and 0 for -1100: the Taylor series of
// the fraction.
// (The library's exp and division take three times as many instructions; a
// wave forms a value per expert.)
__device__ __forceinline__ double pow2(double y)
{
    const double n = __builtin_rint(y), f = y - n;
    double p = 2.5678435993488196e-11;
    p = __builtin_fma(p, f, 4.44553827187081e-10);
    p = __builtin_fma(p, f, 7.054911620801121e-09);
    p = __builtin_fma(p, f, 1.0178086009239696e-07);
    p = __builtin_fma(p, f, 1.3215486790144305e-06);
    p = __builtin_fma(p, f, 1.5252733804059838e-05);
    p = __builtin_fma(p, f, 0.00015403530393381606);
    p = __builtin_fma(p, f, 0.0013333558146428441);
    p = __builtin_fma(p, f, 0.009618129107628477);
    p = __builtin_fma(p, f, 0.055504108664821576);
    p = __builtin_fma(p, f, 0.2402265069591007);
    p = __builtin_fma(p, f, 0.6931471805599453);
    p = __builtin_fma(p, f, 1.0);
    return __builtin_amdgcn_ldexp(p, (int)n);
}
constexpr double kLog2e = 1.4426950408889634;
__device__ __forceinline__ double reciprocal(double d)
{
    double r = __builtin_amdgcn_rcp(d);
    r = __builtin_fma(r, __builtin_fma(-d, r, 1.0), r);
    return __builtin_fma(r, __builtin_fma(-d, r, 1.0), r);
}

// A lane's VPL logits of a row of E; those past the end are not numbers.
template <int VPL, bool BF16>
__device__ __forceinline__ void load_logits(const void* p, size_t row, int E, int lane, float (&x)[VPL])
{
    // (all loads are under way before the first is used)
    if constexpr (!BF16 && VPL >= 4) {
        if (E % 4 == 0) {
#pragma unroll
            for (int v = 0; v < VPL; v += 4) {
                const float4 w = *(const float4*)((const float*)p + row + min(lane * VPL + v, E - 4));
                x[v] = w.x; x[v + 1] = w.y; x[v + 2] = w.z; x[v + 3] = w.w;
            }
            return;
        }
    }
    if constexpr (BF16 && VPL >= 8) {
        if (E % 8 == 0) {
#pragma unroll
            for (int v = 0; v < VPL; v += 8)
                load_bf16<8>((const uint16_t*)p + row + min(lane * VPL + v, E - 8), &x[v]);
            return;
        }
    }
#pragma unroll
    for (int v = 0; v < VPL; ++v) {
        const size_t at = row + min(lane * VPL + v, E - 1);
        x[v] = BF16 ? bf16_value(((const uint16_t*)p)[at]) : ((const float*)p)[at];
    }
}

__device__ __forceinline__ float logit(const void* x, int bf16, size_t at)
{
    return bf16 ? bf16_value(((const uint16_t*)x)[at]) : ((const float*)x)[at];
}

// The k largest keys, ties to the lower expert; lane j gets the j-th expert,
// and its key (0: there is none).
template <int VPL, typename KEY>
__device__ __forceinline__ int choose(KEY (&key)[VPL], int k, int lane, uint32_t& mine_key)
{
    int mine = 0;
    mine_key = 0;
    for (int j = 0; j < k; ++j) {
        KEY best = key[0];
        int at = lane * VPL;
#pragma unroll
        for (int v = 1; v < VPL; ++v) {
            const bool more = key[v] > best;
            best = more ? key[v] : best;
            at = more ? lane * VPL + v : at;
        }
        const uint32_t hi = (uint32_t)(best >> (8 * sizeof(KEY) - 32));
        const uint32_t most = wave_max(hi);
        uint64_t who = __ballot(hi == most);
        if constexpr (sizeof(KEY) == 8) {
            if (who & (who - 1)) {
                const uint32_t lo = (who >> lane) & 1 ? (uint32_t)best : 0u;
                who &= __ballot(lo == wave_max(lo));
            }
        }
        const int from = __ffsll((long long)who) - 1;
        const int e = __builtin_amdgcn_readlane(at, from);
        mine = lane == j ? e : mine;
        mine_key = lane == j ? most : mine_key;
#pragma unroll
        for (int v = 0; v < VPL; ++v)
            key[v] = lane * VPL + v == e ? 0 : key[v];
    }
    return mine;
}
__device__ __forceinline__ float key_value(uint32_t key)
{
    return __uint_as_float(key & 0x80000000u ? key ^ 0x80000000u : ~key);
}
// Whether two of the first n picks, one after the other, or the last of them
// and the next, are closer than their errors: `error`, and 2^-22 of either's
// size.  (A lane without a pick has key 0.  The pick behind lane 63's is not known
// and counts as close: topk = 64 with a bias goes on in 64 bits, 24 us for 1024
// tokens of 256 experts, where topk = 62 takes 17.)
__device__ __forceinline__ bool too_close(uint32_t key, int n, int lane, float error)
{
    const uint32_t after = __shfl_down(key, 1, 64);
    const float a = key_value(key), b = key_value(after);
    const float gap = a - b;
    return __any(lane < n && after != 0 && gap < kInf && gap <= error + 0x1p-22f * (fabsf(a) + fabsf(b)));
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

// The first n picks in the order of their sigmoids and biases in 64 bits, where
// nothing else comes into question; `real`: a lane's pick is one.
__device__ __forceinline__ int exact_order(const RouteArgs& a, int id, bool real, int n, int lane,
                                           size_t row, bool bf16)
{
    double c = -kInf;
    if (real) {
        const float x = logit(a.logits, bf16, row + id);
        const double e = pow2(fmin(fmax((double)x * -kLog2e, -1000.0), 1000.0));
        const double p = reciprocal(1.0 + e) + (double)a.bias[id];
        c = x == x && p == p ? p : (double)-kInf;
    } else {
        id = 0x7FFFFFFF;  // behind all that are
    }
    int rank = 0;
    for (int i = 0; i < n; ++i) {
        const double other = from_lane(c, i);
        const int its = __builtin_amdgcn_readlane(id, i);
        rank += other > c || (other == c && (its < id || (its == id && i < lane)));
    }
    return __builtin_amdgcn_ds_permute((lane < n ? rank : lane) << 2, id);
}

// What a lane knows of the experts: lane l holds l VPL .. of them.
template <int VPL>
struct Experts {
    int E, lane;
    int size;   // experts of a group
    int lanes;  // lanes of a group, a power of two, or 0 where it does not fill lanes
    float bias[VPL];
    int group[VPL];

    __device__ __forceinline__ Experts(const RouteArgs& a, int l) : E(a.sort.E), lane(l)
    {
        size = E / a.groups;
        lanes = size % VPL ? 0 : size / VPL;
        lanes = lanes & (lanes - 1) ? 0 : lanes;
#pragma unroll
        for (int v = 0; v < VPL; ++v) {
            const int e = min(lane * VPL + v, E - 1);
            bias[v] = a.bias ? a.bias[e] : 0.0f;
            group[v] = min(e / size, 63);
        }
    }
    __device__ __forceinline__ bool has(int v) const { return lane * VPL + v < E; }

    // The open groups by the values c (`buffer`: 64 VPL of them, the wave's);
    // margin: how far the last open one is from the next.
    template <typename T>
    __device__ __forceinline__ uint64_t open(const RouteArgs& a, const T (&c)[VPL], T* buffer,
                                             T& margin) const
    {
        // the two largest of each group, in its first lane
        const T none = -kInf;
        T first = none, second = none;
        const auto add = [&](T x) {
            second = fmax(second, fmin(first, x));
            first = fmax(first, x);
        };
        const auto join = [&](T f, T s2) {
            second = fmax(fmax(second, s2), fmin(first, f));
            first = fmax(first, f);
        };
        if (lanes) {
#pragma unroll
            for (int v = 0; v < VPL; ++v)
                add(has(v) && c[v] == c[v] ? c[v] : none);
            // neighbours, pairs, halves and rows of 16 lanes trade theirs
            if (lanes > 1)
                join(dpp_or<0xB1, 0xF>(none, first), dpp_or<0xB1, 0xF>(none, second));
            if (lanes > 2)
                join(dpp_or<0x4E, 0xF>(none, first), dpp_or<0x4E, 0xF>(none, second));
            if (lanes > 4)
                join(dpp_or<0x141, 0xF>(none, first), dpp_or<0x141, 0xF>(none, second));
            if (lanes > 8)
                join(dpp_or<0x140, 0xF>(none, first), dpp_or<0x140, 0xF>(none, second));
            for (int d = 16; d < lanes; d <<= 1)
                join(__shfl_xor(first, d, 64), __shfl_xor(second, d, 64));
        } else {
#pragma unroll
            for (int v = 0; v < VPL; ++v)
                buffer[lane * VPL + v] = c[v] == c[v] ? c[v] : none;
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            if (lane < a.groups)
                for (int i = 0; i < size; ++i)
                    add(buffer[lane * size + i]);
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        }
        if (a.group_best > 1 && size > 1)
            first += second;
        // (+infinity and -infinity, of biases, are no number: below all others)
        first = first == first ? first : none;
        // a group's rank: how many are better, or as good and before it
        const int step = lanes ? lanes : 1;  // lanes from group to group
        int rank = 0;
        for (int g = 0; g < a.groups; ++g) {
            const T other = from_lane(first, g * step);
            rank += other > first || (other == first && g * step < lane);
        }
        const bool real = lane % step == 0 && lane < a.groups * step;
        const uint64_t kept = __ballot(real && rank < a.keep);
        const T last = from_lane(first, __ffsll((long long)__ballot(real && rank == a.keep - 1)) - 1);
        const T next = from_lane(first, __ffsll((long long)__ballot(real && rank == a.keep)) - 1);
        margin = last - next;
        // (one bit per group)
        uint64_t bits = 0;
        for (uint64_t left = kept; left; left &= left - 1)
            bits |= 1ull << ((__ffsll((long long)left) - 1) / step);
        return bits;
    }
};

// The choice in 64 bits: lane j gets the j-th expert.
template <int VPL>
__device__ __forceinline__ int exact_choice(const RouteArgs& a, const Experts<VPL>& ex,
                                            const float (&x)[VPL], float m, double* buffer)
{
    double c[VPL];
    if (a.score == SCORE_SOFTMAX) {
        double sum = 0.0;
#pragma unroll
        for (int v = 0; v < VPL; ++v) {
            const double e = pow2(fmax(((double)x[v] - (double)m) * kLog2e, -1100.0));
            c[v] = x[v] > -kInf ? e : 0.0;
            sum += c[v];
        }
        sum = wave_sum(sum);
        const double scale = sum > 0.0 ? reciprocal(sum) : 0.0;
#pragma unroll
        for (int v = 0; v < VPL; ++v)
            c[v] = x[v] == x[v] ? c[v] * scale : kNan;
    } else {
#pragma unroll
        for (int v = 0; v < VPL; ++v) {
            const double e = pow2(fmin(fmax((double)x[v] * -kLog2e, -1000.0), 1000.0));
            const double p = reciprocal(1.0 + e);
            c[v] = x[v] == x[v] ? p : kNan;
        }
    }
#pragma unroll
    for (int v = 0; v < VPL; ++v)
        c[v] += (double)ex.bias[v];
    uint32_t unused;
    double margin;
    const uint64_t open = a.keep < a.groups ? ex.open(a, c, buffer, margin) : ~0ull;
    uint64_t key[VPL];
#pragma unroll
    for (int v = 0; v < VPL; ++v) {
        // without a bias the logits decide
        const uint64_t k = a.bias ? order_key(c[v]) : (uint64_t)order_key(x[v]) << 32;
        key[v] = ex.has(v) && ((open >> ex.group[v]) & 1) ? k : 0;
    }
    return choose(key, a.sort.k, ex.lane, unused);
}

// Tokens blockIdx.x * chunk ..; PLAN_COUNT: and the chunk's counts; PLAN_ALL:
// one workgroup, all tokens, and the sort.
template <int VPL, bool BF16, int WAVES, int PLAN>
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
        for (int e = threadIdx.x; e < hist_stride(E); e += WAVES * 64)
            counts[e] = 0;
        __syncthreads();
    }
    const bool grouped = a.keep < a.groups;
    const Experts<VPL> ex(a, lane);

    const int t0 = blockIdx.x * s.chunk, t1 = min(s.T, t0 + s.chunk);
    float next[VPL];
    if (t0 + wave < t1)
        load_logits<VPL, BF16>(a.logits, (size_t)(t0 + wave) * E, E, lane, next);
    for (int t = t0 + wave; t < t1; t += WAVES) {
        float x[VPL];
        float m = -kInf;
        bool bad = false;  // a row whose softmax is not a number
#pragma unroll
        for (int v = 0; v < VPL; ++v)
            x[v] = lane * VPL + v < E ? next[v] : -kInf;
        if (t + WAVES < t1)  // (the next token's are on their way under this one)
            load_logits<VPL, BF16>(a.logits, (size_t)(t + WAVES) * E, E, lane, next);
#pragma unroll
        for (int v = 0; v < VPL; ++v) {
            m = fmaxf(m, x[v]);
            bad |= !(x[v] < kInf);
        }
        bad = __any(bad);
        float z = 0.0f;
        // scores, and what two of them may be off by (a sigmoid 1.1 2^-22)
        float c[VPL];
        float error = 0x1p-20f;
        if (a.score == SCORE_SOFTMAX) {
            m = wave_max(m);
            if (!a.renorm || grouped || a.bias) {
#pragma unroll
                for (int v = 0; v < VPL; ++v) {
                    c[v] = m > -kInf ? exp_f(x[v] - m) : 0.0f;
                    z += c[v];
                }
                z = wave_sum(z);
            }
        }
        int id = 0;
        float l = 0.0f;  // lane j: the j-th expert and its logit
        uint32_t picked;
        bool again = false;  // too close to call
        uint64_t open = ~0ull;  // groups to choose from
        if (grouped || a.bias) {
            if (a.score == SCORE_SOFTMAX) {
                // (p D < 0.4 for p = e^-D; the sum's error adds 40 u of p <= 1 / z)
                const float iz = z > 0.0f ? 1.0f / z : 0.0f;
                error = 0x1p-22f * (0.5f + 42.0f * iz);
#pragma unroll
                for (int v = 0; v < VPL; ++v)
                    c[v] *= iz;
            } else {
#pragma unroll
                for (int v = 0; v < VPL; ++v)
                    c[v] = sigmoid_f(x[v]);
            }
#pragma unroll
            for (int v = 0; v < VPL; ++v)
                c[v] += ex.bias[v];
            if (grouped) {
                // (the sums' roundings, of four values and two sums; an infinite
                // value, from a bias, has none: 25 us with one such bias for the
                // prompt above, as without, and 37 where every token is formed again,
                // as with one of -1e9)
                float most = 0.0f;
#pragma unroll
                for (int v = 0; v < VPL; ++v)
                    most = fmaxf(most, fabsf(c[v]) < kInf ? fabsf(c[v]) : 0.0f);
                const float group_error = 0x1p-20f * wave_max(most);
                float margin;
                open = ex.open(a, c, (float*)group_value[wave], margin);
                again = !(margin > 2.0f * error + group_error);
            }
        }
        uint32_t key[VPL];
#pragma unroll
        for (int v = 0; v < VPL; ++v)
            key[v] = ex.has(v) && ((open >> ex.group[v]) & 1) ? order_key(a.bias ? c[v] : x[v]) : 0;
        id = choose(key, a.bias ? k + 2 : k, lane, picked);
        if (a.bias && too_close(picked, k, lane, error)) {
            // sigmoids: the picks and the next two in 64 bits, if no others come
            // into question
            const uint32_t after = k + 1 < 64 ? (uint32_t)__builtin_amdgcn_readlane((int)picked, k + 1) : 1u;
            const float last = key_value(__builtin_amdgcn_readlane((int)picked, k - 1)), next = key_value(after);
            const bool enough = after == 0 || last - next > error + 0x1p-22f * (fabsf(last) + fabsf(next));
            if (a.score == SCORE_SIGMOID && !again && enough && k + 2 <= 64)
                id = exact_order(a, id, picked != 0, k + 2, lane, (size_t)t * E, BF16);
            else
                again = true;
        }
        if (again)
            id = exact_choice(a, ex, x, m, group_value[wave]);
        if (lane < k)
            l = again || a.bias || bad ? logit(a.logits, BF16, (size_t)t * E + id) : key_value(picked);
        float w = 0.0f;
        if (a.score == SCORE_SOFTMAX && a.renorm)
            m = wave_max(lane < k ? l : -kInf);
        if (lane < k) {
            if (a.score == SCORE_SIGMOID)
                w = sigmoid_f(l);
            else
                w = bad ? kNan : (m > -kInf ? exp_f(l - m) : 0.0f);
        }
        if (a.renorm) {
            z = wave_sum(w);
            // sigmoids next to nothing (kDeep): relative to the largest they are not
            if (a.score == SCORE_SIGMOID && z < kDeep) {
                m = wave_max(lane < k ? l : -kInf);
                w = lane < k && m > kNothing ? exp_f(l - m) : 0.0f;
                z = wave_sum(w);
            }
        }
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
        for (int e = threadIdx.x; e < hist_stride(E); e += WAVES * 64)
            s.hist[(size_t)blockIdx.x * hist_stride(E) + e] = counts[e];
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
    for (int e = threadIdx.x; e < hist_stride(a.E); e += 256)
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
    for (int e = threadIdx.x; e < hist_stride(a.E); e += 256)
        a.hist[(size_t)blockIdx.x * hist_stride(a.E) + e] = counts[e];
}

// Places the choices of `per` chunks.
__global__ __launch_bounds__(1024) void moe_place_kernel(SortArgs a)
{
    constexpr int N = 1024;
    __shared__ SortShared<N / 64> s;
    const int c0 = blockIdx.x * a.per, c1 = min(a.chunks, c0 + a.per);
    for (int e = threadIdx.x; e < a.E; e += N)
        s.base[e] = s.total[e] = 0;
    __syncthreads();
    // the counts of all chunks, and of those before c0: the threads share the
    // chunks of four experts
    const int fours = hist_stride(a.E) / 4, parts = N / fours;
    const int f = threadIdx.x % fours, p = threadIdx.x / fours;
    if (p < parts) {
        int4 sum = {0, 0, 0, 0}, before = {0, 0, 0, 0};
#pragma unroll 8
        for (int c = p; c < a.chunks; c += parts) {
            const int4 n = *(const int4*)(a.hist + (size_t)c * (4 * fours) + 4 * f);
            const int in = c < c0 ? -1 : 0;
            sum.x += n.x; sum.y += n.y; sum.z += n.z; sum.w += n.w;
            before.x += n.x & in; before.y += n.y & in; before.z += n.z & in; before.w += n.w & in;
        }
        const int all[4] = {sum.x, sum.y, sum.z, sum.w}, less[4] = {before.x, before.y, before.z, before.w};
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (4 * f + i < a.E) {
                atomicAdd(&s.total[4 * f + i], all[i]);
                atomicAdd(&s.base[4 * f + i], less[i]);
            }
    }
    __syncthreads();
    const int placed = scan_experts(s, a.E, a.offsets, blockIdx.x == 0);
    const int n = a.T * a.k;
    for (int i = placed + blockIdx.x * N + (int)threadIdx.x; i < n; i += gridDim.x * N)
        a.rows[i] = -1;
    place_choices(s, a, c0 * a.chunk * a.k, min(a.T, c1 * a.chunk) * a.k,
                  [&](int i) { return a.ids[i]; });
}

// dx of w = scale p[ids] (or renormalised), a wave per token (8192 tokens, fp32,
// top-8: 64 experts 5.2 us, 256 6.8, 512, which lanes store one by one, 15.5):
//   softmax      dx = p (dp - <dp, p>), dp = scale dw at the chosen
//   renormalised the same over the chosen alone
//   sigmoid      dx = dw p (1 - p), renormalised (dw - <dw, r>) r (1 - p)
template <int VPL, bool BF16>
__global__ __launch_bounds__(256) void moe_route_backward_kernel(RouteBackwardArgs a)
{
    const int lane = threadIdx.x & 63;
    const int t = blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    if (t >= a.T)
        return;
    const size_t row = (size_t)t * a.E;
    const bool dense = a.score == SCORE_SOFTMAX && !a.renorm;
    float all[VPL];
    if (dense)
        load_logits<VPL, BF16>(a.logits, row, a.E, lane, all);
    const int id = lane < a.k ? a.ids[(size_t)t * a.k + lane] : -1;
    const bool live = (unsigned)id < (unsigned)a.E;
    const float dw = live ? a.scale * a.dweights[(size_t)t * a.k + lane] : 0.0f;
    const float xc = live ? logit(a.logits, BF16, row + id) : -kInf;
    float g;      // the gradient that reaches logit `id`
    float x[VPL], p[VPL];
    float dot = 0.0f;
    if (dense) {
        float m = -kInf, z = 0.0f;
#pragma unroll
        for (int v = 0; v < VPL; ++v) {
            x[v] = lane * VPL + v < a.E ? all[v] : -kInf;
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
        if (a.renorm) {
            float s = live ? (xc < 0.0f ? e * i : i) : 0.0f;
            float z = wave_sum(s);
            if (z < kDeep) {
                const float m = wave_max(xc);
                s = live && m > kNothing ? expf(xc - m) : 0.0f;
                z = wave_sum(s);
            }
            const float r = z == 0.0f ? 0.0f : s / z;
            g = r * (xc < 0.0f ? i : e * i) * (dw - wave_sum(dw * r));
        } else {
            g = dw * (e * i * i);
        }
        g = live ? g : 0.0f;
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
            if constexpr (BF16)
                ((uint16_t*)a.dlogits)[row + e] = bf16_one(d[v]);
            else
                ((float*)a.dlogits)[row + e] = d[v];
        }
    }
}

// f(integral_constant<experts per lane>, integral_constant<bf16>)
template <bool BF16, typename F>
hipError_t with_vpl(int E, F&& f)
{
    constexpr std::integral_constant<bool, BF16> type = {};
    if (E <= 64)
        return f(std::integral_constant<int, 1>{}, type);
    if (E <= 128)
        return f(std::integral_constant<int, 2>{}, type);
    if (E <= 256)
        return f(std::integral_constant<int, 4>{}, type);
    if (E <= 512)
        return f(std::integral_constant<int, 8>{}, type);
    return f(std::integral_constant<int, 16>{}, type);
}
template <typename F>
hipError_t with_logits(int E, int bf16, F&& f)
{
    return bf16 ? with_vpl<true>(E, f) : with_vpl<false>(E, f);
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
    // Chunks of 16 tokens (one for each wave) up to 4096, then of 32; at most
    // 512 of them, and at most 256 workgroups that place whole batches of 1024
    // choices or, of large chunks, one each.
    const int64_t chunk = ((int64_t)a.T + 511) / 512;
    a.chunk = a.T <= 4096 ? 16 : (int)(chunk < 32 ? 32 : (chunk + 31) / 32 * 32);
    a.chunks = (a.T + a.chunk - 1) / a.chunk;
    const int batch = 1024 / (a.chunk * a.k), least = (a.chunks + 255) / 256;
    a.per = batch > least ? batch : least;
    return (int64_t)a.chunks * hist_stride(a.E) * 4;
}

hipError_t launch_moe_route(const RouteArgs& a, hipStream_t stream)
{
    const SortArgs& s = a.sort;
    hipError_t rc = with_logits(s.E, a.bf16, [&](auto V, auto B) {
        constexpr int VPL = decltype(V)::value;
        constexpr bool BF16 = decltype(B)::value;
        if (!s.offsets) {
            RouteArgs b = a;
            b.sort.chunk = s.T > kLaunchWaves ? 8 : 4;
            moe_route_kernel<VPL, BF16, 4, PLAN_NONE>
                <<<(s.T + b.sort.chunk - 1) / b.sort.chunk, 256, 0, stream>>>(b);
        } else if (!s.hist) {
            // (the groups' values of 16 waves would not fit in LDS)
            constexpr int WAVES = VPL >= 16 ? 8 : 16;
            moe_route_kernel<VPL, BF16, WAVES, PLAN_ALL><<<1, WAVES * 64, 0, stream>>>(a);
        } else {
            constexpr int WAVES = VPL >= 16 ? 8 : 16;
            moe_route_kernel<VPL, BF16, WAVES, PLAN_COUNT><<<s.chunks, WAVES * 64, 0, stream>>>(a);
        }
        return hipGetLastError();
    });
    if (rc != hipSuccess || !s.hist)
        return rc;
    moe_place_kernel<<<(s.chunks + s.per - 1) / s.per, 1024, 0, stream>>>(s);
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
    moe_place_kernel<<<(a.chunks + a.per - 1) / a.per, 1024, 0, stream>>>(a);
    return hipGetLastError();
}

hipError_t launch_moe_route_backward(const RouteBackwardArgs& a, hipStream_t stream)
{
    return with_logits(a.E, a.bf16, [&](auto V, auto B) {
        constexpr bool BF16 = decltype(B)::value;
        hipError_t rc = hipSuccess;
        for (int t = 0; t < a.T && rc == hipSuccess; t += kLaunchWaves) {
            RouteBackwardArgs b = a;
            const size_t row = (size_t)t * a.E * (BF16 ? 2 : 4);
            b.logits = (const char*)a.logits + row;
            b.dlogits = (char*)a.dlogits + row;
            b.ids = a.ids + (size_t)t * a.k;
            b.dweights = a.dweights + (size_t)t * a.k;
            b.T = a.T - t < kLaunchWaves ? a.T - t : kLaunchWaves;
            moe_route_backward_kernel<decltype(V)::value, BF16><<<(b.T + 3) / 4, 256, 0, stream>>>(b);
            rc = hipGetLastError();
        }
        return rc;
    });
}

}  // namespace qll
