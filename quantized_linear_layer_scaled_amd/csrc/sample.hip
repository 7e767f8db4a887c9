// Sampling from rows of logits for gfx950: temperature, top-k, top-p and
// min-p, and one token per row from a given random number.
//
//   d_i = (max - x_i) / T, weights w_i = e^-d_i; the tokens in the order of
//   falling logits, ties by rising index; kept are the first top_k of them,
//   of these the ones before which less than top_p of their weight lies, and of
//   these the ones with w >= min_p, the first token always.  The token is the
//   first of the order up to which more than u of the kept weight lies.
//
// Every set of that definition is a front part of one order, so a row needs
// no sorting: only where in the order a count, a weight or a value is reached.
// A row is mostly read once.  Its values go to one of kBins bins of
// (ref - x) / T, 1 / kPerUnit wide, each by one LDS addition that carries a
// count and a weight, and those among the largest also to a list; ref and the
// list's threshold come from a sample of the row.  Prefix sums over the bins
// say in which bin an answer lies.  Mostly (top-k, a peaked distribution) the
// list holds all values down to there; they are sorted and added up one by one.
// Else a second pass gathers the bins that matter.
//
// A token is right or wrong, so weights are formed to well below a token's
// share: within a bin w = e^-(b / kPerUnit) (1 - g), g = 1 - e^-(f / kPerUnit)
// with f the fraction of the bin (64-bit arithmetic, four terms: 2^-37), and
// the additions are integers: the count above, g in `ebits` fractional bits
// below (34 for vocabularies below 2^18), which no order of additions changes.
// Weights below e^-31.9 of the largest are left out: 2^20 of them are less than
// 1.5e-8 of the total, below the last bit of u next to 1 (6e-8).
//
// The bins cover 16 T above ref and 32 T below; a row whose maximum lies above
// starts again with ref = the maximum.  A bin that holds more values than the
// list (equal logits, a wide temperature) is narrowed down by further passes
// over its keys, 4096 ways each; equal keys are counted by blocks of the row.
// So two kinds of rows are read twice that need not be: at a low temperature one
// with a winner outside of the sample, and one of which a wave samples nothing but
// -infinity (a masked block): the threshold is then the lowest number, and the list
// overflows.
//
// A workgroup takes a row, or one of `parts` of it where there are few rows;
// then a second launch adds the parts' bins and finishes.
//
// Measured: one row of 151936 bf16 logits in 8 parts 9.8 us, the second launch
// 13 where the list holds the answer and up to 42 for a flat row under top-p;
// 256 fp32 rows of mixed options 85: 33 for the read (4.7 TB/s), then the
// flattest row's second read 30 and its two searches 16; 48 rows of 50021 under
// top-p 10 and 33.  With 24 likely tokens, T = 0.8 and top-p the second launch takes
// 12 for one row, 18 with an eighth masked, and 23 at T = 0.2 with one value far
// above; 256 rows 68, 86 and 62.  Past the first read a row is a chain of short
// steps of one workgroup.  (The second read over as many workgroups as the first:
// 26 us in place of 36 for one row, but 29 in place of 21 for 48, the joining of the
// parts taking 6.)  The kernels that finish a row hold every search: 128 registers
// and 15 to 28 more that are spilled (56 to 96 bytes a lane; the kernel that reads a
// part takes 56 to 68), so that the second read has none for more loads, and 62 to
// 66 KB of code, most of which a row fetches for the first time.
#include "ffn_epilogue.h"
#include "sample_internal.h"

namespace qll {

namespace {

constexpr int kThreads = 1024;
constexpr int kWaves = kThreads / 64;
constexpr int kPer = 3;                  // bins of a thread
constexpr int kBins = kPer * kThreads;
constexpr int kPerUnit = 64;             // bins per unit of (ref - x) / T
// the bin of ref, 16 units above (a thread's first, whose weight at ref is
// exactly 1: equal weights stay equal)
constexpr int kAbove = 16 * kPerUnit / kPer * kPer + kPer;
constexpr int kCap = 4096;               // values that are kept beside the bins
constexpr int kFew = 256;                // values that are sorted
constexpr int kSub = 4096;               // ways a bin is narrowed down
constexpr float kInf = __builtin_inff();
constexpr float kMax = 3.402823466e38f;

// A value that is the same in every lane, in scalar registers: the row's
// numbers would take most of the vector registers.
template <typename T>
__device__ __forceinline__ T uniform(T v)
{
    if constexpr (sizeof(T) == 8) {
        const uint64_t u = __builtin_bit_cast(uint64_t, v);
        const uint32_t lo = __builtin_amdgcn_readfirstlane((int)(uint32_t)u);
        const uint32_t hi = __builtin_amdgcn_readfirstlane((int)(u >> 32));
        return __builtin_bit_cast(T, ((uint64_t)hi << 32) | lo);
    } else {
        return __builtin_bit_cast(T, __builtin_amdgcn_readfirstlane(__builtin_bit_cast(int, v)));
    }
}

// Unsigned numbers in the order of the values; NaN as -inf, -0 as 0.
__device__ __forceinline__ uint32_t key_of(float v)
{
    v = v != v ? -kInf : v + 0.0f;
    const uint32_t b = __float_as_uint(v);
    return b ^ ((uint32_t)((int)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ float value_of(uint32_t key)
{
    return __uint_as_float(key & 0x80000000u ? key ^ 0x80000000u : ~key);
}
__device__ __forceinline__ uint64_t entry(float x, int i)
{
    return ((uint64_t)~key_of(x) << 32) | (uint32_t)i;
}
__device__ __forceinline__ uint32_t entry_key(uint64_t e) { return ~(uint32_t)(e >> 32); }

// What a part of a row leaves for the second launch.
struct Part {
    uint64_t bins[kBins];
    uint64_t list[kSamplePartList];
    uint32_t n;  // values for the list (more than it holds: not all are there)
    float max;
    float ref, threshold;
};

struct Shared {
    uint64_t bins[kBins];        // then: weight before each bin, as doubles
    uint32_t counts[kBins + 1];  // values before each bin
    uint64_t cand[kCap];         // values of some bins
    uint64_t list[kSub];         // few values, sorted, or the finer bins of a search
    double sums[kFew];           // weight up to and with each of these
    double wave_weight[kWaves];
    uint32_t wave_count[kWaves];
    float wave_max[kWaves];
    uint32_t n, ncand;
    int found, last, index;
};

// A place in the order.
struct Place {
    uint32_t key;
    int index;      // of the token, or -1: it is the rank-th with this key
    int rank;       // (from 1)
    double weight;  // of one value
    double upto;    // weight up to and with this place
};

// Values of a row, 16 bytes at a time.
template <bool BF16>
struct Row {
    static constexpr int VE = BF16 ? 8 : 4;
    const void* p;
    int V;

    __device__ __forceinline__ int vectors() const { return V / VE; }
    __device__ __forceinline__ u32x4_any load(int v) const
    {
        return *(const u32x4_any*)((const char*)p + (size_t)v * 16);
    }
    static __device__ __forceinline__ void widen(const u32x4_any& w, float (&x)[VE])
    {
#pragma unroll
        for (int e = 0; e < VE; ++e) {
            if constexpr (BF16)
                x[e] = __uint_as_float(e & 1 ? w[e / 2] & 0xFFFF0000u : w[e / 2] << 16);
            else
                x[e] = __uint_as_float(w[e]);
        }
    }
    __device__ __forceinline__ float at(int i) const
    {
        return BF16 ? bf16_value(((const uint16_t*)p)[i]) : ((const float*)p)[i];
    }
    // f(values, index of the first, how many) for vectors v0 .. v1 - 1, and
    // the values behind the last whole vector where `tail`
    template <typename F>
    __device__ __forceinline__ void each(int v0, int v1, bool tail, F&& f) const
    {
        // (the next vectors are loaded before these are used)
        constexpr int U = 16 / VE;
        int v = v0 + (int)threadIdx.x;
        u32x4_any next[U];
        if (v < v1) {
#pragma unroll
            for (int k = 0; k < U; ++k)
                next[k] = load(min(v + k * kThreads, v1 - 1));
        }
        for (; v < v1; v += U * kThreads) {
            u32x4_any w[U];
#pragma unroll
            for (int k = 0; k < U; ++k)
                w[k] = next[k];
            if (v + U * kThreads < v1) {
#pragma unroll
                for (int k = 0; k < U; ++k)
                    next[k] = load(min(v + (U + k) * kThreads, v1 - 1));
            }
#pragma unroll
            for (int k = 0; k < U; ++k) {
                float x[VE];
                widen(w[k], x);
                if (v + k * kThreads < v1)
                    f(x, (v + k * kThreads) * VE);
            }
        }
        const int i = vectors() * VE + (int)threadIdx.x;
        if (tail && i < V) {
            float x[VE];
#pragma unroll
            for (int e = 0; e < VE; ++e)
                x[e] = -kInf;
            x[0] = at(i);
            f(x, i);
        }
    }
    template <typename F>
    __device__ __forceinline__ void each(F&& f) const
    {
        each(0, vectors(), true, f);
    }
};

// The order of a row's weights.
struct Scale {
    double ref, per;  // bins: (ref - x) per + kAbove
    double one, unit;  // 2^ebits, 2^-ebits
    double top;       // steps(maximum): the place of weight 1
    int shift;        // of the count

    __device__ __forceinline__ double steps(float x) const
    {
        return __builtin_fma(ref - (double)x, per, (double)kAbove);
    }
    static __device__ __forceinline__ bool inside(double y)
    {
        return fabs(y - kBins / 2) < kBins / 2;  // (0 to 1e-13 is outside)
    }
    // the bin of a value, -1 for none
    __device__ __forceinline__ int bin(float x) const
    {
        const double y = steps(x);
        return inside(y) ? (int)y : -1;
    }
    // what a value adds to its bin
    __device__ __forceinline__ uint64_t share(double y) const
    {
        const double f = __builtin_amdgcn_fract(y);
        const double h = 1.0 / kPerUnit;
        double q = -h * h * h * h / 24.0 * one;
        q = __builtin_fma(q, f, h * h * h / 6.0 * one);
        q = __builtin_fma(q, f, -h * h / 2.0 * one);
        q = __builtin_fma(q, f, h * one);
        // the integer next to q f stands in the low bits of 2^52 + q f
        q = __builtin_fma(q, f, 4503599627370496.0);
        return (uint64_t)(uint32_t)__builtin_bit_cast(uint64_t, q) | (1ull << shift);
    }
    __device__ __forceinline__ uint32_t count(uint64_t sum) const { return (uint32_t)(sum >> shift); }
    // a bin's weight over that of its upper end
    __device__ __forceinline__ double part(uint64_t sum) const
    {
        return (double)count(sum) - (double)(sum & ((1ull << shift) - 1)) * unit;
    }
    __device__ __forceinline__ double weight_at(double y) const
    {
        return exp((top - y) * (1.0 / kPerUnit));
    }
    __device__ __forceinline__ double weight(uint32_t key) const
    {
        return weight_at(steps(value_of(key)));
    }
};

template <int CTRL, int ROWS>
__device__ __forceinline__ uint32_t dpp(uint32_t v)
{
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, ROWS, 0xF, false);
}
template <int CTRL, int ROWS>
__device__ __forceinline__ double dpp(double v)
{
    const uint64_t u = __builtin_bit_cast(uint64_t, v);
    return __builtin_bit_cast(double, ((uint64_t)dpp<CTRL, ROWS>((uint32_t)(u >> 32)) << 32) |
                                          dpp<CTRL, ROWS>((uint32_t)u));
}
// Inclusive prefix sums over a wave.
template <typename T>
__device__ __forceinline__ T wave_scan(T v)
{
    v += dpp<0x111, 0xF>(v);  // row_shr 1, 2, 4, 8
    v += dpp<0x112, 0xF>(v);
    v += dpp<0x114, 0xF>(v);
    v += dpp<0x118, 0xF>(v);
    v += dpp<0x142, 0xA>(v);  // row_bcast 15, 31
    v += dpp<0x143, 0xC>(v);
    return v;
}
__device__ __forceinline__ float wave_max(float v)
{
#pragma unroll
    for (int d = 1; d < 64; d <<= 1)
        v = fmaxf(v, __shfl_xor(v, d, 64));
    return v;
}

// Exclusive prefix sums of a count and a weight over the threads; the totals
// go to every thread.
__device__ __forceinline__ void scan_threads(Shared& s, uint32_t& count, double& weight,
                                             uint32_t& all, double& total)
{
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const uint32_t c = wave_scan(count);
    const double w = wave_scan(weight);
    if (lane == 63) {
        s.wave_count[wave] = c;
        s.wave_weight[wave] = w;
    }
    // (the sum before a lane is its neighbour's, not a difference: that would
    // round)
    const uint32_t before_c = __shfl_up(c, 1, 64);
    const double before_w = __shfl_up(w, 1, 64);
    __syncthreads();
    uint32_t base_c = 0;
    double base_w = 0.0;
    all = 0;
    total = 0.0;
#pragma unroll
    for (int v = 0; v < kWaves; ++v) {
        if (v == wave) {
            base_c = all;
            base_w = total;
        }
        all += s.wave_count[v];
        total += s.wave_weight[v];
    }
    __syncthreads();
    count = base_c + (lane ? before_c : 0);
    weight = base_w + (lane ? before_w : 0.0);
}

// First i of [0, n) with past(i), else n - 1; past is false, then true.
template <typename F>
__device__ __forceinline__ int first_of(int n, F&& past)
{
    int lo = 0, hi = n - 1;
    while (lo < hi) {
        const int mid = (lo + hi) / 2;
        if (past(mid))
            hi = mid;
        else
            lo = mid + 1;
    }
    return lo;
}

template <bool BF16>
struct Sampler {
    Shared& s;
    const Row<BF16> row;
    Scale scale;
    double total;  // weight of all bins
    uint32_t all;  // their values
    int lo[2], hi[2];  // cand holds the bins lo[i] .. hi[i]

    // ref and the list's threshold from a sample: 16 values of every thread,
    // from four places of the row.  The threshold is the least of the waves'
    // maxima, each of 1024 values: about 1 in 370 values lies above.
    __device__ __forceinline__ void sample(float& ref, float& threshold)
    {
        constexpr int S = 16 / Row<BF16>::VE;
        const int nv = row.vectors();
        const int chunk = kThreads / 4;
        const int quarter = max(nv / 4, 1);
        float m = -kInf;
        bool any = false;
#pragma unroll
        for (int k = 0; k < S; ++k) {
            const int v = (int)(threadIdx.x / chunk) * quarter + k * chunk + (int)(threadIdx.x % chunk);
            if (k * chunk + (int)(threadIdx.x % chunk) < quarter && v < nv) {
                float x[Row<BF16>::VE];
                Row<BF16>::widen(row.load(v), x);
#pragma unroll
                for (int e = 0; e < Row<BF16>::VE; ++e)
                    m = fmaxf(m, x[e]);
                any = true;
            }
        }
        m = wave_max(m);
        any = __any(any);
        if ((threadIdx.x & 63) == 0)
            s.wave_max[threadIdx.x >> 6] = any ? m : kInf;
        __syncthreads();
        ref = -kInf;
        threshold = kInf;
#pragma unroll
        for (int w = 0; w < kWaves; ++w) {
            const float v = s.wave_max[w];
            threshold = fminf(threshold, v);
            ref = v < kInf ? fmaxf(ref, v) : ref;
        }
        ref = uniform(ref);
        threshold = uniform(threshold == kInf ? -kMax : fmaxf(threshold, -kMax));
        __syncthreads();
    }

    __device__ __forceinline__ void clear_bins()
    {
        for (int i = threadIdx.x; i < kBins; i += kThreads)
            s.bins[i] = 0;
        __syncthreads();
    }

    __device__ __forceinline__ void keep(float x, int i)
    {
        const uint32_t to = atomicAdd(&s.ncand, 1u);
        if (to < kCap)
            s.cand[to] = entry(x, i);
    }

    // Vectors v0 .. v1 - 1 to the bins (where `binned`), values from the
    // threshold on to cand; returns the workgroup's maximum.
    __device__ __forceinline__ float stream(int v0, int v1, bool tail, bool binned, float threshold)
    {
        constexpr int VE = Row<BF16>::VE;
        float m = -kInf;
        row.each(v0, v1, tail, [&](const float (&x)[VE], int i) {
            float most = x[0];
#pragma unroll
            for (int e = 1; e < VE; ++e)
                most = fmaxf(most, x[e]);
            m = fmaxf(m, most);
            if (binned) {
#pragma unroll
                for (int e = 0; e < VE; ++e) {
                    const double y = scale.steps(x[e]);
                    if (Scale::inside(y))
                        atomicAdd((unsigned long long*)&s.bins[(int)y],
                                  (unsigned long long)scale.share(y));
                }
            }
            if (most >= threshold) {
#pragma unroll
                for (int e = 0; e < VE; ++e)
                    if (x[e] >= threshold)
                        keep(x[e], i + e);
            }
        });
        m = wave_max(m);
        if ((threadIdx.x & 63) == 0)
            s.wave_max[threadIdx.x >> 6] = m;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < kWaves; ++w)
            m = fmaxf(m, s.wave_max[w]);
        return uniform(m);
    }

    // The bins to prefix sums.
    __device__ __forceinline__ void scan_bins()
    {
        double* before = (double*)s.bins;
        uint32_t c = 0, mine_c[kPer];
        double w = 0.0, mine_w[kPer];
        double e = scale.weight_at((double)(threadIdx.x * kPer));
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const uint64_t v = s.bins[threadIdx.x * kPer + i];
            mine_c[i] = scale.count(v);
            mine_w[i] = scale.part(v) * e;
            e *= 0.9844964370054085;  // e^(-1 / kPerUnit)
            c += mine_c[i];
            w += mine_w[i];
        }
        scan_threads(s, c, w, all, total);
        all = uniform(all);
        total = uniform(total);
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            s.counts[threadIdx.x * kPer + i] = c;
            before[threadIdx.x * kPer + i] = w;
            if (mine_c[i] && c + mine_c[i] == all)
                s.last = threadIdx.x * kPer + i;
            c += mine_c[i];
            w += mine_w[i];
        }
        if (threadIdx.x == 0)
            s.counts[kBins] = all;
        __syncthreads();
    }
    __device__ __forceinline__ double weight_before(int b) const
    {
        return b < kBins ? ((const double*)s.bins)[b] : total;
    }
    __device__ __forceinline__ uint32_t count_in(int b0, int b1) const
    {
        return s.counts[b1 + 1] - s.counts[b0];
    }

    // The first bin up to which past(count, weight) holds, else the last that
    // holds values: every wave by itself, 64 bins a look, and no barrier.
    template <typename F>
    __device__ __forceinline__ int bin_by(F&& past) const
    {
        constexpr int EACH = kBins / 64;
        static_assert(EACH <= 64);
        const int lane = threadIdx.x & 63;
        auto look = [&](int b) {  // first lane whose bin is past it, 64 for none
            const uint32_t c = s.counts[b + 1];
            const uint64_t yes = __ballot(c > 0 && past(c, weight_before(b + 1)));
            return yes ? __ffsll((long long)yes) - 1 : 64;
        };
        const int run = look(lane * EACH + EACH - 1);
        if (run == 64)
            return uniform(s.last);
        return uniform(run * EACH + look(run * EACH + min(lane, EACH - 1)));
    }

    // The least key that fits (fits is false, then true), next to where it is
    // expected: 64 keys around, one per lane, else by halves.
    template <typename F>
    static __device__ __forceinline__ uint32_t least_key(double guess, uint32_t top, F&& fits)
    {
        const float near = (float)fmin(fmax(guess, -(double)kMax), (double)kMax);
        const uint32_t first = min(key_of(near), top) - 32;
        const uint32_t mine = first + (threadIdx.x & 63);
        const uint64_t yes = __ballot(mine >= top || fits(mine));
        if ((yes & 1) == 0 && yes)
            return uniform(first + __ffsll((long long)yes) - 1);
        uint32_t a = key_of(-kMax), b = top;
        while (a < b) {
            const uint32_t mid = a + (b - a) / 2;
            if (fits(mid))
                b = mid;
            else
                a = mid + 1;
        }
        return uniform(a);
    }
    // The keys of the bins b0 .. b1.
    __device__ __forceinline__ void keys_of(int b0, int b1, uint32_t& from, uint32_t& to) const
    {
        // the least key of bin b or one before, infinity's if no value lies there
        auto first = [&](int b) {
            return least_key(scale.ref - (b + 1 - kAbove) / scale.per, key_of(kInf), [&](uint32_t key) {
                return scale.steps(value_of(key)) < (double)(b + 1);
            });
        };
        from = first(b1);
        to = b0 ? first(b0 - 1) - 1 : key_of(kMax);
    }

    // The row's values in the bins b0 .. b1 or c0 .. c1 to cand; they fit.
    __device__ __forceinline__ void gather(int b0, int b1, int c0, int c1)
    {
        uint32_t from, to, from2 = 1, to2 = 0;
        keys_of(b0, b1, from, to);
        if (c0 <= c1)
            keys_of(c0, c1, from2, to2);
        fetch(from, to, from2, to2);
        lo[0] = b0;
        hi[0] = b1;
        lo[1] = c0;
        hi[1] = c1;
    }
    // Values with a key in [from, to] or [from2, to2] (none where from2 > to2).
    __device__ __forceinline__ void fetch(uint32_t from, uint32_t to, uint32_t from2, uint32_t to2)
    {
        constexpr int VE = Row<BF16>::VE;
        const float x0 = value_of(from), x1 = value_of(to);
        const bool two = from2 <= to2;
        const float z0 = two ? value_of(from2) : 1.0f, z1 = two ? value_of(to2) : 0.0f;
        __syncthreads();
        if (threadIdx.x == 0)
            s.ncand = 0;
        __syncthreads();
        row.each([&](const float (&x)[VE], int i) {
            // at least 0 where a value lies between (comparisons would need
            // scalar instructions for each; differences have the right sign)
            float in[VE];
#pragma unroll
            for (int e = 0; e < VE; ++e)
                in[e] = fminf(x[e] - x0, x1 - x[e]);
            if (two)
#pragma unroll
                for (int e = 0; e < VE; ++e)
                    in[e] = fmaxf(in[e], fminf(x[e] - z0, z1 - x[e]));
            float any = in[0];
#pragma unroll
            for (int e = 1; e < VE; ++e)
                any = fmaxf(any, in[e]);
            if (any >= 0.0f) {
#pragma unroll
                for (int e = 0; e < VE; ++e)
                    if (in[e] >= 0.0f)
                        keep(x[e], i + e);
            }
        });
        __syncthreads();
    }
    __device__ __forceinline__ bool holds(int b0, int b1) const
    {
        return (b0 >= lo[0] && b1 <= hi[0]) || (b0 >= lo[1] && b1 <= hi[1]);
    }

    // The values with a key in [from, to], n <= kFew of them and all in cand,
    // sorted to the list, and the prefix sums of their weights on top of
    // `before`.
    __device__ __forceinline__ void collect(uint32_t from, uint32_t to, int n, double before)
    {
        uint32_t* rank = (uint32_t*)(s.list + 2 * kFew);
        __syncthreads();
        if (threadIdx.x == 0)
            s.n = 0;
        __syncthreads();
        const int have = min((int)s.ncand, kCap);
        for (int i = threadIdx.x; i < have; i += kThreads) {
            const uint64_t v = s.cand[i];
            const uint32_t key = entry_key(v);
            if (key >= from && key <= to) {
                const uint32_t at = atomicAdd(&s.n, 1u);
                if (at < kFew)
                    s.list[at] = v;
            }
        }
        if (threadIdx.x < kFew)
            rank[threadIdx.x] = 0;
        __syncthreads();
        // 4, 8 or 16 threads per value share the comparisons
        const int wide = n <= 64 ? 6 : (n <= 128 ? 7 : 8);
        const int i = threadIdx.x & ((1 << wide) - 1), part = threadIdx.x >> wide;
        const uint64_t mine = i < n ? s.list[i] : 0;
        if ((i & ~63) < n) {
            uint32_t r = 0;
#pragma unroll 4
            for (int j = part; j < n; j += kThreads >> wide)
                r += s.list[j] < mine;
            if (r)
                atomicAdd(&rank[i], r);
        }
        __syncthreads();
        if (part == 0 && i < n)
            s.list[rank[i]] = mine;
        __syncthreads();
        uint32_t c = 0, ca;
        const double w = part == 0 && i < n ? scale.weight(entry_key(s.list[i])) : 0.0;
        double sum = w, all_w;
        scan_threads(s, c, sum, ca, all_w);
        if (part == 0)
            s.sums[i] = before + sum + w;
        __syncthreads();
    }

    // The place in bin b where past(count, weight), inclusive, first holds: the
    // bin's keys are narrowed down until few values are left, or one key.
    template <typename F>
    __device__ __forceinline__ Place find(int b, F&& past)
    {
        uint32_t from, to;
        keys_of(b, b, from, to);
        const bool held = holds(b, b);
        uint32_t count = s.counts[b];
        double weight = weight_before(b);
        int n = (int)count_in(b, b);
        Place at;
        at.index = -1;
        at.rank = 0;
        while (n > kFew && from < to) {
            const int shift = max(0, 32 - __clz(to - from) - 12);
            __syncthreads();
            for (int i = threadIdx.x; i < kSub; i += kThreads)
                s.list[i] = 0;
            if (threadIdx.x == 0) {
                s.found = kSub;
                s.n = 0;
            }
            __syncthreads();
            auto add = [&](float x) {
                const uint32_t key = key_of(x);
                if (key >= from && key <= to)
                    atomicAdd((unsigned long long*)&s.list[(to - key) >> shift],
                              (unsigned long long)scale.share(scale.steps(x)));
            };
            if (held) {
                const int have = min((int)s.ncand, kCap);
                for (int i = threadIdx.x; i < have; i += kThreads)
                    add(value_of(entry_key(s.cand[i])));
            } else {
                constexpr int VE = Row<BF16>::VE;
                row.each([&](const float (&x)[VE], int) {
#pragma unroll
                    for (int e = 0; e < VE; ++e)
                        add(x[e]);
                });
            }
            __syncthreads();
            // this thread's four, and those before them
            constexpr int PER = kSub / kThreads;
            const double unit = scale.weight_at((double)b);
            uint32_t c = 0, ca, mine_c[PER];
            double w = 0.0, wa, mine_w[PER];
#pragma unroll
            for (int e = 0; e < PER; ++e) {
                const uint64_t v = s.list[threadIdx.x * PER + e];
                mine_c[e] = scale.count(v);
                mine_w[e] = scale.part(v) * unit;
                c += mine_c[e];
                w += mine_w[e];
            }
            scan_threads(s, c, w, ca, wa);
            // the first of them where the search ends, else the last that holds any
            // (one thread of a wave names its)
            uint32_t before_c[PER];
            double before_w[PER];
            int first = -1, last = -1;
#pragma unroll
            for (int e = 0; e < PER; ++e) {
                before_c[e] = c;
                before_w[e] = w;
                c += mine_c[e];
                w += mine_w[e];
                if (mine_c[e]) {
                    if (first < 0 && past(count + c, weight + w))
                        first = (int)threadIdx.x * PER + e;
                    last = (int)threadIdx.x * PER + e;
                }
            }
            const int lane = threadIdx.x & 63;
            const uint64_t firsts = __ballot(first >= 0), lasts = __ballot(last >= 0);
            if (firsts && lane == __ffsll((long long)firsts) - 1)
                atomicMin(&s.found, first);
            if (lasts && lane == 63 - __clzll((long long)lasts))
                atomicMax(&s.n, (uint32_t)last);
            __syncthreads();
            const int found = uniform(s.found < kSub ? s.found : (int)s.n);
#pragma unroll
            for (int e = 0; e < PER; ++e)
                if ((int)threadIdx.x * PER + e == found) {
                    s.wave_count[0] = before_c[e];
                    s.wave_count[1] = mine_c[e];
                    s.wave_weight[0] = before_w[e];
                }
            __syncthreads();
            count = uniform(count + s.wave_count[0]);
            n = uniform((int)s.wave_count[1]);
            weight = uniform(weight + s.wave_weight[0]);
            const uint32_t top = to - ((uint32_t)found << shift);
            const uint32_t span = (1u << shift) - 1;
            from = top - from > span ? top - span : from;
            to = top;
            __syncthreads();
        }
        if (n > kFew) {  // equal keys
            at.key = from;
            at.weight = scale.weight(from);
            at.rank = 1 + first_of(n, [&](int r) {
                return past(count + r + 1, weight + (double)(r + 1) * at.weight);
            });
            at.upto = weight + (double)at.rank * at.weight;
            return at;
        }
        if (!held) {
            fetch(from, to, 1, 0);
            hi[0] = hi[1] = -1;
        }
        collect(from, to, n, weight);
        const int i = first_of(n, [&](int e) { return past(count + e + 1, s.sums[e]); });
        at.key = entry_key(s.list[i]);
        at.index = (int)(uint32_t)s.list[i];
        at.upto = s.sums[i];
        at.weight = scale.weight(at.key);
        __syncthreads();
        return at;
    }

    // Index of the rank-th value with this key: by blocks of the row, then
    // value by value.
    __device__ __forceinline__ int index_of(uint32_t key, int rank)
    {
        uint32_t* blocks = (uint32_t*)s.list;
        const int size = (row.V + kSub - 1) / kSub;
        __syncthreads();
        for (int i = threadIdx.x; i < kSub; i += kThreads)
            blocks[i] = 0;
        __syncthreads();
        constexpr int VE = Row<BF16>::VE;
        const int n = row.V;
        row.each([&](const float (&x)[VE], int i) {
#pragma unroll
            for (int e = 0; e < VE; ++e)
                if (key_of(x[e]) == key && i + e < n)
                    atomicAdd(&blocks[(i + e) / size], 1u);
        });
        __syncthreads();
        constexpr int PER = kSub / kThreads;
        uint32_t c = 0, ca;
        double w = 0.0, wa;
#pragma unroll
        for (int e = 0; e < PER; ++e)
            c += blocks[threadIdx.x * PER + e];
        scan_threads(s, c, w, ca, wa);
#pragma unroll
        for (int e = 0; e < PER; ++e) {
            const uint32_t mine = blocks[threadIdx.x * PER + e];
            if (c < (uint32_t)rank && (uint32_t)rank <= c + mine) {
                s.index = (threadIdx.x * PER + e) * size;
                s.n = (uint32_t)rank - c;
            }
            c += mine;
        }
        __syncthreads();
        // every wave looks through the block, 64 values at a time
        int i = s.index, left = (int)s.n;
        const int lane = threadIdx.x & 63;
        for (; ; i += 64) {
            const bool hit = i + lane < row.V && key_of(row.at(min(i + lane, row.V - 1))) == key;
            const uint64_t hits = __ballot(hit);
            const int here = __popcll(hits);
            if (left <= here || i >= row.V) {
                const uint64_t mine = __ballot(hit && __popcll(hits & ((2ull << lane) - 1)) == left);
                i += __ffsll((long long)mine) - 1;
                break;
            }
            left -= here;
        }
        __syncthreads();
        return i;
    }
};

enum Mode : int { WHOLE = 0, PART, JOIN };

template <bool BF16, int MODE>
__global__ __launch_bounds__(kThreads) void sample_kernel(SampleArgs a)
{
    __shared__ Shared s;
    const int b = MODE == PART ? blockIdx.x / a.parts : blockIdx.x;
    const Row<BF16> row = {(const char*)a.logits + (size_t)b * a.ld * (BF16 ? 2 : 4), a.V};
    // options that are off: k of V or more, p of 1 or more, m of 0 or less
    const float T = a.temperature ? a.temperature[b] : 1.0f;
    const int opt_k = a.top_k ? a.top_k[b] : 0;
    const float opt_p = a.top_p ? a.top_p[b] : 1.0f;
    const float opt_m = a.min_p ? a.min_p[b] : 0.0f;
    const float opt_u = MODE == PART ? 0.0f : a.u[b];
    const double least = uniform(opt_m > 0.0f ? (double)opt_m : 0.0);
    const int k = least > 1.0 ? 1 : (opt_k > 0 && opt_k < a.V ? opt_k : a.V);
    const double p = uniform(opt_p < 1.0f ? fmax((double)opt_p, 0.0) : 1.0);
    const double u = uniform(opt_u > 0.0f ? (double)opt_u : 0.0);  // (a NaN is 0)
    const bool greedy = !(T > 0.0f);
    const double inv_t = uniform(greedy ? 1.0 : 1.0 / (double)T);

    Sampler<BF16> w = {s, row, {}, 0.0, 0, {0, 0}, {-1, -1}};
    Scale& sc = w.scale;
    sc.per = uniform(fmax(fmin((double)kPerUnit * inv_t, 1e300), 1e-300));
    sc.one = uniform((double)(1ull << a.ebits));
    sc.unit = 1.0 / sc.one;
    sc.shift = a.ebits - 6 + (32 - __clz(a.V));
    auto finish = [&](int token, double prob) {
        if (threadIdx.x == 0) {
            a.tokens[b] = token;
            if (a.probs)
                a.probs[b] = (float)prob;
        }
    };

    // ---- bins and list ----
    float ref, threshold, m;
    Part* const parts = (Part*)a.ws + (size_t)b * a.parts;
    if constexpr (MODE == JOIN) {
        ref = parts[0].ref;
        threshold = parts[0].threshold;
        // a lane per part: maxima, and where a part's list starts
        const int lane = threadIdx.x & 63;
        const bool mine = lane < a.parts;
        m = uniform(wave_max(mine ? parts[lane].max : -kInf));
        const uint32_t n = mine ? parts[lane].n : 0;
        const bool whole = !__any(n > kSamplePartList);
        const uint32_t end = wave_scan(n);
        const uint32_t all = __shfl(end, 63, 64);
        if (whole && all <= kCap)
            for (int q = threadIdx.x >> 6; q < a.parts; q += kWaves) {
                const uint32_t have = __shfl(n, q, 64), at = __shfl(end, q, 64) - have;
                for (uint32_t i = lane; i < have; i += 64)
                    s.cand[at + i] = parts[q].list[i];
            }
        if (threadIdx.x == 0)
            s.ncand = whole ? all : kCap + 1;
        sc.ref = uniform((double)ref);
        if (!greedy) {
            uint64_t sum[kPer] = {};
#pragma unroll 4
            for (int q = 0; q < a.parts; ++q)
#pragma unroll
                for (int i = 1; i < kPer; ++i)
                    sum[i] += parts[q].bins[threadIdx.x + i * kThreads];
            // (mostly there is nothing that far above ref)
            if (!(sc.steps(m) >= (double)kThreads))
#pragma unroll 4
                for (int q = 0; q < a.parts; ++q)
                    sum[0] += parts[q].bins[threadIdx.x];
#pragma unroll
            for (int i = 0; i < kPer; ++i)
                s.bins[threadIdx.x + i * kThreads] = sum[i];
        }
        __syncthreads();
    } else {
        w.sample(ref, threshold);
        sc.ref = uniform((double)ref);
        if (threadIdx.x == 0)
            s.ncand = 0;
        if constexpr (MODE == PART) {
            w.clear_bins();
            const int nv = row.vectors();
            const int q = (int)(blockIdx.x % a.parts);
            const int v0 = (int)((int64_t)nv * q / a.parts), v1 = (int)((int64_t)nv * (q + 1) / a.parts);
            m = w.stream(v0, v1, q == a.parts - 1, !greedy, threshold);
            Part& part = parts[q];
            if (!greedy) {
#pragma unroll
                for (int i = 0; i < kPer; ++i)
                    part.bins[threadIdx.x + i * kThreads] = s.bins[threadIdx.x + i * kThreads];
            }
            const uint32_t n = s.ncand;
            for (uint32_t i = threadIdx.x; i < n && i < kSamplePartList; i += kThreads)
                part.list[i] = s.cand[i];
            if (threadIdx.x == 0) {
                part.n = n;
                part.max = m;
                part.ref = ref;
                part.threshold = threshold;
            }
            return;
        }
    }
    // the stream's maximum; a row beyond the bins goes again, from its maximum
    // (the list is there)
    for (bool again = MODE == JOIN; ; again = true) {
        if (again) {
            if (greedy || !(m < kInf) || m == -kInf || Scale::inside(sc.steps(m)))
                break;
            sc.ref = uniform((double)m);
        }
        w.clear_bins();
        m = w.stream(0, row.vectors(), true, !greedy, again ? kInf : threshold);
    }
    const bool listed = s.ncand <= kCap;  // (the list is whole)
    if (m == -kInf) {  // nothing to choose from
        finish(-1, 0.0);
        return;
    }
    // the answer: a token, or the rank-th with a key
    uint32_t key = key_of(m);
    int rank = 1;
    double share = 1.0;
    if (greedy && listed) {
        // the largest logit: the first of the list
        if (threadIdx.x == 0)
            s.index = a.V;
        __syncthreads();
        for (int i = threadIdx.x; i < (int)s.ncand; i += kThreads)
            if (entry_key(s.cand[i]) == key_of(m))
                atomicMin(&s.index, (int)(uint32_t)s.cand[i]);
        __syncthreads();
        finish(s.index, 1.0);
        return;
    }
    if (!greedy && m == kInf) {
        // only infinite logits have weight, all the same
        constexpr int VE = Row<BF16>::VE;
        int n = 0;
        row.each([&](const float (&x)[VE], int) {
#pragma unroll
            for (int e = 0; e < VE; ++e)
                n += x[e] == kInf;
        });
        uint32_t c = n, all;
        double cw = 0.0, aw;
        __syncthreads();
        scan_threads(s, c, cw, all, aw);
        n = min((int)all, k);
        if (p < 1.0)
            n = 1 + first_of(n, [&](int i) { return (double)(i + 1) >= p * n; });
        rank = 1 + first_of(n, [&](int i) { return (double)(i + 1) > u * n; });
        share = 1.0 / n;
    }
    if (!greedy && m < kInf) {
    sc.top = uniform(sc.steps(m));
    w.scan_bins();
    // every value of the bins before the threshold's is in the list
    w.hi[0] = -1;
    if (listed) {
        const double y = sc.steps(threshold);
        w.hi[0] = (y < (double)kBins ? (int)y : kBins) - 1;
    }

    // ---- what is kept ----
    const bool by_k = (uint32_t)k < w.all, by_p = p < 1.0, by_m = least > 0.0 && least <= 1.0;
    // the least key with e^((x - m) / T) >= min_p
    uint32_t floor_key = 0;
    if (by_m)
        floor_key = w.least_key((double)m + log(least) / inv_t, key_of(m), [&](uint32_t key) {
            return exp(((double)value_of(key) - (double)m) * inv_t) >= least;
        });
    const double total = w.total;
    int cut = s.last;
    if (by_k) {
        cut = w.bin_by([&](uint32_t c, double) { return c >= (uint32_t)k; });
    } else {
        if (by_p)
            cut = w.bin_by([&](uint32_t, double x) { return x >= p * total; });
        if (by_m) {
            const int f = sc.bin(value_of(floor_key));
            cut = f < 0 ? cut : min(cut, f);
        }
    }
    const bool cuts = by_k || by_p || by_m;
    const int n = (int)w.count_in(0, cut);
    if (n <= kFew && (cuts || w.holds(0, cut))) {
        // everything that matters, sorted
        uint32_t from = 0, to = 0xFFFFFFFFu;
        w.keys_of(0, cut, from, to);
        if (!w.holds(0, cut))
            w.fetch(from, to, 1, 0);
        w.collect(from, to, n, 0.0);
        int keep = by_k ? min(n, k) : n;
        const double of = by_k || cut == s.last ? s.sums[keep - 1] : total;
        if (by_p)
            keep = 1 + first_of(keep, [&](int i) { return s.sums[i] >= p * of; });
        if (by_m)
            keep = max(1, first_of(keep + 1, [&](int i) { return i >= keep || entry_key(s.list[i]) < floor_key; }));
        const double z = s.sums[keep - 1];
        const int i = first_of(keep, [&](int j) { return s.sums[j] > u * z; });
        finish((int)(uint32_t)s.list[i], sc.weight(entry_key(s.list[i])) / z);
        return;
    }

    // one search after the other: where top-k ends, where top-p ends, the token
    double z = total;
    Place at;
    at.key = 0;
    for (int stage = by_k ? 0 : (by_p ? 1 : 2); stage < 3; ++stage) {
        if (stage == 1 && !by_p)
            continue;
        if (stage == 2 && by_m && floor_key > at.key) {
            // the weight down to the floor's key: its bin's values above it
            const int f0 = sc.bin(value_of(floor_key));
            const int f = f0 < 0 ? s.last : f0;
            constexpr int VE = Row<BF16>::VE;
            double sum = 0.0;
            const float least_x = value_of(floor_key);
            row.each([&](const float (&x)[VE], int) {
#pragma unroll
                for (int e = 0; e < VE; ++e)
                    if (x[e] >= least_x && sc.bin(x[e]) == f)
                        sum += sc.weight(key_of(x[e]));
            });
            uint32_t c = 0, ca;
            double wa;
            scan_threads(s, c, sum, ca, wa);
            z = uniform(fmin(z, w.weight_before(f) + wa));
        }
        const double target = uniform((stage == 1 ? p : u) * z);
        auto past = [&](uint32_t c, double x) {
            return stage == 0 ? c >= (uint32_t)k : (stage == 1 ? x >= target : x > target);
        };
        const int f = w.bin_by(past);
        if (!w.holds(f, f)) {
            // one pass: all that matters, or this bin and those that the token
            // can lie in
            int b0 = f, b1 = f, c0 = 1, c1 = 0;
            if (cuts && n <= kCap) {
                b0 = 0;
                b1 = cut;
            } else if (stage == 1) {
                const double a0 = u * w.weight_before(f), a1 = u * w.weight_before(f + 1);
                c0 = w.bin_by([&](uint32_t, double x) { return x > a0; });
                c1 = w.bin_by([&](uint32_t, double x) { return x > a1; });
                if ((uint64_t)w.count_in(f, f) + w.count_in(c0, c1) > kCap) {
                    c0 = 1;
                    c1 = 0;
                }
            }
            if (w.count_in(b0, b1) <= kCap)
                w.gather(b0, b1, c0, c1);
        }
        at = w.find(f, past);
        if (stage < 2)
            z = uniform(fmin(z, at.upto));
    }
    share = at.weight / z;
    if (at.rank == 0) {
        finish(at.index, share);
        return;
    }
    key = at.key;
    rank = at.rank;
    }
    finish(w.index_of(key, rank), share);
}

template <bool BF16>
hipError_t launch(const SampleArgs& a, hipStream_t stream)
{
    if (a.parts == 1) {
        sample_kernel<BF16, WHOLE><<<a.B, kThreads, 0, stream>>>(a);
        return hipGetLastError();
    }
    sample_kernel<BF16, PART><<<a.B * a.parts, kThreads, 0, stream>>>(a);
    const hipError_t rc = hipGetLastError();
    if (rc != hipSuccess)
        return rc;
    sample_kernel<BF16, JOIN><<<a.B, kThreads, 0, stream>>>(a);
    return hipGetLastError();
}

}  // namespace

int sample_parts(int64_t B, int64_t V)
{
    // Parts of 8192 values and more, as many as fill the compute units.  Past 8 of
    // them, of 32768 and more: each part costs the second launch 0.4 us (a row
    // of 151936 in 8, 11 and 16 parts: 9.8 + 12.7 us, 8.5 + 14.6, 7.5 + 15.9).
    const int64_t by_values = V / 8192, by_rows = B ? 256 / B : 1, by_join = V / 32768;
    const int64_t most = by_join < 8 ? 8 : (by_join > 16 ? 16 : by_join);
    int64_t n = by_values < by_rows ? by_values : by_rows;
    n = n > most ? most : n;
    return (int)(n < 1 ? 1 : n);
}
int64_t sample_part_bytes() { return (int64_t)sizeof(Part); }

hipError_t launch_sample(const SampleArgs& a, hipStream_t stream)
{
    return a.bf16 ? launch<true>(a, stream) : launch<false>(a, stream);
}

}  // namespace qll
