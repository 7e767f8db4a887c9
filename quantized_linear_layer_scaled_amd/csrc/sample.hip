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
// A workgroup takes a row.  One pass finds the maximum; a second one puts
// every value into one of kBins bins of d, 1 / kPerUnit wide, by one LDS
// addition that carries a count and a weight; prefix sums over the bins then
// say in which bin an answer lies, and a third pass gathers the few values of
// that bin, or of all bins up to it where these are few too, which is the usual
// case with top-k or a peaked distribution; they are sorted in LDS.
//
// A token is right or wrong, so weights are formed to well below a token's
// share: within a bin w = e^-(b / kPerUnit) (1 - g), g = 1 - e^-(f / kPerUnit)
// with f the fraction of the bin (64-bit arithmetic, four terms: 2^-42), and
// the additions are integers: the count above, g in `ebits` fractional bits
// below (35 for vocabularies below 2^18), which no order of additions changes.
// Weights below e^-32 of the largest are left out: 2^20 of them are less than
// 1.4e-8 of the total, below the last bit of u next to 1 (6e-8).
//
// A bin that holds more values than the list (equal logits, a wide
// temperature) is narrowed down by further passes over its keys, 4096 ways
// each; equal keys are counted by blocks of the row.
#include "ffn_epilogue.h"
#include "sample_internal.h"

namespace qll {

namespace {

constexpr int kThreads = 1024;
constexpr int kWaves = kThreads / 64;
constexpr int kBins = 4096;
constexpr int kPerUnit = 128;  // bins per unit of d
constexpr int kCap = 4096;     // values in the list
constexpr float kInf = __builtin_inff();

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

struct Shared {
    uint64_t bins[kBins];      // then: weight before each bin, as doubles
    uint32_t counts[kBins + 1];  // values before each bin
    uint64_t list[kCap];       // ~key, index
    double sums[kCap];         // weight up to and with each list entry
    double wave_weight[kWaves];
    uint32_t wave_count[kWaves];
    float wave_max[kWaves];
    uint32_t n;
    int index;
};

// A place in the order.
struct Place {
    uint32_t key;
    int index;      // of the token, or -1 where nobody asked for it
    double weight;  // of one value
    double upto;    // weight up to and with this place
};

template <bool BF16>
struct Row {
    const void* p;
    int V;
    // f(value, index) for all values
    template <typename F>
    __device__ __forceinline__ void each(F&& f) const
    {
        constexpr int VE = BF16 ? 8 : 4;
        constexpr int U = 4;
        const int nv = V / VE;
        for (int v0 = threadIdx.x; v0 < nv; v0 += U * kThreads) {
            u32x4_any w[U];
#pragma unroll
            for (int k = 0; k < U; ++k)
                if (v0 + k * kThreads < nv)
                    w[k] = *(const u32x4_any*)((const char*)p + (size_t)(v0 + k * kThreads) * 16);
#pragma unroll
            for (int k = 0; k < U; ++k) {
                const int at = (v0 + k * kThreads) * VE;
                if (v0 + k * kThreads < nv) {
#pragma unroll
                    for (int e = 0; e < VE; ++e) {
                        float x;
                        if constexpr (BF16)
                            x = __uint_as_float(e & 1 ? w[k][e / 2] & 0xFFFF0000u : w[k][e / 2] << 16);
                        else
                            x = __uint_as_float(w[k][e]);
                        f(x, at + e);
                    }
                }
            }
        }
        const int i = nv * VE + (int)threadIdx.x;
        if (i < V)
            f(at(i), i);
    }
    __device__ __forceinline__ float at(int i) const
    {
        return BF16 ? bf16_value(((const uint16_t*)p)[i]) : ((const float*)p)[i];
    }
};

// The order of a row's weights.
struct Scale {
    double max, per;  // d * kPerUnit = (max - x) * per
    double inv_t;
    double one;  // 2^ebits
    int shift;   // of the count

    __device__ __forceinline__ double steps(float x) const { return (max - (double)x) * per; }
    // the bin of a value, -1 for none; y: steps(x)
    __device__ __forceinline__ int bin(double y) const { return y < (double)kBins ? (int)y : -1; }
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
    __device__ __forceinline__ double weight(uint64_t sum, int bin) const
    {
        const double g = (double)(sum & ((1ull << shift) - 1)) / one;
        return ((double)count(sum) - g) * exp(-(double)bin / kPerUnit);
    }
    __device__ __forceinline__ double weight(uint32_t key) const
    {
        return exp(-(max - (double)value_of(key)) * inv_t);
    }
};

// Exclusive prefix sums of a count and a weight over the threads; the totals
// go to every thread.
__device__ __forceinline__ void scan_threads(Shared& s, uint32_t& count, double& weight,
                                             uint32_t& all, double& total)
{
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    uint32_t c = count;
    double w = weight;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const uint32_t oc = __shfl_up(c, d, 64);
        const double ow = __shfl_up(w, d, 64);
        if (lane >= d) {
            c += oc;
            w += ow;
        }
    }
    if (lane == 63) {
        s.wave_count[wave] = c;
        s.wave_weight[wave] = w;
    }
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

// Sorts the n values of the list: a bitonic network.
__device__ void sort_list(Shared& s, int n)
{
    int size = 1;
    while (size < n)
        size <<= 1;
    for (int i = n + (int)threadIdx.x; i < size; i += kThreads)
        s.list[i] = ~0ull;
    __syncthreads();
    for (int k = 2; k <= size; k <<= 1)
        for (int j = k >> 1; j > 0; j >>= 1) {
            for (int t = threadIdx.x; t < size / 2; t += kThreads) {
                const int i = 2 * t - (t & (j - 1));
                const uint64_t a = s.list[i], b = s.list[i + j];
                if ((a > b) == ((i & k) == 0)) {
                    s.list[i] = b;
                    s.list[i + j] = a;
                }
            }
            __syncthreads();
        }
}

template <bool BF16>
struct Sampler {
    Shared& s;
    const Row<BF16> row;
    Scale scale;

    __device__ __forceinline__ uint32_t list_key(int i) const { return ~(uint32_t)(s.list[i] >> 32); }

    // Values with a key in [lo, hi] and a bin in [b0, b1] to the list.
    __device__ int gather(int b0, int b1, uint32_t lo, uint32_t hi)
    {
        __syncthreads();
        if (threadIdx.x == 0)
            s.n = 0;
        __syncthreads();
        row.each([&](float x, int i) {
            const uint32_t key = key_of(x);
            if (key >= lo && key <= hi) {
                const int b = scale.bin(scale.steps(x));
                if (b >= b0 && b <= b1) {
                    const uint32_t at = atomicAdd(&s.n, 1u);
                    if (at < kCap)
                        s.list[at] = ((uint64_t)~key << 32) | (uint32_t)i;
                }
            }
        });
        __syncthreads();
        const int n = min((int)s.n, kCap);
        sort_list(s, n);
        return n;
    }

    // The prefix sums of the list's weights on top of `before`.
    __device__ void list_sums(int n, double before)
    {
        double w[kCap / kThreads], total = 0.0, all;
        uint32_t c = 0, ca;
        const int i0 = threadIdx.x * (kCap / kThreads);
#pragma unroll
        for (int e = 0; e < kCap / kThreads; ++e) {
            w[e] = i0 + e < n ? scale.weight(list_key(i0 + e)) : 0.0;
            total += w[e];
        }
        scan_threads(s, c, total, ca, all);
        total += before;
#pragma unroll
        for (int e = 0; e < kCap / kThreads; ++e) {
            total += w[e];
            s.sums[i0 + e] = total;
        }
        __syncthreads();
    }

    // The place in the values of bin b (count and weight before it given) where
    // `past(count, weight)`, inclusive, first holds.
    template <typename F>
    __device__ Place find(int b, int n, uint32_t count, double weight, bool want_index, F&& past)
    {
        uint32_t lo = 0, hi = 0xFFFFFFFFu;
        // the keys around the bin (the bin itself is checked exactly)
        {
            const double x1 = scale.max - b / scale.per, x0 = scale.max - (b + 1) / scale.per;
            const double slack = 1e-6 * (fabs(x0) + fabs(x1)) + 1e-37;
            hi = key_of((float)(x1 + slack));
            lo = key_of((float)(x0 - slack));
        }
        Place at;
        at.index = -1;
        // (the sums of this search go where the list is not: bins hold prefix
        // sums that later searches use, so they are kept)
        while (n > kCap && lo < hi) {
            // narrow the keys down 4096 ways
            uint64_t* sub = s.list;
            const int shift = max(0, 32 - __clz(hi - lo) - 12);
            __syncthreads();
            for (int i = threadIdx.x; i < kBins; i += kThreads)
                sub[i] = 0;
            __syncthreads();
            row.each([&](float x, int) {
                const uint32_t key = key_of(x);
                if (key >= lo && key <= hi) {
                    const double y = scale.steps(x);
                    if (scale.bin(y) == b)
                        atomicAdd((unsigned long long*)&sub[(hi - key) >> shift],
                                  (unsigned long long)scale.share(y));
                }
            });
            __syncthreads();
            // this thread's four, and those before them
            constexpr int PER = kBins / kThreads;
            uint32_t c = 0, ca, mine_c[PER];
            double w = 0.0, wa, mine_w[PER];
#pragma unroll
            for (int e = 0; e < PER; ++e) {
                const uint64_t v = sub[threadIdx.x * PER + e];
                mine_c[e] = scale.count(v);
                mine_w[e] = scale.weight(v, b);
                c += mine_c[e];
                w += mine_w[e];
            }
            scan_threads(s, c, w, ca, wa);
            // the first of them where the search ends, else the last that holds any
            if (threadIdx.x == 0) {
                s.index = kBins;
                s.n = 0;
            }
            __syncthreads();
            uint32_t before_c[PER];
            double before_w[PER];
#pragma unroll
            for (int e = 0; e < PER; ++e) {
                before_c[e] = c;
                before_w[e] = w;
                c += mine_c[e];
                w += mine_w[e];
                if (mine_c[e]) {
                    if (past(count + c, weight + w))
                        atomicMin(&s.index, (int)threadIdx.x * PER + e);
                    atomicMax(&s.n, (uint32_t)(threadIdx.x * PER + e));
                }
            }
            __syncthreads();
            const int found = s.index < kBins ? s.index : (int)s.n;
            __syncthreads();
#pragma unroll
            for (int e = 0; e < PER; ++e)
                if ((int)threadIdx.x * PER + e == found) {
                    s.wave_count[0] = before_c[e];
                    s.wave_count[1] = mine_c[e];
                    s.wave_weight[0] = before_w[e];
                }
            __syncthreads();
            count += s.wave_count[0];
            n = (int)s.wave_count[1];
            weight += s.wave_weight[0];
            const uint32_t top = hi - ((uint32_t)found << shift);
            const uint32_t span = (1u << shift) - 1;
            lo = top - lo > span ? top - span : lo;
            hi = top;
            __syncthreads();
        }
        if (n > kCap) {  // equal keys
            at.key = lo;
            at.weight = scale.weight(lo);
            const int rank = 1 + first_of(n, [&](int r) {
                return past(count + r + 1, weight + (double)(r + 1) * at.weight);
            });
            at.upto = weight + (double)rank * at.weight;
            if (want_index)
                at.index = index_of(lo, rank);
            return at;
        }
        n = gather(b, b, lo, hi);
        list_sums(n, weight);
        const int i = first_of(n, [&](int e) { return past(count + e + 1, s.sums[e]); });
        at.key = list_key(i);
        at.index = (int)(uint32_t)s.list[i];
        at.upto = s.sums[i];
        at.weight = scale.weight(at.key);
        __syncthreads();
        return at;
    }

    // Index of the rank-th value with this key: by blocks of the row, then
    // value by value.
    __device__ int index_of(uint32_t key, int rank)
    {
        uint32_t* blocks = (uint32_t*)s.list;
        const int size = (row.V + kBins - 1) / kBins;
        __syncthreads();
        for (int i = threadIdx.x; i < kBins; i += kThreads)
            blocks[i] = 0;
        __syncthreads();
        row.each([&](float x, int i) {
            if (key_of(x) == key)
                atomicAdd(&blocks[i / size], 1u);
        });
        __syncthreads();
        constexpr int PER = kBins / kThreads;
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
                int left = rank - (int)c;
                for (int i = (threadIdx.x * PER + e) * size; i < row.V; ++i)
                    if (key_of(row.at(i)) == key && --left == 0) {
                        s.index = i;
                        break;
                    }
            }
            c += mine;
        }
        __syncthreads();
        const int i = s.index;
        __syncthreads();
        return i;
    }
};

template <bool BF16>
__global__ __launch_bounds__(kThreads) void sample_kernel(SampleArgs a)
{
    __shared__ Shared s;
    const int b = blockIdx.x;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const Row<BF16> row = {(const char*)a.logits + (size_t)b * a.ld * (BF16 ? 2 : 4), a.V};
    const float T = a.temperature ? a.temperature[b] : 1.0f;
    auto finish = [&](int token, double prob) {
        if (threadIdx.x == 0) {
            a.tokens[b] = token;
            if (a.probs)
                a.probs[b] = (float)prob;
        }
    };

    float m = -kInf;
    row.each([&](float x, int) { m = fmaxf(m, x); });
#pragma unroll
    for (int d = 1; d < 64; d <<= 1)
        m = fmaxf(m, __shfl_xor(m, d, 64));
    if (lane == 0)
        s.wave_max[wave] = m;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kWaves; ++w)
        m = fmaxf(m, s.wave_max[w]);
    if (m == -kInf) {  // nothing to choose from
        finish(-1, 0.0);
        return;
    }
    float u = a.u[b];
    u = u > 0.0f ? u : 0.0f;  // (a NaN is 0)
    Sampler<BF16> sampler = {s, row, {}};
    Scale& sc = sampler.scale;
    if (!(T > 0.0f)) {  // the largest logit
        finish(sampler.index_of(key_of(m), 1), 1.0);
        return;
    }
    // options that are off: k of V or more, p of 1 or more, m of 0 or less
    int k = a.top_k && a.top_k[b] > 0 && a.top_k[b] < a.V ? a.top_k[b] : a.V;
    const double p = a.top_p && a.top_p[b] < 1.0f ? fmax((double)a.top_p[b], 0.0) : 1.0;
    const double floor_w = a.min_p && a.min_p[b] > 0.0f ? (double)a.min_p[b] : 0.0;
    if (floor_w > 1.0)
        k = 1;
    sc.max = (double)m;
    sc.inv_t = 1.0 / (double)T;
    sc.per = fmax(fmin((double)kPerUnit * sc.inv_t, 1e300), 1e-300);
    sc.one = (double)(1ull << a.ebits);
    sc.shift = a.ebits - 7 + (32 - __clz(a.V));
    if (m == kInf) {
        // only infinite logits have weight, all the same
        int n = 0;
        row.each([&](float x, int) { n += x == kInf; });
#pragma unroll
        for (int d = 1; d < 64; d <<= 1)
            n += __shfl_xor(n, d, 64);
        __syncthreads();
        if (lane == 0)
            s.wave_count[wave] = n;
        __syncthreads();
        n = 0;
#pragma unroll
        for (int w = 0; w < kWaves; ++w)
            n += (int)s.wave_count[w];
        n = min(n, k);
        if (p < 1.0)
            n = 1 + first_of(n, [&](int i) { return (double)(i + 1) >= p * n; });
        const int r = first_of(n, [&](int i) { return (double)(i + 1) > (double)u * n; });
        finish(sampler.index_of(key_of(m), r + 1), 1.0 / n);
        return;
    }

    // ---- bins ----
    for (int i = threadIdx.x; i < kBins; i += kThreads)
        s.bins[i] = 0;
    __syncthreads();
    row.each([&](float x, int) {
        const double y = sc.steps(x);
        if (y < (double)kBins)
            atomicAdd((unsigned long long*)&s.bins[(int)y], (unsigned long long)sc.share(y));
    });
    __syncthreads();
    double* before = (double*)s.bins;
    uint32_t all;
    double total;
    {
        constexpr int PER = kBins / kThreads;
        uint32_t c = 0, mine_c[PER];
        double w = 0.0, mine_w[PER];
#pragma unroll
        for (int e = 0; e < PER; ++e) {
            const uint64_t v = s.bins[threadIdx.x * PER + e];
            mine_c[e] = sc.count(v);
            mine_w[e] = sc.weight(v, threadIdx.x * PER + e);
            c += mine_c[e];
            w += mine_w[e];
        }
        scan_threads(s, c, w, all, total);
#pragma unroll
        for (int e = 0; e < PER; ++e) {
            s.counts[threadIdx.x * PER + e] = c;
            before[threadIdx.x * PER + e] = w;
            c += mine_c[e];
            w += mine_w[e];
        }
        if (threadIdx.x == 0)
            s.counts[kBins] = all;
        __syncthreads();
    }
    auto count_upto = [&](int i) { return s.counts[i + 1]; };
    auto weight_upto = [&](int i) { return i + 1 < kBins ? before[i + 1] : total; };
    // the last bin that holds any
    const int last = first_of(kBins, [&](int i) { return count_upto(i) == all; });
    auto bin_by = [&](auto&& past) {
        return min(last, first_of(kBins, [&](int i) { return past(count_upto(i), weight_upto(i)); }));
    };

    const bool by_k = (uint32_t)k < all, by_p = p < 1.0, by_w = floor_w > 0.0 && floor_w <= 1.0;
    // the lowest key with w >= min_p (at most the maximum's)
    uint32_t floor_key = 0;
    if (by_w) {
        uint32_t lo = key_of(-kInf), hi = key_of(m);
        while (lo < hi) {
            const uint32_t mid = lo + (hi - lo) / 2;
            if (sc.weight(mid) >= floor_w)
                hi = mid;
            else
                lo = mid + 1;
        }
        floor_key = lo;
    }
    const int bin_k = by_k ? bin_by([&](uint32_t c, double) { return c >= (uint32_t)k; }) : last;
    int cut = bin_k;
    if (!by_k) {
        if (by_p)
            cut = min(cut, bin_by([&](uint32_t, double w) { return w >= p * total; }));
        if (by_w) {
            const int f = sc.bin(sc.steps(value_of(floor_key)));
            cut = min(cut, f < 0 ? last : f);
        }
    }
    if (count_upto(cut) <= kCap && (by_k || by_p || by_w || all <= kCap)) {
        // everything that matters, sorted
        const int n = sampler.gather(0, cut, 0, 0xFFFFFFFFu);
        sampler.list_sums(n, 0.0);
        const double* upto = s.sums;
        int keep = by_k ? min(n, k) : n;
        const double of = by_k ? upto[keep - 1] : total;
        if (by_p)
            keep = 1 + first_of(keep, [&](int i) { return upto[i] >= p * of; });
        if (by_w)
            keep = max(1, first_of(keep + 1, [&](int i) { return i >= keep || sampler.list_key(i) < floor_key; }));
        const double z = keep == n && !by_k && !by_p && !by_w ? total : upto[keep - 1];
        const int i = first_of(keep, [&](int j) { return upto[j] > (double)u * z; });
        finish((int)(uint32_t)s.list[i], sc.weight(sampler.list_key(i)) / z);
        return;
    }

    // one search after the other
    double z = total;
    uint32_t end_key = 0;
    Place end;
    if (by_k) {
        const int f = bin_k;
        end = sampler.find(f, count_upto(f) - s.counts[f], s.counts[f], before[f], false,
                           [&](uint32_t c, double) { return c >= (uint32_t)k; });
        z = end.upto;
        end_key = end.key;
    }
    if (by_p) {
        const double target = p * z;
        auto past = [&](uint32_t, double w) { return w >= target; };
        const int f = bin_by(past);
        end = sampler.find(f, count_upto(f) - s.counts[f], s.counts[f], before[f], false, past);
        z = fmin(z, end.upto);
        end_key = end.key;
    }
    if (by_w && floor_key > end_key) {
        // the weight down to the floor's key: its bin's values above it
        int f = sc.bin(sc.steps(value_of(floor_key)));
        if (f < 0)
            f = last;
        double w = 0.0;
        row.each([&](float x, int) {
            const double y = sc.steps(x);
            if (key_of(x) >= floor_key && sc.bin(y) == f)
                w += exp(-(sc.max - (double)x) * sc.inv_t);
        });
        uint32_t c = 0, ca;
        double wa;
        scan_threads(s, c, w, ca, wa);
        z = fmin(z, before[f] + wa);
    }
    const double target = (double)u * z;
    auto past = [&](uint32_t, double w) { return w > target; };
    const int f = bin_by(past);
    const Place at = sampler.find(f, count_upto(f) - s.counts[f], s.counts[f], before[f], true, past);
    finish(at.index, at.weight / z);
}

}  // namespace

hipError_t launch_sample(const SampleArgs& a, hipStream_t stream)
{
    if (a.bf16)
        sample_kernel<true><<<a.B, kThreads, 0, stream>>>(a);
    else
        sample_kernel<false><<<a.B, kThreads, 0, stream>>>(a);
    return hipGetLastError();
}

}  // namespace qll
