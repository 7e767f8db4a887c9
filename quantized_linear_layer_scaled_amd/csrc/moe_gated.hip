// The experts' gated products for gfx950: every row of A, or the token that
// rows[] names, times its expert's gate and up weights.
//
//   out[i] = act(sum_k A[t][k] Bg[e][n][k] sa[t] sg[e][n]) *
//            (sum_k A[t][k] Bu[e][n][k] sa[t] su[e][n]),  t = rows[i], e owns i
//
// A workgroup finds its expert from the offsets (find_tile, lane-parallel
// over 64 experts) and computes a row tile of it with the building blocks of
// the dense feed-forward products; the tokens are gathered by the copies
// themselves, so no sorted copy of A is made.  The number of row tiles is
// known on the device alone: the grid holds the most there can be (R / rows of
// a tile + min(E, R)), and workgroups past the last tile leave at once.
//
// The sums are the matrix core's e4m3 steps into fp32, as in every FP8 product
// here.  A step adds its 128 products more coarsely than fp32 additions would:
// sums are off by up to 2^-12 of their terms' magnitudes.  Kept, since a bf16
// output's rounding is larger: for 2048 tokens, N = 1536, K = 2048 (norms) fp32
// outputs are 5.9e-5 off, against 6e-7 for exact products added in fp32, and bf16
// outputs 1.659e-3, against 1.658e-3 for the exact result rounded to bf16.
#include "ffn_alt.h"
#include "moe_internal.h"

namespace qll {

namespace {

// Inclusive prefix maxima and sums of a wave's values (at least 0).
template <int CTRL, int ROWS>
__device__ __forceinline__ int from_before(int v)
{
    return __builtin_amdgcn_update_dpp(0, v, CTRL, ROWS, 0xF, false);
}
template <typename F>
__device__ __forceinline__ int wave_prefix(int v, F&& f)
{
    v = f(v, from_before<0x111, 0xF>(v));  // row_shr 1, 2, 4, 8
    v = f(v, from_before<0x112, 0xF>(v));
    v = f(v, from_before<0x114, 0xF>(v));
    v = f(v, from_before<0x118, 0xF>(v));
    v = f(v, from_before<0x142, 0xA>(v));  // row_bcast 15, 31
    v = f(v, from_before<0x143, 0xC>(v));
    return v;
}

// 64 experts from `base` on, one per lane: their rows [lo, hi), with the
// offsets read as running maxima in [0, R], and the tiles of BQ rows up to and
// with them; `carry` and `before` hold what precedes.
template <int BQ>
__device__ __forceinline__ void expert_rows(const GroupedArgs& a, int base, int lane, int& carry,
                                            int& before, int& lo, int& hi, int& upto)
{
    const int j = base + lane;
    const bool live = j < a.E;
    const int first = live ? a.offsets[j] : 0, last = live ? a.offsets[j + 1] : 0;
    lo = wave_prefix(min(max(first, 0), a.f.R), [](int x, int y) { return max(x, y); });
    lo = max(lo, carry);
    hi = live ? max(lo, min(max(last, 0), a.f.R)) : lo;
    upto = before + wave_prefix((hi - lo + BQ - 1) / BQ, [](int x, int y) { return x + y; });
    carry = __builtin_amdgcn_readlane(hi, 63);
    before = __builtin_amdgcn_readlane(upto, 63);
}

// f becomes the arguments of expert e, whose rows end at m1.
__device__ __forceinline__ void set_expert(const GroupedArgs& a, FfnArgs& f, int e, int m1)
{
    const size_t weights = (size_t)e * (size_t)a.f.C * (size_t)a.f.ldp;
    f.P[0] = a.f.P[0] + weights;
    f.P[1] = a.f.P[1] + weights;
    f.sp[0] = a.f.sp[0] + (size_t)e * a.f.C;
    f.sp[1] = a.f.sp[1] + (size_t)e * a.f.C;
    f.R = m1;
}

// Tiles are numbered expert by expert, within one column by column, so that
// the row tiles that share an expert's weights run at the same time on an XCD
// and read them from its L2 (which takes a run of the numbers, see xcd_tile):
// number t of `total` row tiles times tc columns.
__device__ __forceinline__ int xcd_run(int bid, int all)
{
    int t, one;
    xcd_tile(bid, 1, all, 1, one, t);
    return t;
}

// Tile `bid` of all (BQ rows by 1 / tc of the columns): false past the last;
// else f becomes the arguments of its expert, rows r0 .. f.R - 1.
template <int BQ>
__device__ __forceinline__ bool find_tile(const GroupedArgs& a, unsigned bid, int tc, int lane,
                                          FfnArgs& f, int& r0, int& tile_c)
{
    int carry = 0, total = 0, lo, hi, upto;
    for (int base = 0; base < a.E; base += 64)
        expert_rows<BQ>(a, base, lane, carry, total, lo, hi, upto);
    if ((int64_t)bid >= (int64_t)total * tc)
        return false;
    const int t = xcd_run((int)bid, total * tc);
    const int row = t / tc;  // (of this expert, as are the tiles of a run of tc)
    int base = 0;
    uint64_t hit = a.E <= 64 ? __ballot(upto > row) : 0;
    if (a.E > 64) {
        carry = total = 0;
        for (; !hit; base += 64) {
            expert_rows<BQ>(a, base, lane, carry, total, lo, hi, upto);
            hit = __ballot(upto > row);
        }
        base -= 64;
    }
    const int L = __ffsll((long long)hit) - 1;
    const int last = __builtin_amdgcn_readlane(upto, L);
    r0 = __builtin_amdgcn_readlane(lo, L);
    const int m1 = __builtin_amdgcn_readlane(hi, L);
    const int n = (m1 - r0 + BQ - 1) / BQ;  // the expert's row tiles
    const int local = t - (last - n) * tc;
    tile_c = local / n;
    r0 += (local - tile_c * n) * BQ;
    f = a.f;
    set_expert(a, f, base + L, m1);
    return true;
}

// Resource of the rows of A that a tile from r0 on reads: all tokens, or the
// tile's own rows.
template <int BQ>
__device__ __forceinline__ const uint8_t* row_base(const FfnArgs& f, int r0, uint32_t& bytes)
{
    if (f.rows) {
        bytes = (uint32_t)f.tokens * (uint32_t)f.ldq;
        return f.Q[0];
    }
    bytes = (uint32_t)min(f.R - r0, BQ) * (uint32_t)f.ldq;
    return f.Q[0] + (size_t)r0 * (size_t)f.ldq;
}
// Offset of row r0 + i there, out of range where there is none.
__device__ __forceinline__ uint32_t row_offset(const FfnArgs& f, int r0, int i)
{
    if (r0 + i >= f.R)
        return kOutOfRange;
    if (!f.rows)
        return (uint32_t)i * (uint32_t)f.ldq;
    const int t = f.rows[r0 + i];
    return (unsigned)t < (unsigned)f.tokens ? (uint32_t)t * (uint32_t)f.ldq : kOutOfRange;
}

// Ring of S stages, as ffn_ring_kernel.
template <int BP, int BQ, int WP, int WQ, int S>
__global__ __launch_bounds__(WP* WQ * 64, 2) void moe_ring_kernel(GroupedArgs a)
{
    using Copies = FfnCopies<true, LAY_NT, true, BP, BQ, WP, WQ>;
    using SP = typename Copies::SP;
    using SQ = typename Copies::SQ;
    constexpr int SLOT = Copies::SLOT;
    constexpr int LPT = 2 * (SP::LD + SQ::LD);
    constexpr int WAVES = WP * WQ;
    constexpr int TC = BP / 2;
    __shared__ __attribute__((aligned(1024))) uint8_t ring[S * SLOT];

    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wp = wave % WP, wq = wave / WP;
    int tile_c, r0;
    FfnArgs f;
    if (!find_tile<BQ>(a, blockIdx.x, (a.f.C + TC - 1) / TC, lane, f, r0, tile_c))
        return;
    const int c0 = tile_c * TC;
    const Copies cp(f, wave, lane);
    const uint32_t ldp = (uint32_t)f.ldp;

    FfnSource<false> src_p[2];
#pragma unroll
    for (int h = 0; h < 2; ++h)
        src_p[h].set(f.P[h], ldp, c0, f.C, f.klen, 1, cp.vp, cp.chp);
    uint32_t bytes;
    const uint8_t* from = row_base<BQ>(f, r0, bytes);
    const v4i rs_q = buffer_rsrc(from, bytes);
    uint32_t row[2][SQ::LD];
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int i = 0; i < SQ::LD; ++i) {
            int line, ch;
            SQ::source(i, wave, lane, line, ch);
            row[h][i] = row_offset(f, r0, ffn_tile_row<SQ, false>(h, line));
        }
    uint32_t kq = cp.chq * 16;  // this lane's chunk of the next stage
    const uint32_t to = __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)ring + wave * 1024);
    auto issue = [&](int s) __attribute__((always_inline)) {
        const uint32_t at = to + (uint32_t)s * SLOT;
        const bool in = kq < (uint32_t)f.klen;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
#pragma unroll
            for (int i = 0; i < SP::LD; ++i)
                dma16(src_p[h].v + cp.shift_p(h, i), src_p[h].rs,
                      at + h * SP::HB + i * (WAVES * 1024));
#pragma unroll
            for (int i = 0; i < SQ::LD; ++i)
                dma16(in ? row[h][i] + kq : kOutOfRange, rs_q,
                      at + 2 * SP::HB + h * SQ::HB + i * (WAVES * 1024));
        }
#pragma unroll
        for (int h = 0; h < 2; ++h)
            src_p[h].next(ldp, c0, cp.chp);
        kq += 128;
    };

    v4f acc[2][SP::NB][2][SQ::NB];
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int j = 0; j < SP::NB; ++j)
#pragma unroll
            for (int q = 0; q < 2; ++q)
#pragma unroll
                for (int i = 0; i < SQ::NB; ++i)
                    acc[h][j][q][i] = v4f{0, 0, 0, 0};

    uint4 fp[2][2][SP::NB][2], fq[2][2][SQ::NB][2];
    auto read = [&](auto SET, int s) __attribute__((always_inline)) {
        constexpr int set = decltype(SET)::value;
        const uint8_t* sp = ring + s * SLOT;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
#pragma unroll
            for (int j = 0; j < SP::NB; ++j)
                ffn_frag<SP, false>(sp + h * SP::HB, wp, j, lane, fp[set][h][j]);
#pragma unroll
            for (int i = 0; i < SQ::NB; ++i)
                ffn_frag<SQ, false>(sp + 2 * SP::HB + h * SQ::HB, wq, i, lane, fq[set][h][i]);
        }
    };
    using I0 = std::integral_constant<int, 0>;
    using I1 = std::integral_constant<int, 1>;
    const int n = f.nks;
#pragma unroll
    for (int s = 0; s < S; ++s)
        if (s < n)
            issue(s);
    wait_younger<S - 1, LPT>(min(S - 1, n - 1));
    read(I0{}, 0);
    int slot = 0;
    auto stage = [&](auto SET, auto OTHER, int k) __attribute__((always_inline)) {
        constexpr int set = decltype(SET)::value;
        const int next = slot + 1 == S ? 0 : slot + 1;
        if (k + 1 < n) {
            wait_younger<S - 2, LPT>(min(S - 2, n - 2 - k));
            if (k + S < n)
                issue(slot);
            read(OTHER, next);
        }
        slot = next;
#pragma unroll
        for (int q = 0; q < 2; ++q)
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int j = 0; j < SP::NB; ++j)
#pragma unroll
                    for (int i = 0; i < SQ::NB; ++i)
                        acc[h][j][q][i] =
                            ffn_mfma<true>(fp[set][h][j], fq[set][q][i], acc[h][j][q][i]);
    };
    for (int k = 0; k < n; k += 2) {
        stage(I0{}, I1{}, k);
        if (k + 1 < n)
            stage(I1{}, I0{}, k + 1);
    }
    ffn_finish<SP, SQ, true, EPI_GROUPED>(f, acc, c0, r0, 0, wp, wq, WQ, lane);
}

// The 256x256 tile over experts (see ffn_alt.h).  A workgroup works on several
// tiles, so it keeps the experts' rows and tiles in LDS.
constexpr int kAltExperts = 1024;
struct Grouped {
    static constexpr bool GATHER = true;
    const GroupedArgs& g;
    const int *lo, *hi, *upto;  // of each expert (see expert_rows)
    int tr, tc, lane;
    __device__ __forceinline__ int tiles() const { return tr * tc; }
    __device__ __forceinline__ void at(int t, FfnArgs& f, int& r0, int& c0) const
    {
        t = xcd_run(t, tr * tc);
        const int tile = t / tc;
        uint64_t hit = 0;
        int base = -64;
        while (!hit) {  // (tile < tr = the last of upto)
            base += 64;
            hit = __ballot(base + lane < g.E && upto[min(base + lane, g.E - 1)] > tile);
        }
        const int e = base + __ffsll((long long)hit) - 1;
        r0 = __builtin_amdgcn_readfirstlane(lo[e]);
        const int m1 = __builtin_amdgcn_readfirstlane(hi[e]);
        const int last = __builtin_amdgcn_readfirstlane(upto[e]);
        const int n = (m1 - r0 + 255) / 256;  // the expert's row tiles
        const int local = t - (last - n) * tc;
        c0 = local / n * 128;
        r0 += local % n * 256;
        set_expert(g, f, e, m1);
    }
    __device__ __forceinline__ void rows(const FfnArgs& f, int r0, v4i& rs) const
    {
        uint32_t bytes;
        const uint8_t* from = row_base<256>(f, r0, bytes);
        rs = buffer_rsrc(from, bytes);
    }
    __device__ __forceinline__ uint32_t row(const FfnArgs& f, int r0, int i) const
    {
        return row_offset(f, r0, i);
    }
};

__global__ __launch_bounds__(512, 2) void moe_alt_kernel(GroupedArgs a)
{
    __shared__ int lo[kAltExperts], hi[kAltExperts], upto[kAltExperts];
    const int lane = threadIdx.x & 63;
    int carry = 0, total = 0;
    for (int base = 0; base < a.E; base += 64) {
        int l, h, u;
        expert_rows<256>(a, base, lane, carry, total, l, h, u);
        if (threadIdx.x < 64 && base + lane < a.E) {
            lo[base + lane] = l;
            hi[base + lane] = h;
            upto[base + lane] = u;
        }
    }
    __syncthreads();
    const Grouped where = {a, lo, hi, upto, total, (a.f.C + 127) / 128, lane};
    ffn_alt_tiles<true, LAY_NT, EPI_GROUPED>(a.f, where, blockIdx.x, gridDim.x);
}

// Few rows and few tiles, as ffn_skinny_kernel: 8 columns (their gate and up
// rows make one block of 16) of 16 rows, K split over the W waves.
template <int W>
__global__ __launch_bounds__(W * 64) void moe_skinny_kernel(GroupedArgs a)
{
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int i = lane & 15, g = lane >> 4;
    int r0, tile_c;
    FfnArgs f;
    if (!find_tile<16>(a, blockIdx.x, (a.f.C + 7) / 8, lane, f, r0, tile_c))
        return;
    const int c0 = tile_c * 8;
    const int kbytes = f.klen;
    uint32_t bytes;
    const uint8_t* from = row_base<16>(f, r0, bytes);
    const __amdgpu_buffer_rsrc_t rq =
        __builtin_amdgcn_make_buffer_rsrc((void*)from, (short)0, (int)bytes, 0x00020000);
    const uint8_t* pp = (i >= 8 ? f.P[1] : f.P[0]) + (size_t)min(c0 + (i & 7), f.C - 1) * f.ldp + g * 16;
    const uint32_t vq = row_offset(f, r0, i) + g * 16;
    v4f acc = {0, 0, 0, 0};
    const int steps = (kbytes + 127) >> 7;
    for (int s = wave; s < steps; s += W) {
        uint4 p[2], q[2];
#pragma unroll
        for (int ks = 0; ks < 2; ++ks) {
            const int off = s * 128 + ks * 64;
            const bool in = off + g * 16 < kbytes;  // else past the row's end: zeros
            const uint32_t keep = in ? 0xFFFFFFFFu : 0u;
            const uint4 v = *(const uint4*)(pp + (in ? off : -16 * g));
            p[ks] = make_uint4(v.x & keep, v.y & keep, v.z & keep, v.w & keep);
            q[ks] = __builtin_bit_cast(uint4, __builtin_amdgcn_raw_buffer_load_b128(
                                                  rq, (int)(in ? vq + off : kOutOfRange), 0, 0));
        }
        acc = mfma_step<OP_FP8>(p, q, acc);
    }

    // partial sums [wave][row][block row]
    __shared__ __attribute__((aligned(16))) float red[W][16][16];
    *(float4*)&red[wave][i][g * 4] = make_float4(acc[0], acc[1], acc[2], acc[3]);
    __syncthreads();
    if (threadIdx.x < 256) {
        const int br = threadIdx.x & 15, r = r0 + (int)(threadIdx.x >> 4);
        float v = 0.0f;
#pragma unroll
        for (int w = 0; w < W; ++w)
            v += red[w][threadIdx.x >> 4][br];
        const int c = c0 + br;
        const float u = __shfl_xor(v, 8, 64);
        if (br < 8 && c < f.C && r < f.R) {
            const float s = grouped_scale(f, r);
            float z = v * s * f.sp[0][c];
            with_act(f.act, [&](auto A) { z = act_value<decltype(A)::value>(z); });
            store_value(f, z * (u * s * f.sp[1][c]), r, c);
        }
    }
}

// The kernels, by the rows of a tile and the columns it writes.
struct Shape {
    int rows, cols, threads;
};
enum Pick : int { FEW = 0, SMALL, MID, LARGE, ALT };
constexpr Shape kShapes[] = {{16, 8, 512}, {64, 32, 256}, {64, 64, 256}, {128, 128, 512}, {256, 128, 512}};

// Most workgroups that have a tile.
int64_t grid_of(const Shape& s, const GroupedArgs& a)
{
    const int64_t rows = a.f.R / s.rows + (a.E < a.f.R ? a.E : a.f.R);
    return rows * ((a.f.C + s.cols - 1) / s.cols);
}
bool launchable(const Shape& s, const GroupedArgs& a)
{
    return grid_of(s, a) * s.threads < (int64_t)1 << 32;
}
// About as many tiles as there are where every other expert has a ragged one.
int64_t likely(const Shape& s, const GroupedArgs& a)
{
    const int64_t rows = a.f.R / s.rows + (a.E < a.f.R ? a.E + 1 : a.f.R + 1) / 2;
    return rows * ((a.f.C + s.cols - 1) / s.cols);
}

// Measured (us), skewed routing, few-row kernel / tiles of 64x32, 64x64, 128x128
// and 256x128 outputs.  E = 64 experts of N = 1536, K = 2048, top-8: 1 token
// 14.3, 11.6, 12.8, 19, 21; 4 tokens -, 29.0, 27.5, 32, 35; 67 tokens -, 73, 72,
// 75, 78; 256 (32 rows an expert) -, 89, 82, 86, 85; 512 -, 110, 97, 93, 100; 1024
// -, 157, 132, 114, 121; 2048 -, 249, 208, 174, 152; 4096 -, 432, 360, 301, 243.
// Few tiles: E = 64, N = 512, 1 token 6.3, 9.0, 11.1, 18, 20; E = 8, N = 1536, 2048
// rows -, 31, 27.4, 23.7, 30.2.  The rule takes the mean, since the loads are known on
// the device alone: 2048 rows of 8 among 64 experts take tiles for fewer rows, 25.7
// us against 22.8 where these 8 are all there are; with half of 2048 rows at one of
// 64 it is 84, the time of the weights.
int pick(const GroupedArgs& a)
{
    const int64_t per = a.f.R / a.E;
    if (per >= 192 && a.E <= kAltExperts && likely(kShapes[ALT], a) >= 256)
        return ALT;
    if (per >= 48 && likely(kShapes[LARGE], a) >= 128 && launchable(kShapes[LARGE], a))
        return LARGE;
    if (per <= 8 && grid_of(kShapes[SMALL], a) < 256)
        return FEW;
    if (grid_of(kShapes[MID], a) <= 256 || !launchable(kShapes[MID], a))
        return launchable(kShapes[SMALL], a) ? SMALL : LARGE;
    return MID;
}

}  // namespace

bool moe_gated_fits(const GroupedArgs& a) { return launchable(kShapes[pick(a)], a); }

hipError_t launch_moe_gated(const GroupedArgs& a, hipStream_t stream)
{
    const int shape = pick(a);
    const unsigned grid = (unsigned)grid_of(kShapes[shape], a);
    switch (shape) {
    case FEW:
        moe_skinny_kernel<8><<<grid, 512, 0, stream>>>(a);
        break;
    case SMALL:  // three workgroups per CU
        moe_ring_kernel<64, 64, 2, 2, 3><<<grid, 256, 0, stream>>>(a);
        break;
    case MID:  // two
        moe_ring_kernel<128, 64, 2, 2, 3><<<grid, 256, 0, stream>>>(a);
        break;
    case LARGE:  // one, as below
        moe_ring_kernel<256, 128, 4, 2, 3><<<grid, 512, 0, stream>>>(a);
        break;
    default:
        moe_alt_kernel<<<256, 512, 0, stream>>>(a);
    }
    return hipGetLastError();
}

}  // namespace qll
