// The experts' gated products for gfx950: every row of A, or the token that
// rows[] names, times its expert's gate and up weights.
//
//   out[i] = act(sum_k A[t][k] Bg[e][n][k] sa[t] sg[e][n]) *
//            (sum_k A[t][k] Bu[e][n][k] sa[t] su[e][n]),  t = rows[i], e owns i
//
// A workgroup finds its expert from the offsets (group_tile, lane-parallel
// over 64 experts) and computes a row tile of it with the building blocks of
// the dense feed-forward products; the tokens are gathered by the copies
// themselves, so no sorted copy of A is made.  The number of row tiles is
// known on the device alone: the grid holds the most there can be (R / rows of
// a tile + min(E, R)), and workgroups past the last tile leave at once.
#include "ffn_tile.h"
#include "moe_internal.h"

namespace qll {

namespace {

// Row tile t of BQ rows: false past the last one; else f becomes the
// arguments of its expert, rows r0 .. f.R - 1.
template <int BQ>
__device__ __forceinline__ bool find_tile(const GroupedArgs& a, int t, int lane, FfnArgs& f, int& r0)
{
    int e, m1;
    group_tile(a.offsets, a.E, a.f.R, t, BQ, lane, e, r0, m1);
    e = __builtin_amdgcn_readfirstlane(e);
    r0 = __builtin_amdgcn_readfirstlane(r0);
    if (e < 0)
        return false;
    f = a.f;
    const size_t weights = (size_t)e * (size_t)f.C * (size_t)f.ldp;
    f.P[0] += weights;
    f.P[1] += weights;
    f.sp[0] += (size_t)e * f.C;
    f.sp[1] += (size_t)e * f.C;
    f.R = __builtin_amdgcn_readfirstlane(m1);
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
    const int tc = (a.f.C + TC - 1) / TC;
    const int tr = __builtin_amdgcn_readfirstlane(group_row_tiles(a.offsets, a.E, a.f.R, BQ, lane));
    if ((int64_t)blockIdx.x >= (int64_t)tr * tc)
        return;
    int tile_r, tile_c, r0;
    xcd_tile(blockIdx.x, tr, tc, 4, tile_r, tile_c);
    FfnArgs f;
    if (!find_tile<BQ>(a, tile_r, lane, f, r0))
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
    ffn_finish<SP, SQ, true, EPI_GROUPED>(f, acc, c0, r0, tile_r, wp, wq, WQ, lane);
}

// Few rows per expert, as ffn_skinny_kernel: 8 columns (their gate and up rows
// make one block of 16) of TB * 16 rows, K split over the W waves.
template <int TB, int W>
__global__ __launch_bounds__(W * 64) void moe_skinny_kernel(GroupedArgs a)
{
    static_assert(W >= 4 * TB, "a thread per sum");
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int i = lane & 15, g = lane >> 4;
    const unsigned blocks = (unsigned)(a.f.C + 7) / 8;
    const int tile = (int)(blockIdx.x / blocks);
    const int c0 = (int)(blockIdx.x - tile * blocks) * 8;
    FfnArgs f;
    int r0;
    if (!find_tile<TB * 16>(a, tile, lane, f, r0))
        return;
    const int kbytes = f.klen;
    uint32_t bytes;
    const uint8_t* from = row_base<TB * 16>(f, r0, bytes);
    const __amdgpu_buffer_rsrc_t rq =
        __builtin_amdgcn_make_buffer_rsrc((void*)from, (short)0, (int)bytes, 0x00020000);
    const uint8_t* pp = (i >= 8 ? f.P[1] : f.P[0]) + (size_t)min(c0 + (i & 7), f.C - 1) * f.ldp + g * 16;
    uint32_t vq[TB];
    v4f acc[TB];
#pragma unroll
    for (int t = 0; t < TB; ++t) {
        vq[t] = row_offset(f, r0, 16 * t + i) + g * 16;
        acc[t] = v4f{0, 0, 0, 0};
    }
    const int steps = (kbytes + 127) >> 7;
    for (int s = wave; s < steps; s += W) {
        uint4 p[2], q[TB][2];
#pragma unroll
        for (int ks = 0; ks < 2; ++ks) {
            const int off = s * 128 + ks * 64;
            const bool in = off + g * 16 < kbytes;  // else past the row's end: zeros
            const uint32_t keep = in ? 0xFFFFFFFFu : 0u;
            const uint4 v = *(const uint4*)(pp + (in ? off : -16 * g));
            p[ks] = make_uint4(v.x & keep, v.y & keep, v.z & keep, v.w & keep);
#pragma unroll
            for (int t = 0; t < TB; ++t)
                q[t][ks] = __builtin_bit_cast(
                    uint4, __builtin_amdgcn_raw_buffer_load_b128(
                               rq, (int)(in ? vq[t] + off : kOutOfRange), 0, 0));
        }
#pragma unroll
        for (int t = 0; t < TB; ++t)
            acc[t] = mfma_step<OP_FP8>(p, q[t], acc[t]);
    }

    // partial sums [wave][row][block row]
    __shared__ __attribute__((aligned(16))) float red[W][TB * 16][16];
#pragma unroll
    for (int t = 0; t < TB; ++t)
        *(float4*)&red[wave][16 * t + i][g * 4] =
            make_float4(acc[t][0], acc[t][1], acc[t][2], acc[t][3]);
    __syncthreads();
    if (threadIdx.x < TB * 256) {
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
constexpr Shape kShapes[] = {{16, 8, 512}, {64, 32, 256}, {128, 64, 256}};

int64_t grid_of(const Shape& s, const GroupedArgs& a)
{
    const int64_t rows = a.f.R / s.rows + (a.E < a.f.R ? a.E : a.f.R);
    return rows * ((a.f.C + s.cols - 1) / s.cols);
}
bool launchable(const Shape& s, const GroupedArgs& a)
{
    return grid_of(s, a) * s.threads < (int64_t)1 << 32;
}

int pick(const GroupedArgs& a)
{
    const int64_t per = a.f.R / a.E;
    if (per <= 12 && launchable(kShapes[0], a))
        return 0;
    return per <= 48 && launchable(kShapes[1], a) ? 1 : 2;
}

}  // namespace

bool moe_gated_fits(const GroupedArgs& a) { return launchable(kShapes[pick(a)], a); }

hipError_t launch_moe_gated(const GroupedArgs& a, hipStream_t stream)
{
    const int shape = pick(a);
    const unsigned grid = (unsigned)grid_of(kShapes[shape], a);
    if (shape == 0)
        moe_skinny_kernel<1, 8><<<grid, 512, 0, stream>>>(a);
    else if (shape == 1)
        moe_ring_kernel<64, 64, 2, 2, 4><<<grid, 256, 0, stream>>>(a);
    else
        moe_ring_kernel<128, 128, 2, 2, 2><<<grid, 256, 0, stream>>>(a);
    return hipGetLastError();
}

}  // namespace qll
