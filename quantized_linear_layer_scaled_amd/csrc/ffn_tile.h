// Tiled matrix products of the feed-forward operators for gfx950.
//
//   out[r][c] = epilogue(sum_k Q[r][k] P[c][k])
//
// P is the operand along the output's columns and takes the row side of the
// matrix cores, Q the one along its rows: a lane then holds 4 consecutive
// output columns of one row per 16x16 block, and with the P rows of two
// blocks interleaved by fours, 8 of them.  So outputs, residuals and biases
// move as 8- or 16-byte vectors straight from the accumulators, with no trip
// through LDS, and the gate and up sums of one output are in one lane.
//
// A tile is BP x BQ over WP x WQ waves; each operand's tile rows come in two
// halves.  A stage is 128 bytes of a K-contiguous row (64 bf16 or 128 e4m3
// elements).  LDS images of one half of H rows, H * 128 bytes either way:
//   K-contiguous operand: [H][128 bytes], 16-byte chunks XOR-swizzled by row;
//   K-strided operand (bf16): [64 k][H * 2 bytes], as it lies in memory; the
//     fragments are read with ds_read_b64_tr_b16, which hands lane i of 16
//     the i-th column of a 4 x 16 block.  32-byte pairs of chunks are
//     XOR-swizzled by k so that the eight k lines that 32 lanes read at once
//     fall on distinct banks.
// Lane group g = lane / 16 takes the 16-byte chunks 2 g and 2 g + 1 of a
// stage (K elements 16 g .. 16 g + 15 of 64 in bf16): a reordering of K that
// both operands share.  The LDS serves a b128 read 16 lanes at a time, from
// two neighbouring groups; chunks g and g + 4 instead, with the same swizzle,
// cost two passes for each (counters: 4 conflict cycles on 4 per read; none
// this way).
// Copies go from global memory to LDS directly (buffer_load_dwordx4 ... lds)
// through resources that end where the matrix ends: rows past the end, and K
// past the end of a strided operand, read as zeros; K past the end of a
// contiguous row gets an offset out of range.  No operand size overflows the
// 32-bit offsets: a contiguous operand's cover 256 rows, a strided one's 64 k
// lines from a 64-bit base that moves on with the stages.
#pragma once

#include "ffn_epilogue.h"
#include "gemm_pipe.h"

namespace qll {

typedef short v4s __attribute__((ext_vector_type(4)));

// Bank swizzles (see the header comment).  NB: interleaved blocks per half.
// P, contiguous: the 16 rows of a fragment are 4 NB a + 4 j + b (a, b < 4).
template <int NB>
__device__ __forceinline__ int ffn_swz(int row)
{
    return ((row & 3) | (((row / (4 * NB)) & 1) << 2)) ^ ((row / (8 * NB)) & 1);
}
// strided: 32-byte pair key of k line `k` for lines of H * 2 bytes
template <int H>
__device__ __forceinline__ int ffn_kkey(int k)
{
    if constexpr (H >= 128)
        return (k & 3) | (((k >> 4) & 1) << 2);
    else if constexpr (H == 64)
        return ((k >> 1) & 1) | (((k >> 4) & 1) << 1);
    else
        return (k >> 4) & 1;
}

// One operand's geometry within a tile of B rows over W waves (WAVES in all):
// STR strided, ILV the blocks of a half interleaved by fours.
template <int B, int W, int WAVES, bool STR, bool ILV>
struct FfnSide {
    static constexpr int H = B / 2;               // rows of a half
    static constexpr int HB = H * 128;            // its bytes in LDS
    static constexpr int SH = H / W;              // a wave's rows of a half
    static constexpr int NB = SH / 16;            // its 16-row blocks
    static constexpr int LD = HB / 1024 / WAVES;  // copies per wave and half
    static constexpr int NBI = ILV ? NB : 1;      // interleaved blocks
    static constexpr int CPL = H / 8;             // strided: chunks per k line
    static_assert(SH % 16 == 0 && HB % (1024 * WAVES) == 0 && H <= 128, "tile geometry");

    // local row of fragment row i of block j, within the wave's share
    static __device__ __forceinline__ int frag_row(int j, int i)
    {
        return ILV ? 4 * NB * (i >> 2) + 4 * j + (i & 3) : 16 * j + i;
    }
    // copy i of this wave: this lane's LDS line and logical 16-byte chunk
    static __device__ __forceinline__ void source(int i, int wave, int lane, int& line, int& ch)
    {
        const int L = (i * WAVES + wave) * 64 + lane;
        if constexpr (STR) {
            line = L / CPL;
            ch = (L % CPL) ^ (ffn_kkey<H>(line) << 1);
        } else {
            line = L / 8;
            ch = (L % 8) ^ ffn_swz<NBI>(line);
        }
    }
};

// Row of the tile that local row r of half h stands for.  SPLIT: the halves
// interleave per wave share (a wave's 2 SH rows are consecutive); else half h
// is rows h * H .. of the tile.
template <typename S, bool SPLIT>
__device__ __forceinline__ int ffn_tile_row(int h, int r)
{
    return SPLIT ? (r / S::SH) * 2 * S::SH + h * S::SH + r % S::SH : h * S::H + r;
}

template <bool FP8>
__device__ __forceinline__ v4f ffn_mfma(const uint4 (&p)[2], const uint4 (&q)[2], v4f c)
{
    if constexpr (FP8) {
        return mfma_step<OP_FP8>(p, q, c);
    } else {
        c = mfma_step<OP_BF16>(&p[0], &q[0], c);
        return mfma_step<OP_BF16>(&p[1], &q[1], c);
    }
}

// Fragment (16 rows, one 128-byte stage: two 16-byte pieces per lane) of
// block j of this wave's share of a half.
template <typename S, bool STR>
__device__ __forceinline__ void ffn_frag(const uint8_t* half, int w, int j, int lane, uint4 (&f)[2])
{
    const int i = lane & 15, g = lane >> 4;
    if constexpr (STR) {
        const int pair = (w * S::SH) / 16 + j;
#pragma unroll
        for (int ks = 0; ks < 2; ++ks) {
            v4s t[2];
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                const int k = g * 16 + ks * 8 + s * 4 + (i >> 2);
                const uint8_t* p = half + k * (S::H * 2) + ((pair ^ ffn_kkey<S::H>(k)) << 5) +
                                   ((i & 3) << 3);
                t[s] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                    (__attribute__((address_space(3))) v4s*)p);
            }
            const uint2 lo = __builtin_bit_cast(uint2, t[0]), hi = __builtin_bit_cast(uint2, t[1]);
            f[ks] = make_uint4(lo.x, lo.y, hi.x, hi.y);
        }
    } else {
        const int row = w * S::SH + S::frag_row(j, i);
        const int key = ffn_swz<S::NBI>(row);
#pragma unroll
        for (int ks = 0; ks < 2; ++ks)
            f[ks] = *(const uint4*)(half + row * 128 + (((2 * g + ks) ^ key) << 4));
    }
}

// The epilogue of one wave: acc[h][j][hq][i], see FfnSide for the rows.
template <typename SP, typename SQ, bool DUAL, int EPI>
__device__ __forceinline__ void ffn_finish(const FfnArgs& a, v4f (&acc)[2][SP::NB][2][SQ::NB],
                                           int c0, int r0, int tile_r, int wp, int wq, int wqn,
                                           int lane)
{
    // vectors of W consecutive columns (JV blocks), NV of them per half
    constexpr int W = 4 * SP::NBI;
    constexpr int JV = W / 4;
    constexpr int NV = SP::NB / JV;
    static_assert(SP::NBI <= 2, "interleave at most two blocks");
    // (opaque, so that a loop over tiles does not keep what is derived from
    // it in registers through the products)
    asm volatile("" : "+v"(lane));
    const int g = lane >> 4;
    // f(h, jv, first column): the wave's column vectors
    auto columns = [&](auto&& f) __attribute__((always_inline)) {
#pragma unroll
        for (int h = 0; h < (DUAL ? 1 : 2); ++h)
#pragma unroll
            for (int jv = 0; jv < NV; ++jv) {
                const int local = wp * SP::SH + SP::frag_row(jv * JV, 4 * g);
                f(h, jv, c0 + ffn_tile_row<SP, !DUAL>(h, local));
            }
    };
    // f(v, u, row): the sums of one column vector, row by row
    auto rows = [&](int h, int jv, auto&& f) __attribute__((always_inline)) {
#pragma unroll
        for (int hq = 0; hq < 2; ++hq) {
            // (a limit on how many rows' loads are in registers)
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int i = 0; i < SQ::NB; ++i) {
                float v[W], u[W];
#pragma unroll
                for (int e = 0; e < W; ++e) {
                    v[e] = acc[h][jv * JV + e / 4][hq][i][e & 3];
                    u[e] = DUAL ? acc[1][jv * JV + e / 4][hq][i][e & 3] : 0.0f;
                }
                f(v, u, r0 + hq * SQ::H + wq * SQ::SH + 16 * i + (lane & 15));
            }
        }
    };
    auto run = [&](auto A) __attribute__((always_inline)) {
        columns([&](int h, int jv, int c) __attribute__((always_inline)) {
            float cs[W];
#pragma unroll
            for (int e = 0; e < W; ++e)
                cs[e] = 0.0f;
            ColumnVector<W> cv;
            load_columns<EPI, W>(a, c, cv);
            rows(h, jv, [&](float* v, float* u, int r) __attribute__((always_inline)) {
                ffn_store_act<EPI, W, decltype(A)::value>(a, v, u, r, c, cv, cs);
            });
            if constexpr (EPI == EPI_DZ) {
                // the wave's column sums over its rows (16 lanes share a
                // column vector): one row of `partial` per tile and wave
                // row, added up in a fixed order by launch_colsum_finish
#pragma unroll
                for (int e = 0; e < W; ++e)
#pragma unroll
                    for (int d = 1; d < 16; d <<= 1)
                        cs[e] += __shfl_xor(cs[e], d, 64);
                if (a.partial && (lane & 15) == 0 && c < a.C)
                    store_f32<W>(a.partial + (size_t)(tile_r * wqn + wq) * a.C + c, cs);
            }
        });
    };
    if constexpr (EPI == EPI_PARTIAL || EPI == EPI_PLAIN)
        run(std::integral_constant<int, ACT_NONE>{});
    else
        with_act(a.act, run);
}

// A wave's copies of a tile: per-lane source offsets relative to the tile's
// corner.
template <bool FP8, int LAY, bool DUAL, int BP, int BQ, int WP, int WQ>
struct FfnCopies {
    static constexpr int WAVES = WP * WQ;
    static constexpr bool PSTR = LAY != LAY_NT, QSTR = LAY == LAY_TN;
    static_assert(!FP8 || LAY == LAY_NT, "e4m3 operands are K-contiguous");
    using SP = FfnSide<BP, WP, WAVES, PSTR, !PSTR>;
    using SQ = FfnSide<BQ, WQ, WAVES, QSTR, false>;
    static constexpr int SLOT = (BP + BQ) * 128;

    const FfnArgs& a;
    // the source offsets of copy 0 of half 0; the others differ by the same
    // scalar in every lane
    uint32_t vp, vq;
    int chp, chq;
    static constexpr int LINES_P = PSTR ? WAVES * 64 / SP::CPL : WAVES * 8;
    static constexpr int LINES_Q = QSTR ? WAVES * 64 / SQ::CPL : WAVES * 8;
    static_assert((PSTR || LINES_P % SP::SH == 0) && LINES_P % 32 == 0 && LINES_Q % 32 == 0,
                  "copies of a half repeat the swizzle");

    __device__ __forceinline__ FfnCopies(const FfnArgs& args, int w, int lane)
        : a(args)
    {
        int line;
        SP::source(0, w, lane, line, chp);
        vp = PSTR ? (uint32_t)line * (uint32_t)a.ldp + 2 * ffn_tile_row<SP, !DUAL>(0, chp * 8)
                  : (uint32_t)ffn_tile_row<SP, !DUAL>(0, line) * (uint32_t)a.ldp + chp * 16;
        SQ::source(0, w, lane, line, chq);
        vq = QSTR ? (uint32_t)line * (uint32_t)a.ldq + 2 * ffn_tile_row<SQ, false>(0, chq * 8)
                  : (uint32_t)ffn_tile_row<SQ, false>(0, line) * (uint32_t)a.ldq + chq * 16;
    }
    // what copy i of half h adds (DUAL: the two weights have a base each)
    __device__ __forceinline__ uint32_t shift_p(int h, int i) const
    {
        const int hh = DUAL ? 0 : h;
        return PSTR ? (uint32_t)(i * LINES_P) * (uint32_t)a.ldp + 2 * ffn_tile_row<SP, !DUAL>(hh, 0)
                    : (uint32_t)ffn_tile_row<SP, !DUAL>(hh, i * LINES_P) * (uint32_t)a.ldp;
    }
    __device__ __forceinline__ uint32_t shift_q(int h, int i) const
    {
        return QSTR ? (uint32_t)(i * LINES_Q) * (uint32_t)a.ldq + 2 * ffn_tile_row<SQ, false>(h, 0)
                    : (uint32_t)ffn_tile_row<SQ, false>(h, i * LINES_Q) * (uint32_t)a.ldq;
    }
};

// One operand's source of the copies of a tile: its resource and this lane's
// offset at the stage being copied.  A K-contiguous operand keeps its resource
// (the tile's rows) and moves the offset; past the end of K the offset is out
// of range.  A K-strided one keeps the offset and moves the resource by 64 k
// lines; it ends where the matrix does.  All of it is 32-bit arithmetic once
// per stage, so that a copy is one addition and the load.
template <bool STR>
struct FfnSource {
    v4i rs;
    uint32_t v;
    int lines;  // strided: k lines from the stage to the end of the matrix
    int kleft;  // contiguous: bytes of K from the stage to the end

    // tile corner at row (column) x0 of `extent`; ch: this lane's chunk
    __device__ __forceinline__ void set(const uint8_t* base, uint32_t ld, int x0, int extent,
                                        int klen, int esz, uint32_t v0, int ch)
    {
        v = v0;
        if constexpr (STR) {
            const uint64_t at = (uint64_t)(uintptr_t)base + 2 * (int64_t)x0;
            rs.x = (int)(uint32_t)at;
            rs.y = (int)(uint32_t)(at >> 32) & 0xFFFF;
            rs.w = 0x00020000;
            lines = klen;
            limit(ld, x0);
        } else {
            // (offsets stay below 256 rows, a row past `extent` is out of range)
            const int rows = min(extent - x0, 256);
            rs = buffer_rsrc(base + (int64_t)x0 * ld, (uint32_t)rows * ld);
            kleft = klen * esz;
            clip(ch);
        }
    }
    // on by n stages
    __device__ __forceinline__ void skip(int n, uint32_t ld, int x0, int ch)
    {
        if constexpr (STR) {
            const uint64_t at =
                (((uint64_t)(uint32_t)rs.y << 32) | (uint32_t)rs.x) + (uint64_t)n * 64u * ld;
            rs.x = (int)(uint32_t)at;
            rs.y = (int)(uint32_t)(at >> 32);
            lines -= 64 * n;
            limit(ld, x0);
        } else {
            v += 128u * (uint32_t)n;
            kleft -= 128 * n;
            clip(ch);
        }
    }
    __device__ __forceinline__ void limit(uint32_t ld, int x0)
    {
        // (one stage reads 64 lines: the last of them may end the matrix)
        const int n = max(min(lines, 64), 0) * (int)ld - 2 * x0;
        rs.z = __builtin_amdgcn_readfirstlane(max(n, 0));
    }
    __device__ __forceinline__ void clip(int ch)
    {
        if (kleft < 128 && ch * 16 >= kleft)
            v = kOutOfRange;
    }
    __device__ __forceinline__ void next(uint32_t ld, int x0, int ch)
    {
        if constexpr (STR) {
            const uint64_t at = (((uint64_t)(uint32_t)rs.y << 32) | (uint32_t)rs.x) + 64ull * ld;
            rs.x = (int)(uint32_t)at;
            rs.y = (int)(uint32_t)(at >> 32);
            lines -= 64;
            limit(ld, x0);
        } else {
            v += 128;
            kleft -= 128;
            clip(ch);
        }
    }
};

// Ring of S stages.  At stage kt, once its fragments are in registers and
// stage kt + 1 has landed (one barrier), the copies of stage kt + S go into the
// slot of stage kt, the fragments of stage kt + 1 into the other register set,
// and the products of stage kt run under both.  Two waves per SIMD, from one
// workgroup of eight or two of four.
template <bool FP8, int LAY, int EPI, int BP, int BQ, int WP, int WQ, int S>
__global__ __launch_bounds__(WP* WQ * 64, 2) void ffn_ring_kernel(FfnArgs a)
{
    constexpr bool DUAL = EPI == EPI_GATED || EPI == EPI_DGATED;
    using Copies = FfnCopies<FP8, LAY, DUAL, BP, BQ, WP, WQ>;
    using SP = typename Copies::SP;
    using SQ = typename Copies::SQ;
    constexpr bool PSTR = Copies::PSTR, QSTR = Copies::QSTR;
    constexpr bool SEGS = LAY == LAY_NN;
    constexpr int SLOT = Copies::SLOT;
    constexpr int LPT = 2 * (SP::LD + SQ::LD);  // copies per wave and stage
    constexpr int WAVES = WP * WQ;
    __shared__ __attribute__((aligned(1024))) uint8_t ring[S * SLOT];

    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wp = wave % WP, wq = wave / WP;
    constexpr int TC = DUAL ? BP / 2 : BP;  // output columns of a tile
    const int tr = (a.R + BQ - 1) / BQ, tc = (a.C + TC - 1) / TC;
    int tile_r, tile_c;
    xcd_tile(blockIdx.x, tr, tc, 4, tile_r, tile_c);
    const int r0 = tile_r * BQ, c0 = tile_c * TC;
    const int kt0 = blockIdx.y * a.per;
    const int kt1 = min(a.nseg * a.nks, kt0 + a.per);
    const Copies cp(a, wave, lane);

    FfnSource<PSTR> src_p[DUAL ? 2 : 1];
    FfnSource<QSTR> src_q;
    const uint32_t ldp = (uint32_t)a.ldp, ldq = (uint32_t)a.ldq;
    int left;  // stages of the segment from the next copies' on
    auto seek = [&](int seg, int n) __attribute__((always_inline)) {
#pragma unroll
        for (int h = 0; h < (DUAL ? 2 : 1); ++h) {
            src_p[h].set(a.P[DUAL ? h : seg], ldp, c0, a.C, a.klen, FP8 ? 1 : 2, cp.vp, cp.chp);
            src_p[h].skip(n, ldp, c0, cp.chp);
        }
        src_q.set(a.Q[seg], ldq, r0, a.R, a.klen, FP8 ? 1 : 2, cp.vq, cp.chq);
        src_q.skip(n, ldq, r0, cp.chq);
        left = a.nks - n;
    };
    const uint32_t to = __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)ring + wave * 1024);
    // this wave's copies of the next stage, into slot `s`
    auto issue = [&](int s) __attribute__((always_inline)) {
        const uint32_t at = to + (uint32_t)s * SLOT;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
#pragma unroll
            for (int i = 0; i < SP::LD; ++i)
                dma16(src_p[DUAL ? h : 0].v + cp.shift_p(h, i), src_p[DUAL ? h : 0].rs,
                      at + h * SP::HB + i * (WAVES * 1024));
#pragma unroll
            for (int i = 0; i < SQ::LD; ++i)
                dma16(src_q.v + cp.shift_q(h, i), src_q.rs,
                      at + 2 * SP::HB + h * SQ::HB + i * (WAVES * 1024));
        }
        if (SEGS && --left == 0) {
            seek(1, 0);
            return;
        }
#pragma unroll
        for (int h = 0; h < (DUAL ? 2 : 1); ++h)
            src_p[h].next(ldp, c0, cp.chp);
        src_q.next(ldq, r0, cp.chq);
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
                ffn_frag<SP, PSTR>(sp + h * SP::HB, wp, j, lane, fp[set][h][j]);
#pragma unroll
            for (int i = 0; i < SQ::NB; ++i)
                ffn_frag<SQ, QSTR>(sp + 2 * SP::HB + h * SQ::HB, wq, i, lane, fq[set][h][i]);
        }
    };
    using I0 = std::integral_constant<int, 0>;
    using I1 = std::integral_constant<int, 1>;
    if (kt0 < kt1) {  // (the same for every wave)
        if (SEGS && kt0 >= a.nks)
            seek(1, kt0 - a.nks);
        else
            seek(0, kt0);
        const int n = kt1 - kt0;
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
                                ffn_mfma<FP8>(fp[set][h][j], fq[set][q][i], acc[h][j][q][i]);
        };
        for (int k = 0; k < n; k += 2) {
            stage(I0{}, I1{}, k);
            if (k + 1 < n)
                stage(I1{}, I0{}, k + 1);
        }
    }
    ffn_finish<SP, SQ, DUAL, EPI>(a, acc, c0, r0, tile_r, wp, wq, WQ, lane);
}

}  // namespace qll
