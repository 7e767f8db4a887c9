// The 256x256 tile of the feed-forward products: eight waves in two groups
// that alternate between the matrix cores and everything else.
//
// Waves w and w + 4 share a SIMD.  Group 0 (waves 0-3) and group 1 (4-7) run
// the same sequence of phases, one barrier apart: while one group's waves
// issue matrix instructions (and, among them, copies), the other's read
// fragments from LDS, and at the next barrier they trade places.  A phase is one quadrant
// (P half x Q half) of the wave's 64 x 128 share over one stage, 16 bf16 (or
// 8 e4m3) instructions, 256 cycles:
//
//   phase   fragments read      copy started (2 per wave)   product
//   0       Q0                  P0 of stage k + 2           P0 x Q0
//   1       P1                  Q0 of stage k + 2           P1 x Q0
//   2       Q1                  P1 of stage k + 2           P0 x Q1
//   3       P0 of stage k + 1   Q1 of stage k + 2           P1 x Q1
//
// The two LDS slots hold stages k and k + 1; a half of stage k is overwritten
// one phase after it was read (every wave waits for its reads before the
// barrier that ends a read segment, and both groups have passed one by the
// time either starts the copy).  At the end of the read segment before the
// one that reads a half, five younger copies of two instructions are in
// flight: s_waitcnt vmcnt(10) before that segment's barrier.  So a copy has
// about six phases (3000 cycles) to land.  Copies past the last
// stage are started all the same, which keeps that count; they read in range
// or zeros, into slots nobody reads, and the kernel waits for them at the end
// of the tile.
//
// One workgroup per CU walks over tiles blockIdx.x, + gridDim.x, ... (a
// multiple of 8 workgroups, so each keeps to its XCD's tiles).  The epilogue
// uses no LDS, so the next tile's first two stages are copied while it runs.
//
// Measured (M = 8192, N = 12288, K = 4096, bf16, one product; in brackets the
// same with zeros for inputs, where the clock does not drop): 552 us = 1.49
// PFLOP/s (458); 536 (413) without the epilogue, and no less than that
// without the copies or without the fragment reads.  Copies in the read
// segments instead: 577 us.  Copies spread over the product segment by wave,
// a branch per block: 700.  One stream per wave with reads, copies and
// products interleaved, two barriers per stage: 575.  s_setprio around the
// products: 580.  A fragment layout with two LDS passes per read: 640.  So
// the matrix cores, at the clock they hold under load, bound long products;
// short ones (K = 2048, one tile per CU) also pay the first copies and the
// last stores, which all compute units issue at once.  Tiles of 128 x 256 in
// the same scheme (two or three LDS slots): within 5% of the 128x128 tiles
// of the ring either way, not kept.
#pragma once

#include "ffn_tile.h"

namespace qll {

// The two slots, one object for every product of a kernel.
__device__ __forceinline__ uint8_t* ffn_alt_ring()
{
    __shared__ __attribute__((aligned(1024))) uint8_t ring[2 * 512 * 128];
    return ring;
}

// Where the tiles of a product lie: how many there are, the arguments and the
// corner of tile t, and, with GATHER, the offsets in Q[0] of a tile's rows.
// (an offset out of range stays there)
__device__ __forceinline__ uint32_t gathered(uint32_t in_row, uint32_t row)
{
    return (in_row | row) & kOutOfRange ? kOutOfRange : in_row + row;
}
template <int TC>
struct FfnDense {
    static constexpr bool GATHER = false;
    int tr, tc;
    __device__ __forceinline__ explicit FfnDense(const FfnArgs& a)
        : tr((a.R + 255) / 256), tc((a.C + TC - 1) / TC)
    {
    }
    __device__ __forceinline__ int tiles() const { return tr * tc; }
    __device__ __forceinline__ void at(int t, FfnArgs&, int& r0, int& c0) const
    {
        int tile_r, tile_c;
        xcd_tile(t, tr, tc, 4, tile_r, tile_c);
        r0 = tile_r * 256;
        c0 = tile_c * TC;
    }
};

// Tiles first, first + step, ... of one product.
template <bool FP8, int LAY, int EPI, typename WHERE>
__device__ __forceinline__ void ffn_alt_tiles(const FfnArgs& args, const WHERE& where, int first,
                                              int step)
{
    constexpr bool DUAL = EPI == EPI_GATED || EPI == EPI_DGATED || EPI == EPI_GROUPED;
    constexpr bool GATHER = WHERE::GATHER;
    FfnArgs a = args;  // of the tile whose copies are being started
    using Copies = FfnCopies<FP8, LAY, DUAL, 256, 256, 4, 2>;
    using SP = typename Copies::SP;
    using SQ = typename Copies::SQ;
    constexpr bool PSTR = Copies::PSTR, QSTR = Copies::QSTR;
    constexpr bool SEGS = LAY == LAY_NN;
    constexpr int SLOT = Copies::SLOT;
    uint8_t* const ring = ffn_alt_ring();

    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wp = wave & 3, wq = wave >> 2;  // (wq is the group)
    const int nk = a.nseg * a.nks;
    const Copies cp(args, wave, lane);
    int c0, r0;  // corner of the tile whose copies are being started

    v4f acc[2][SP::NB][2][SQ::NB];

    // sources of the next copies
    FfnSource<PSTR> src_p[DUAL ? 2 : 1];
    FfnSource<QSTR> src_q;
    uint32_t row_q[GATHER ? 2 : 1][GATHER ? SQ::LD : 1];  // GATHER: the rows' offsets
    const uint32_t ldp = (uint32_t)a.ldp, ldq = (uint32_t)a.ldq;
    int kp = 0, kq = 0;
    auto set_p = [&](int seg) __attribute__((always_inline)) {
#pragma unroll
        for (int h = 0; h < (DUAL ? 2 : 1); ++h)
            src_p[h].set(a.P[DUAL ? h : seg], ldp, c0, a.C, a.klen, FP8 ? 1 : 2, cp.vp, cp.chp);
    };
    auto set_q = [&](int seg) __attribute__((always_inline)) {
        if constexpr (GATHER) {
            // the offset within a row moves on with the stages, as for
            // contiguous rows
            where.rows(a, r0, src_q.rs);
            src_q.v = cp.chq * 16;
            src_q.kleft = a.klen;
            src_q.clip(cp.chq);
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int i = 0; i < SQ::LD; ++i) {
                    int line, ch;
                    SQ::source(i, wave, lane, line, ch);
                    row_q[h][i] = where.row(a, r0, ffn_tile_row<SQ, false>(h, line));
                }
            return;
        }
        src_q.set(a.Q[seg], ldq, r0, a.R, a.klen, FP8 ? 1 : 2, cp.vq, cp.chq);
    };
    // (only the input gradient has a second segment)
    auto next_p = [&]() __attribute__((always_inline)) {
        if (SEGS && ++kp == a.nks) {
            set_p(1);
            return;
        }
#pragma unroll
        for (int h = 0; h < (DUAL ? 2 : 1); ++h)
            src_p[h].next(ldp, c0, cp.chp);
    };
    auto next_q = [&]() __attribute__((always_inline)) {
        if (SEGS && ++kq == a.nks) {
            set_q(1);
            return;
        }
        src_q.next(ldq, r0, cp.chq);
    };
    // copy i (of 2) of a half; `to`: where this wave's 1 KiB of a copy go
    const uint32_t to = __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)ring + wave * 1024);
    auto copy_p = [&](int h, int i, uint8_t* slot) __attribute__((always_inline)) {
        dma16(src_p[DUAL ? h : 0].v + cp.shift_p(h, i), src_p[DUAL ? h : 0].rs,
              to + (uint32_t)(slot - ring) + h * SP::HB + i * 8192);
    };
    auto copy_q = [&](int h, int i, uint8_t* slot) __attribute__((always_inline)) {
        uint32_t v;
        if constexpr (GATHER)
            v = gathered(src_q.v, row_q[h][i]);
        else
            v = src_q.v + cp.shift_q(h, i);
        dma16(v, src_q.rs, to + (uint32_t)(slot - ring) + 2 * SP::HB + h * SQ::HB + i * 8192);
    };

    uint4 fp[2][SP::NB][2], fq[SQ::NB][2];
    auto read_p = [&](int h, const uint8_t* slot) __attribute__((always_inline)) {
#pragma unroll
        for (int j = 0; j < SP::NB; ++j)
            ffn_frag<SP, PSTR>(slot + h * SP::HB, wp, j, lane, fp[h][j]);
    };
    auto read_q = [&](int h, const uint8_t* slot) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < SQ::NB; ++i)
            ffn_frag<SQ, QSTR>(slot + 2 * SP::HB + h * SQ::HB, wq, i, lane, fq[i]);
    };
    // ends a read segment: the wave's reads are back, the copies that the
    // next segment reads have landed
    auto end_read = [&]() __attribute__((always_inline)) {
        wait_vm_barrier<10>();
        __builtin_amdgcn_sched_barrier(0);
    };
    // a quadrant's products; the two copies copy(0), copy(1) go out among them
    auto product = [&](int h, int q, auto&& copy) __attribute__((always_inline)) {
#pragma unroll
        for (int j = 0; j < SP::NB; ++j)
#pragma unroll
            for (int i = 0; i < SQ::NB; ++i) {
                acc[h][j][q][i] = ffn_mfma<FP8>(fp[h][j], fq[i], acc[h][j][q][i]);
                const int n = j * SQ::NB + i;
                __builtin_amdgcn_sched_barrier(0);
                if (n == 1 || n == 4)
                    copy(n == 1 ? 0 : 1);
                __builtin_amdgcn_sched_barrier(0);
            }
        __builtin_amdgcn_sched_barrier(0);
        asm volatile("s_barrier" ::: "memory");
        __builtin_amdgcn_sched_barrier(0);
    };
    auto stage = [&](uint8_t* slot, uint8_t* other) __attribute__((always_inline)) {
        read_q(0, slot);
        end_read();
        product(0, 0, [&](int i) __attribute__((always_inline)) { copy_p(0, i, slot); });
        read_p(1, slot);
        end_read();
        product(1, 0, [&](int i) __attribute__((always_inline)) { copy_q(0, i, slot); });
        read_q(1, slot);
        end_read();
        product(0, 1, [&](int i) __attribute__((always_inline)) { copy_p(1, i, slot); });
        next_p();
        read_p(0, other);
        end_read();
        product(1, 1, [&](int i) __attribute__((always_inline)) { copy_q(1, i, slot); });
        next_q();
    };

    // the first two stages of tile t
    auto start = [&](int t) __attribute__((always_inline)) {
        where.at(t, a, r0, c0);
        kp = kq = 0;
        set_p(0);
        set_q(0);
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            uint8_t* slot = ring + s * SLOT;
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    copy_p(h, i, slot);
                    copy_q(h, i, slot);
                }
            next_p();
            next_q();
        }
    };

    const int tiles = where.tiles();
    if (first >= tiles)
        return;
    start(first);
    for (int t = first; t < tiles; t += step) {
        const int rt = r0, ct = c0;
        const FfnArgs at = a;
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int j = 0; j < SP::NB; ++j)
#pragma unroll
                for (int q = 0; q < 2; ++q)
#pragma unroll
                    for (int i = 0; i < SQ::NB; ++i)
                        acc[h][j][q][i] = v4f{0, 0, 0, 0};
        // the copies have landed, and so have the stores of the tile before
        // (they share the counter)
        wait_vm_barrier<0>();
        __builtin_amdgcn_sched_barrier(0);
        read_p(0, ring);
        end_read();
        if (wq == 1)
            asm volatile("s_barrier" ::: "memory");
        for (int kt = 0; kt < nk; kt += 2) {
            stage(ring, ring + SLOT);
            if (kt + 1 < nk)
                stage(ring + SLOT, ring);
        }
        if (wq == 0)
            asm volatile("s_barrier" ::: "memory");
        // Copies started past the last stage still write this LDS.  Then the
        // next tile's first stages travel while this one's epilogue runs.
        wait_vm_barrier<0>();
        __builtin_amdgcn_sched_barrier(0);
        if (t + step < tiles)
            start(t + step);
        ffn_finish<SP, SQ, DUAL, EPI>(at, acc, ct, rt, rt / 256, wp, wq, 2, lane);
    }
}

template <bool FP8, int LAY, int EPI>
__global__ __launch_bounds__(512, 2) void ffn_alt_kernel(FfnArgs a)
{
    constexpr int TC = EPI == EPI_GATED || EPI == EPI_DGATED ? 128 : 256;
    ffn_alt_tiles<FP8, LAY, EPI>(a, FfnDense<TC>(a), blockIdx.x, gridDim.x);
}

// Two products in one launch, the input's and the weights' gradients of a
// backward pass: their tiles are numbered one after the other, so that they
// fill the compute units together where neither does alone.  (Template only
// so that every unit that includes this may define it.)
template <int LAY_A, int LAY_B>
__global__ __launch_bounds__(512, 2) void ffn_alt_pair_kernel(FfnArgs a, FfnArgs b)
{
    const int tiles_a = ((a.R + 255) / 256) * ((a.C + 255) / 256);
    const int G = gridDim.x;
    ffn_alt_tiles<false, LAY_A, EPI_PLAIN>(a, FfnDense<256>(a), blockIdx.x, G);
    // the first tile of b whose number, after a's, is this workgroup's
    const int skip = tiles_a % G;
    const int first = (int)blockIdx.x - skip;
    __syncthreads();
    ffn_alt_tiles<false, LAY_B, EPI_PLAIN>(b, FfnDense<256>(b), first < 0 ? first + G : first, G);
}

}  // namespace qll
