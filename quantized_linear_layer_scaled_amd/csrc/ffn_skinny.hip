// Kernels for few rows, and the launches of the feed-forward products.
#include "ffn_skinny.h"

#include "ffn_launch.h"

namespace qll {

hipError_t ffn_launch_nt_fp8(int, int, const FfnArgs&, hipStream_t);
hipError_t ffn_launch_nt_bf16(int, int, const FfnArgs&, hipStream_t);
hipError_t ffn_launch_nt_grad(int, int, const FfnArgs&, hipStream_t);
hipError_t ffn_launch_nn(int, int, const FfnArgs&, hipStream_t);
hipError_t ffn_launch_tn(int, int, const FfnArgs&, hipStream_t);

// Measured per call (us): the 256x256 tile against the 128x128 ones, gated FP8
// M = 1024, N = 6144, K = 2048 (192 tiles of the 256 CUs): 28.8 / 36.1; FP8
// M = 2048, N = 4096, K = 12288 (128 tiles): 105 / 90.  128x128 over 4 waves,
// two workgroups per CU, against 8 waves and a deeper ring: bf16 M = 1024,
// N = K = 4096 (256 tiles) 49.7 / 44.5; gated bf16 M = 300, N = 6144, K = 2048
// (288 tiles) 29.3 / 42.1.  128x128 against 64x64: M = 512, N = 4096, K = 2048
// (128 tiles) 25.7 / 20.5; FP8 M = 1024, N = K = 4096 (256 tiles) 25.8 / 34.3.
int ffn_tile_pick(int64_t R, int64_t C, int epi)
{
    if (ffn_tiles(0, R, C, epi) >= 176)
        return 0;
    const int64_t n = ffn_tiles(1, R, C, epi);
    return n > 256 ? 1 : (n >= 192 ? 2 : kFfnSmallest);
}

int ffn_dz_strips(int64_t R, int64_t C)
{
    const FfnTile& t = kFfnTiles[ffn_tile_pick(R, C, EPI_DZ)];
    return (int)((R + t.rows - 1) / t.rows) * t.wave_rows;
}

// Split-K: at most one workgroup per CU and at least 12 stages each.  Unsplit,
// this many pieces (in brackets) and more (us): bf16 M = 64, N = 4096,
// K = 12288 65.6, 26.2 (4), 28.9 with eight; FP8 the same 33.1, 16.8 (4), 19.3;
// bf16 M = 128, N = 4096, K = 2048 14.6, 13.7 (2), 15.1 with four.  Where the
// tiles are as many as the CUs, pieces write more than they gain: FP8 M = 512,
// N = 2048, K = 6144 19.9, 23.1 with three; bf16 M = 512, N = K = 2048 15.2,
// 18.0 with two (long bf16 products gain there: M = 512, N = 2048, K = 6144
// 33.9, 29.0 with two; FP8 M = 256, N = 4096, K = 12288 loses, 34.8, 37.4).
int ffn_splits(int64_t R, int64_t C, int64_t stages)
{
    const int64_t tiles = ffn_tiles(kFfnSmallest, R, C, EPI_LINEAR);
    if (tiles == 0 || ffn_tile_pick(R, C, EPI_LINEAR) != kFfnSmallest)
        return 1;
    const int64_t by_tiles = 256 / tiles;
    const int64_t s = by_tiles < stages / 12 ? by_tiles : stages / 12;
    return (int)(s < 1 ? 1 : (s > 32 ? 32 : s));
}

hipError_t ffn_launch(int fp8, int layout, int epi, FfnArgs a, hipStream_t stream)
{
    const int tile = ffn_tile_pick(a.R, a.C, epi);
    const int total = a.nseg * a.nks;
    a.per = a.splits > 1 ? (total + a.splits - 1) / a.splits : total;
    const int e = a.splits > 1 ? (int)EPI_PARTIAL : epi;
    hipError_t rc;
    if (layout == LAY_NN)
        rc = ffn_launch_nn(tile, e, a, stream);
    else if (layout == LAY_TN)
        rc = ffn_launch_tn(tile, e, a, stream);
    else if (fp8)
        rc = ffn_launch_nt_fp8(tile, e, a, stream);
    else if (epi == EPI_DZ || epi == EPI_DGATED)
        rc = ffn_launch_nt_grad(tile, e, a, stream);
    else
        rc = ffn_launch_nt_bf16(tile, e, a, stream);
    if (rc != hipSuccess || a.splits == 1)
        return rc;
    return ffn_launch_reduce(a, stream);
}

// Up to 16 rows: this kernel / the tile (us, weights from HBM) at 1, 8 and 16
// rows.  Linear bf16 N = 2048, K = 6144 10.8, 11.1, 12.0 / 12.0, 12.7, 12.9; FP8
// the same 7.1, 7.2, 7.6 / 10.6, 11.0, 10.9; bf16 N = 12288, K = 4096 22.4, 22.3,
// 27.5 / 26.1, 25.0, 25.0; FP8 the same 13.6, 13.8, 15.5 / 15.1, 15.2, 15.3.
// Gated bf16 N = 2048, K = 6144 12.8, 13.3, 14.5 / 33.6, 33.8, 33.8; N = 4096,
// K = 12288 38.4, 44.6, 55.3 / 64.4, 64.6, 64.8; FP8 N = 4096, K = 2048 5.8, 6.5,
// 7.5 / 8.4, 8.4, 8.4.  It loses only near 16 rows with many weights, most for
// gated N = 12288, K = 4096: bf16 38.0, 41.4, 52.8 / 44.1, 44.3, 44.4, FP8 19.1,
// 22.6, 27.6 / 24.2, 24.3, 24.6.
// From 17 rows on a workgroup here re-reads the tokens for every 8 or 16
// columns, and the 64x64 tile for every 64 (gated 32), so the tile wins once the
// weights are many.  Measured, this kernel / the tile (us) at 17 and 32 rows:
// linear FP8 N = 4096, K = 2048 (8 MB) 5.4 / 9.0, 6.0 / 8.9; bf16 the same (17
// MB) 8.1 / 11.6, 8.7 / 11.7; FP8 N = 2048, K = 6144 (13 MB) 8.2 / 11.6, 10.1 /
// 12.0; bf16 the same (25 MB) 14.1 / 12.4, 17.1 / 13.4; FP8 N = 4096, K = 12288
// (50 MB) 15.3 / 15.4, 19.2 / 15.4; bf16 N = 12288, K = 4096 28.0 / 23.7, 35.1 /
// 23.9.  The gated tile does not split K, so its time goes with K alone until
// its tiles fill the chip, and the columns decide: bf16 N = 2048, K = 6144 15.3
// / 34.0, 19.0 / 34.1; N = 4096, K = 2048 11.2 / 13.7, 14.1 / 14.0; N = 12288,
// K = 4096 50.2 / 38.8, 66.0 / 38.6.  (Past 2^25 columns 512 threads for each 8
// or 16 of them would be more than a launch holds; the tiles are walked over.)
bool ffn_skinny_fits(int epi, int64_t R, int64_t C, int64_t kbytes)
{
    if (C > (int64_t{1} << 25))
        return false;
    if (R <= 16 || R > 32)
        return R <= 16;
    return epi == EPI_GATED ? C <= 4096 : C * kbytes <= (int64_t{1} << 24);
}

namespace {

template <bool FP8, int EPI, int COLS>
hipError_t skinny(const FfnArgs& a, hipStream_t stream)
{
    const unsigned grid = (unsigned)((a.C + COLS - 1) / COLS);
    if (a.R <= 16)
        ffn_skinny_kernel<FP8, EPI, COLS, 1, 8><<<grid, 512, 0, stream>>>(a);
    else
        ffn_skinny_kernel<FP8, EPI, COLS, 2, 8><<<grid, 512, 0, stream>>>(a);
    return hipGetLastError();
}

// Linear: 8 columns per workgroup below 16 for every compute unit (N = 2048,
// K = 6144, M = 4: 8.9 against 10.5 us with 16; N = 4096, K = 2048: 5.7 either
// way).
template <bool FP8>
hipError_t skinny_epi(int epi, const FfnArgs& a, hipStream_t stream)
{
    if (epi == EPI_GATED)
        return skinny<FP8, EPI_GATED, 8>(a, stream);
    if (a.C < 256 * 16)
        return skinny<FP8, EPI_LINEAR, 8>(a, stream);
    return skinny<FP8, EPI_LINEAR, 16>(a, stream);
}

}  // namespace

hipError_t ffn_launch_skinny(int fp8, int epi, const FfnArgs& a, hipStream_t stream)
{
    return fp8 ? skinny_epi<true>(epi, a, stream) : skinny_epi<false>(epi, a, stream);
}

}  // namespace qll
