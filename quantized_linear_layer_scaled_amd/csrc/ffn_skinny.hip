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
// M = 1024, N = 6144, K = 2048 (192 tiles of the 256 CUs): 28 / 36; FP8
// M = 2048, N = 4096, K = 12288 (128 tiles): 121 / 97.  128x128 over 4 waves,
// two workgroups per CU, against 8 waves and a deeper ring: bf16 M = 1024,
// N = K = 4096 (256 tiles) 55.7 / 46.8; gated bf16 M = 300, N = 6144, K = 2048
// (288 tiles) 30.2 / 48.5.  128x128 against 64x64: M = 512, N = 4096, K = 2048
// (128 tiles) 26.1 / 23.3.
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

// Split-K: about three workgroups per CU, of at least 16 stages each (input
// gradient M = 512, N = 6144, K = 2048: 43 us unsplit, 36 with two pieces, 37
// with four; M = 256, N = 2048, K = 6144: 44, 28, 23).
int ffn_splits(int64_t R, int64_t C, int64_t stages)
{
    const int64_t tiles = ffn_tiles(kFfnSmallest, R, C, EPI_LINEAR);
    if (tiles == 0 || ffn_tile_pick(R, C, EPI_LINEAR) != kFfnSmallest)
        return 1;
    const int64_t by_tiles = 768 / tiles;
    const int64_t s = by_tiles < stages / 16 ? by_tiles : stages / 16;
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

namespace {

template <bool FP8, int EPI, int COLS>
hipError_t skinny(const FfnArgs& a, hipStream_t stream)
{
    ffn_skinny_kernel<FP8, EPI, COLS, 8>
        <<<(unsigned)((a.C + COLS - 1) / COLS), 512, 0, stream>>>(a);
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
