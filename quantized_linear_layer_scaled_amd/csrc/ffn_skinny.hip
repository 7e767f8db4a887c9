// Kernels for few rows, and the launches of the feed-forward products.
#include "ffn_skinny.h"

#include "ffn_launch.h"

namespace qll {

hipError_t ffn_launch_nt_fp8(int, int, const FfnArgs&, hipStream_t);
hipError_t ffn_launch_nt_bf16(int, int, const FfnArgs&, hipStream_t);
hipError_t ffn_launch_nt_grad(int, int, const FfnArgs&, hipStream_t);
hipError_t ffn_launch_nn(int, int, const FfnArgs&, hipStream_t);
hipError_t ffn_launch_tn(int, int, const FfnArgs&, hipStream_t);

// The largest tile that still gives every compute unit one.
int ffn_tile_pick(int64_t R, int64_t C, int epi)
{
    const bool dual = epi == EPI_GATED || epi == EPI_DGATED;
    for (int t = 0; t < 2; ++t) {
        const int64_t B = kFfnTile[t], TC = dual ? B / 2 : B;
        if (((R + B - 1) / B) * ((C + TC - 1) / TC) >= 256)
            return t;
    }
    return 2;
}

int ffn_dz_strips(int64_t R, int64_t C)
{
    const int t = ffn_tile_pick(R, C, EPI_DZ);
    return (int)((R + kFfnTile[t] - 1) / kFfnTile[t]) * kFfnWaveRows[t];
}

int ffn_splits(int64_t R, int64_t C, int64_t stages)
{
    const int t = ffn_tile_pick(R, C, EPI_LINEAR);
    const int64_t B = kFfnTile[t];
    const int64_t tiles = ((R + B - 1) / B) * ((C + B - 1) / B);
    if (t != 2 || tiles >= 256 || stages < 16)
        return 1;
    int64_t s = 512 / tiles;
    s = s < stages / 8 ? s : stages / 8;
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
