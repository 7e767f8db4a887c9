// Tile shapes of the feed-forward products and the rule that picks one.
#pragma once

#include "ffn_alt.h"

namespace qll {

// 0: 256x256 over 8 waves, 1: 128x128 over 4, 2: 64x64 over 4.
constexpr int kFfnTile[3] = {256, 128, 64};
constexpr int kFfnWaveRows[3] = {2, 2, 2};  // waves along the output's rows

int ffn_tile_pick(int64_t R, int64_t C, int epi);

template <bool FP8, int LAY, int EPI>
hipError_t ffn_launch_tile(int tile, const FfnArgs& a, hipStream_t stream)
{
    constexpr bool DUAL = EPI == EPI_GATED || EPI == EPI_DGATED;
    const int B = kFfnTile[tile];
    const int64_t tiles = (int64_t)((a.R + B - 1) / B) * ((a.C + (DUAL ? B / 2 : B) - 1) / (DUAL ? B / 2 : B));
    const dim3 grid((unsigned)tiles, (unsigned)a.splits);
    if constexpr (EPI != EPI_PARTIAL) {  // (only the smallest tile splits K)
        if (tile == 0) {
            // one workgroup per CU
            ffn_alt_kernel<FP8, LAY, EPI>
                <<<(unsigned)(tiles < 256 ? tiles : 256), 512, 0, stream>>>(a);
            return hipGetLastError();
        }
    }
    if (tile == 1)
        ffn_ring_kernel<FP8, LAY, EPI, 128, 128, 2, 2, 2><<<grid, 256, 0, stream>>>(a);
    else
        ffn_ring_kernel<FP8, LAY, EPI, 64, 64, 2, 2, 4><<<grid, 256, 0, stream>>>(a);
    return hipGetLastError();
}

}  // namespace qll
