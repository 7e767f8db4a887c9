// Tile shapes of the feed-forward products and the rule that picks one.
#pragma once

#include "ffn_alt.h"

namespace qll {

// Rows and columns of the tiles, and waves along the rows.
struct FfnTile {
    int rows, cols, wave_rows;
};
constexpr FfnTile kFfnTiles[] = {{256, 256, 2}, {128, 128, 2}, {128, 128, 4}, {64, 64, 2}};
constexpr int kFfnSmallest = 3;

inline int64_t ffn_tiles(int tile, int64_t R, int64_t C, int epi)
{
    const bool dual = epi == EPI_GATED || epi == EPI_DGATED;
    const int64_t TR = kFfnTiles[tile].rows, TC = kFfnTiles[tile].cols / (dual ? 2 : 1);
    return ((R + TR - 1) / TR) * ((C + TC - 1) / TC);
}

template <bool FP8, int LAY, int EPI>
hipError_t ffn_launch_tile(int tile, const FfnArgs& a, hipStream_t stream)
{
    const int64_t tiles = ffn_tiles(tile, a.R, a.C, EPI);
    if constexpr (EPI != EPI_PARTIAL) {  // (only the smallest tile splits K)
        switch (tile) {
        case 0:
            // one workgroup per CU
            ffn_alt_kernel<FP8, LAY, EPI>
                <<<(unsigned)(tiles < 256 ? tiles : 256), 512, 0, stream>>>(a);
            return hipGetLastError();
        case 1:
            // two workgroups per CU
            ffn_ring_kernel<FP8, LAY, EPI, 128, 128, 2, 2, 2>
                <<<(unsigned)tiles, 256, 0, stream>>>(a);
            return hipGetLastError();
        case 2:
            // one workgroup per CU, three stages of copies in flight
            ffn_ring_kernel<FP8, LAY, EPI, 128, 128, 2, 4, 4>
                <<<(unsigned)tiles, 512, 0, stream>>>(a);
            return hipGetLastError();
        }
    }
    ffn_ring_kernel<FP8, LAY, EPI, 64, 64, 2, 2, 4>
        <<<dim3((unsigned)tiles, (unsigned)a.splits), 256, 0, stream>>>(a);
    return hipGetLastError();
}

}  // namespace qll
