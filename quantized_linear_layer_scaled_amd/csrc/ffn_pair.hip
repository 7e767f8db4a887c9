// The two gradient products of a backward pass in one launch.
#include "ffn_launch.h"

namespace qll {

// Both on the 256x256 tile, together: where that fills the compute units and
// no single tile outlasts the average share of the work (by a quarter at
// most).  The whole backward pass with M = N = 4096, K = 2048 (128 tiles of 64
// stages each; alone each runs on 128x128 tiles): 185 us, 204 in two launches.
// M = 8192, N = 12288, K = 4096 gated (512 tiles of 384 stages, 1536 of 128):
// 3505, 3500 in two.
bool ffn_pair_fits(const FfnArgs& in, const FfnArgs& w)
{
    const int64_t ta = ffn_tiles(0, in.R, in.C, EPI_PLAIN), tb = ffn_tiles(0, w.R, w.C, EPI_PLAIN);
    const int64_t sa = (int64_t)in.nseg * in.nks, sb = w.nks;
    const int64_t longest = sa > sb ? sa : sb;
    return ta + tb >= 176 && longest * 256 * 4 <= (ta * sa + tb * sb) * 5;
}

hipError_t ffn_launch_pair(const FfnArgs& in, const FfnArgs& w, hipStream_t stream)
{
    const int64_t tiles = ffn_tiles(0, in.R, in.C, EPI_PLAIN) + ffn_tiles(0, w.R, w.C, EPI_PLAIN);
    ffn_alt_pair_kernel<LAY_NN, LAY_TN>
        <<<(unsigned)(tiles < 256 ? tiles : 256), 512, 0, stream>>>(in, w);
    return hipGetLastError();
}

}  // namespace qll
