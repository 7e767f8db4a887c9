// bf16 feed-forward products, forward (both operands K-contiguous).
#include "ffn_launch.h"

namespace qll {

hipError_t ffn_launch_nt_bf16(int tile, int epi, const FfnArgs& a, hipStream_t stream)
{
    switch (epi) {
    case EPI_LINEAR: return ffn_launch_tile<false, LAY_NT, EPI_LINEAR>(tile, a, stream);
    case EPI_GATED: return ffn_launch_tile<false, LAY_NT, EPI_GATED>(tile, a, stream);
    default: return ffn_launch_tile<false, LAY_NT, EPI_PARTIAL>(tile, a, stream);
    }
}

}  // namespace qll
