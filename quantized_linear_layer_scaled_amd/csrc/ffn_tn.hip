// bf16 products with two K-strided operands (gradient of the weights).
#include "ffn_launch.h"

namespace qll {

hipError_t ffn_launch_tn(int tile, int epi, const FfnArgs& a, hipStream_t stream)
{
    if (epi == EPI_PLAIN)
        return ffn_launch_tile<false, LAY_TN, EPI_PLAIN>(tile, a, stream);
    return ffn_launch_tile<false, LAY_TN, EPI_PARTIAL>(tile, a, stream);
}

}  // namespace qll
