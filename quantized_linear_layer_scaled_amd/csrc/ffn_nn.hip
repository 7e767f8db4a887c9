// bf16 products with a K-strided weight operand (gradient of the input).
#include "ffn_launch.h"

namespace qll {

hipError_t ffn_launch_nn(int tile, int epi, const FfnArgs& a, hipStream_t stream)
{
    if (epi == EPI_PLAIN)
        return ffn_launch_tile<false, LAY_NN, EPI_PLAIN>(tile, a, stream);
    return ffn_launch_tile<false, LAY_NN, EPI_PARTIAL>(tile, a, stream);
}

}  // namespace qll
