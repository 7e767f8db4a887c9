// bf16 feed-forward products of the backward passes that compute the forward
// sums again and turn them into the gradients of the pre-activations.
#include "ffn_launch.h"

namespace qll {

hipError_t ffn_launch_nt_grad(int tile, int epi, const FfnArgs& a, hipStream_t stream)
{
    if (epi == EPI_DZ)
        return ffn_launch_tile<false, LAY_NT, EPI_DZ>(tile, a, stream);
    return ffn_launch_tile<false, LAY_NT, EPI_DGATED>(tile, a, stream);
}

}  // namespace qll
