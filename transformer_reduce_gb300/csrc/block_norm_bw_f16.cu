// block_norm_bw_f16.cu -- norms around a block, backward, __half storage.
#include "block_norm_dispatch.cuh"

namespace lsr {
LSR_BN_BW_INSTANTIATE(__half)
}  // namespace lsr
