// block_norm_bw_f32.cu -- norms around a block, backward, float storage.
#include "block_norm_dispatch.cuh"

namespace lsr {
LSR_BN_BW_INSTANTIATE(float)
}  // namespace lsr
