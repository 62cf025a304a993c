// block_norm_fw_f32.cu -- norms around a block, forward, float storage.
#include "block_norm_dispatch.cuh"

namespace lsr {
LSR_BN_FW_INSTANTIATE(float)
}  // namespace lsr
