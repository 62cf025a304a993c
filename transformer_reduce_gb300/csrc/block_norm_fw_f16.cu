// block_norm_fw_f16.cu -- norms around a block, forward, __half storage.
#include "block_norm_dispatch.cuh"

namespace lsr {
LSR_BN_FW_INSTANTIATE(__half)
}  // namespace lsr
