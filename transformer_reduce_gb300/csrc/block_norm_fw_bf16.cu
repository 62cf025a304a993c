// block_norm_fw_bf16.cu -- norms around a block, forward, __nv_bfloat16 storage.
#include "block_norm_dispatch.cuh"

namespace lsr {
LSR_BN_FW_INSTANTIATE(__nv_bfloat16)
}  // namespace lsr
