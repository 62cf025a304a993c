// block_norm_bw_bf16.cu -- norms around a block, backward, __nv_bfloat16 storage.
#include "block_norm_dispatch.cuh"

namespace lsr {
LSR_BN_BW_INSTANTIATE(__nv_bfloat16)
}  // namespace lsr
