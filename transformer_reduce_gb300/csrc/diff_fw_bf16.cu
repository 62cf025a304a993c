// diff_fw_bf16.cu -- difference of two softmax maps, forward, __nv_bfloat16 storage.
#include "diff_dispatch.cuh"

namespace lsr {
LSR_DIFF_FW_INSTANTIATE(__nv_bfloat16)
}  // namespace lsr
