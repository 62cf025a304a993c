// relpos_fw_bf16.cu -- softmax with a relative position bias, forward, __nv_bfloat16 storage.
#include "relpos_dispatch.cuh"

namespace lsr {
LSR_RELPOS_FW_INSTANTIATE(__nv_bfloat16)
}  // namespace lsr
