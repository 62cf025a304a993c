// relpos_bw_bf16.cu -- softmax with a relative position bias, backward, __nv_bfloat16 storage.
#include "relpos_dispatch.cuh"

namespace lsr {
LSR_RELPOS_BW_INSTANTIATE(__nv_bfloat16)
}  // namespace lsr
