// qk_norm_rope_bf16.cu -- per-head query / key norm with rotation, __nv_bfloat16 storage.
#include "qk_dispatch.cuh"

namespace lsr {
LSR_QK_INSTANTIATE(__nv_bfloat16)
}  // namespace lsr
