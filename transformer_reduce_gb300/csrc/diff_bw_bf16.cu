// diff_bw_bf16.cu -- difference of two softmax maps, backward, __nv_bfloat16 storage.
#include "diff_dispatch.cuh"

namespace lsr {
LSR_DIFF_BW_INSTANTIATE(__nv_bfloat16)
}  // namespace lsr
