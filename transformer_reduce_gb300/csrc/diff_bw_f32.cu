// diff_bw_f32.cu -- difference of two softmax maps, backward, float storage.
#include "diff_dispatch.cuh"

namespace lsr {
LSR_DIFF_BW_INSTANTIATE(float)
}  // namespace lsr
