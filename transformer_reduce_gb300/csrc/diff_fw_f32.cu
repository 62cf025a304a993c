// diff_fw_f32.cu -- difference of two softmax maps, forward, float storage.
#include "diff_dispatch.cuh"

namespace lsr {
LSR_DIFF_FW_INSTANTIATE(float)
}  // namespace lsr
