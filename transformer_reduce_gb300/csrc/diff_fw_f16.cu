// diff_fw_f16.cu -- difference of two softmax maps, forward, __half storage.
#include "diff_dispatch.cuh"

namespace lsr {
LSR_DIFF_FW_INSTANTIATE(__half)
}  // namespace lsr
