// diff_bw_f16.cu -- difference of two softmax maps, backward, __half storage.
#include "diff_dispatch.cuh"

namespace lsr {
LSR_DIFF_BW_INSTANTIATE(__half)
}  // namespace lsr
