// relpos_bw_f16.cu -- softmax with a relative position bias, backward, __half storage.
#include "relpos_dispatch.cuh"

namespace lsr {
LSR_RELPOS_BW_INSTANTIATE(__half)
}  // namespace lsr
