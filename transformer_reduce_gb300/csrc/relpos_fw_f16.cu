// relpos_fw_f16.cu -- softmax with a relative position bias, forward, __half storage.
#include "relpos_dispatch.cuh"

namespace lsr {
LSR_RELPOS_FW_INSTANTIATE(__half)
}  // namespace lsr
