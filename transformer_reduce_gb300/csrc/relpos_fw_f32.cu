// relpos_fw_f32.cu -- softmax with a relative position bias, forward, float storage.
#include "relpos_dispatch.cuh"

namespace lsr {
LSR_RELPOS_FW_INSTANTIATE(float)
}  // namespace lsr
