// relpos_f16.cu -- softmax with a relative position bias, __half storage.
#include "relpos_dispatch.cuh"

namespace lsr {
LSR_RELPOS_INSTANTIATE(__half)
}  // namespace lsr
