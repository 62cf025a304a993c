// qk_norm_rope_f16.cu -- per-head query / key norm with rotation, __half storage.
#include "qk_dispatch.cuh"

namespace lsr {
LSR_QK_INSTANTIATE(__half)
}  // namespace lsr
