// qk_norm_rope_f32.cu -- per-head query / key norm with rotation, float storage.
#include "qk_dispatch.cuh"

namespace lsr {
int64_t qk_bw_parts(int64_t tokens, int64_t Hq, int64_t Hk) {
    return tokens > 0 && Hq + Hk > 0 ? kQkBwBlocks + 1 : 0;
}
LSR_QK_INSTANTIATE(float)
}  // namespace lsr
