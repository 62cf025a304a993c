// relpos_bw_f32.cu -- softmax with a relative position bias, backward, float storage.
#include "relpos_dispatch.cuh"

namespace lsr {
int64_t relpos_bw_slots(int64_t H) { return kRelposBwBlocks + H; }
LSR_RELPOS_BW_INSTANTIATE(float)
}  // namespace lsr
