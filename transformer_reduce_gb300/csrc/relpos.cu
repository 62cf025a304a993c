// relpos.cu -- launchers and instantiations of the softmax with a relative
// position bias, for every storage dtype.
#include "relpos.cuh"
#include "dispatch.cuh"

namespace lsr {

// Blocks of the backward, a constant (not the device's SM count), so that the
// cut of the rows and with it the order of the table gradient's sums depend
// only on the problem.
constexpr int64_t kRelposBwBlocks = 4 * 152;

int64_t relpos_bw_slots(int64_t H) { return kRelposBwBlocks + H; }

// Opt in, once per device, to the most dynamic shared memory a kernel may ask
// for at the largest max_distance.
template <auto K>
static cudaError_t relpos_allow_smem(size_t most) {
    static std::atomic<int> done[kMaxDevices];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < kMaxDevices && done[dev].load(std::memory_order_acquire))
        return cudaSuccess;
    e = cudaFuncSetAttribute(K, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)most);
    if (e == cudaSuccess && dev >= 0 && dev < kMaxDevices)
        done[dev].store(1, std::memory_order_release);
    return e;
}

// Cut of p.rows into at most `blocks` runs of whole groups of G rows.
static unsigned relpos_cut(RelposShape &p, int64_t blocks, int64_t G) {
    p.per = ceil_div(ceil_div(p.rows, blocks), G) * G;
    return (unsigned)ceil_div(p.rows, p.per);
}

constexpr size_t relpos_lut_bytes(int R) { return (size_t)(2 * R + 1) * 4; }

template <typename T>
cudaError_t launch_relpos_fw(T *out, const T *inp, const T *mask, const T *table,
                             const int32_t *bucket, RelposShape p, cudaStream_t st) {
    const size_t smem = relpos_lut_bytes(p.R);
    const int64_t blocks = (int64_t)device_sm_count() * 8;
    if (p.Tk <= kLoopWarpRowMax) {
        const unsigned grid = relpos_cut(p, blocks, 8);
        return launch_pdl(relpos_fw_loop<T, 32>, dim3(grid), dim3(256), smem, st, out, inp, mask,
                          table, bucket, p);
    }
    const unsigned grid = relpos_cut(p, blocks, 1);
    return launch_pdl(relpos_fw_loop<T, 256>, dim3(grid), dim3(256), smem, st, out, inp, mask,
                      table, bucket, p);
}

template <typename T>
cudaError_t launch_relpos_bw(T *dinp, float *dtable, const T *dout, const T *y, const T *mask,
                             const int32_t *bucket, RelposShape p, float *part,
                             cudaStream_t st) {
    cudaError_t e = cudaSuccess;
    p.per = 1;
    if (p.rows > 0 && p.Tk > 0) {
        if (p.Tk <= kLoopWarpRowMax) {
            e = relpos_allow_smem<relpos_bw_loop<T, 32>>(8 * relpos_lut_bytes(kRelposMaxDistance));
            if (e != cudaSuccess) return e;
            const unsigned grid = relpos_cut(p, kRelposBwBlocks, 8);
            e = launch_pdl(relpos_bw_loop<T, 32>, dim3(grid), dim3(256),
                           8 * relpos_lut_bytes(p.R), st, dinp, part, dout, y, mask, p);
        } else {
            const unsigned grid = relpos_cut(p, kRelposBwBlocks, 1);
            e = launch_pdl(relpos_bw_loop<T, 256>, dim3(grid), dim3(256), relpos_lut_bytes(p.R),
                           st, dinp, part, dout, y, mask, p);
        }
        if (e != cudaSuccess) return e;
    } else {
        p.rows_per_head = 0;  // no row: the gradient is zero
    }
    const dim3 grid((unsigned)p.H, (unsigned)ceil_div(p.num_buckets, kRelposFoldBuckets));
    return launch_pdl(relpos_fold, grid, dim3(256), relpos_lut_bytes(p.R), st, dtable,
                      (const float *)part, bucket, p);
}

#define LSR_RELPOS_INSTANTIATE(T)                                                              \
    template cudaError_t launch_relpos_fw<T>(T *, const T *, const T *, const T *,             \
                                             const int32_t *, RelposShape, cudaStream_t); \
    template cudaError_t launch_relpos_bw<T>(T *, float *, const T *, const T *, const T *,    \
                                             const int32_t *, RelposShape, float *,            \
                                             cudaStream_t);
LSR_RELPOS_INSTANTIATE(float)
LSR_RELPOS_INSTANTIATE(__half)
LSR_RELPOS_INSTANTIATE(__nv_bfloat16)
#undef LSR_RELPOS_INSTANTIATE

}  // namespace lsr
