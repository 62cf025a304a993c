// relpos_dispatch.cuh -- launchers of the softmax with a relative position
// bias (instantiated per storage dtype in relpos_f32.cu, relpos_f16.cu and
// relpos_bf16.cu, so that the build compiles them in parallel).
#pragma once

#include "dispatch.cuh"
#include "relpos.cuh"

namespace lsr {

// Most blocks of the backward.  A constant, not the device's SM count, so that
// the cut of the rows, and with it the order of the table gradient's sums,
// depends only on the problem.
constexpr int64_t kRelposSms = 152;
constexpr int64_t kRelposBwBlocks = 4 * kRelposSms;
// Shared memory of an SM that blocks can have, and of a block at most.
constexpr size_t kRelposSmSmem = 220 * 1024;
constexpr size_t kRelposBandMax = 100 * 1024;

// Opt in, once per device, to the most dynamic shared memory a kernel may ask
// for at the largest max_distance.
template <auto K>
cudaError_t relpos_allow_smem(size_t most) {
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

// Cut of p.rows into at most `blocks` runs of whole turns of G rows.
inline unsigned relpos_cut(RelposShape &p, int64_t blocks, int64_t G) {
    p.per = ceil_div(ceil_div(p.rows, blocks), G) * G;
    return (unsigned)ceil_div(p.rows, p.per);
}

// Resident blocks per SM: `most` by registers, fewer if shared memory is short.
inline int64_t relpos_resident(int most, size_t smem) {
    const int64_t fit = (int64_t)(kRelposSmSmem / (smem + 2048));
    return fit < most ? (fit < 1 ? 1 : fit) : most;
}

constexpr size_t relpos_sums_bytes(int R) { return (size_t)(2 * R + 1) * 4; }

// Threads per row and chunks per thread that pick_relpos_bucket can return.
#define LSR_RELPOS_BUCKETS(X)                                                     \
    X(1, 1) X(2, 1) X(4, 1) X(8, 1) X(16, 1) X(32, 1) X(32, 2) X(32, 3) X(32, 4) \
    X(64, 3) X(64, 4) X(128, 3) X(128, 4) X(256, 3) X(256, 4) X(512, 3) X(512, 4)

// Bucket of the register-resident kernels; false: the row is too long
// (or a head's rows pass 32 bits).
// `phase`: elements by which the tensors start past a 16-byte address.
// dense: as many chunks per thread as allowed (the row's own costs are then
// shared by more elements), else as few.
inline bool pick_relpos_bucket(bool dense, const RelposShape &p, int V, int phase, int *tpr, int *cpt) {
    if (p.Tk > (int64_t)512 * 4 * V || p.rows_per_head > INT32_MAX - 512) return false;
    const int64_t chunks = p.Tk % V == 0 && phase == 0 ? p.Tk / V : (p.Tk + 2 * V - 2) / V;
    if (dense) return pick_bucket_dense(chunks, 4, 512, tpr, cpt);
    if (!pick_bucket(chunks, 4, 512, tpr, cpt)) return false;
    if (*tpr > 32) *cpt = (int)ceil_div(chunks, *tpr);
    return true;
}

template <typename T>
int relpos_phase(const void *p) {
    return (int)(reinterpret_cast<uintptr_t>(p) % 16 / sizeof(T));
}

template <typename T, int TPR, int CPT, bool AL>
cudaError_t launch_relpos_fw_vec(T *out, const T *inp, const T *mask, const T *table,
                                 const int32_t *bucket, RelposShape p, int mask_vec,
                                 cudaStream_t st) {
    constexpr auto K = relpos_fw_vec<T, TPR, CPT, AL>;
    const size_t smem = relpos_fw_smem<TPR, CPT>(p.R);
    const cudaError_t e = relpos_allow_smem<K>(relpos_fw_smem<TPR, CPT>(kRelposMaxDistance));
    if (e != cudaSuccess) return e;
    const int64_t blocks =
        device_sm_count() * relpos_resident(relpos_fw_min_blocks<TPR, CPT>(), smem);
    const unsigned grid = relpos_cut(p, blocks, relpos_block<TPR>() / TPR);
    return launch_pdl(K, dim3(grid), dim3(relpos_block<TPR>()), smem, st, out, inp, mask, table,
                      bucket, p, mask_vec);
}

template <typename T>
cudaError_t launch_relpos_fw(T *out, const T *inp, const T *mask, const T *table,
                             const int32_t *bucket, RelposShape p, cudaStream_t st) {
    constexpr int V = Traits<T>::kVec;
    const int phase = relpos_phase<T>(inp);
    int tpr = 0, cpt = 0;
    if (relpos_phase<T>(out) == phase && pick_relpos_bucket(true, p, V, phase, &tpr, &cpt)) {
        const bool al = p.Tk % V == 0 && phase == 0;
        const int mask_vec = relpos_phase<T>(mask) == 0;
#define X(TPR_, CPT_)                                                                     \
    if (tpr == TPR_ && cpt == CPT_)                                                       \
        return al ? launch_relpos_fw_vec<T, TPR_, CPT_, true>(out, inp, mask, table,      \
                                                              bucket, p, mask_vec, st)    \
                  : launch_relpos_fw_vec<T, TPR_, CPT_, false>(out, inp, mask, table,     \
                                                               bucket, p, mask_vec, st);
        LSR_DENSE4_BUCKETS(X)
#undef X
    }
    const size_t smem = relpos_sums_bytes(p.R);
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

// Threads of a backward block whose row groups' arrays fit, 0: not even one
// warp's.
template <int TPR>
int relpos_bw_threads(size_t group_bytes) {
    for (int n = relpos_block<TPR>(); n >= (TPR < 32 ? 32 : TPR); n /= 2)
        if (group_bytes * (n / TPR) <= kRelposBandMax) return n;
    return 0;
}

template <typename T, int TPR, int CPT, bool AL>
cudaError_t launch_relpos_bw_vec(T *dinp, const T *dout, const T *y, const T *mask,
                                 RelposShape &p, float *part, int threads, cudaStream_t st) {
    constexpr auto K = relpos_bw_vec<T, TPR, CPT, AL>;
    const cudaError_t e = relpos_allow_smem<K>(kRelposBandMax);
    if (e != cudaSuccess) return e;
    const int G = threads / TPR;
    const size_t smem = (size_t)relpos_band<Traits<T>::kVec>(p).stride * 16 * G;
    const int64_t blocks =
        kRelposSms * relpos_resident(relpos_bw_resident<TPR, CPT>(), smem);
    const unsigned grid = relpos_cut(p, blocks, G);
    return launch_pdl(K, dim3(grid), dim3(threads), smem, st, dinp, part, dout, y, mask, p);
}

template <typename T>
cudaError_t launch_relpos_bw_rows(T *dinp, const T *dout, const T *y, const T *mask,
                                  RelposShape &p, float *part, cudaStream_t st) {
    constexpr int V = Traits<T>::kVec;
    const int phase = relpos_phase<T>(y);
    int tpr = 0, cpt = 0;
    if (relpos_phase<T>(dout) == phase && relpos_phase<T>(dinp) == phase &&
        pick_relpos_bucket(false, p, V, phase, &tpr, &cpt)) {
        const bool al = p.Tk % V == 0 && phase == 0;
        const size_t group_bytes = (size_t)relpos_band<V>(p).stride * 16;
#define X(TPR_, CPT_)                                                                       \
    if (tpr == TPR_ && cpt == CPT_) {                                                       \
        const int n = relpos_bw_threads<TPR_>(group_bytes);                                 \
        if (n > 0)                                                                          \
            return al ? launch_relpos_bw_vec<T, TPR_, CPT_, true>(dinp, dout, y, mask, p,   \
                                                                  part, n, st)              \
                      : launch_relpos_bw_vec<T, TPR_, CPT_, false>(dinp, dout, y, mask, p,  \
                                                                   part, n, st);            \
    }
        LSR_RELPOS_BUCKETS(X)
#undef X
    }
    if (p.Tk <= kLoopWarpRowMax) {
        const cudaError_t e =
            relpos_allow_smem<relpos_bw_loop<T, 32>>(8 * relpos_sums_bytes(kRelposMaxDistance));
        if (e != cudaSuccess) return e;
        const unsigned grid = relpos_cut(p, kRelposBwBlocks, 8);
        return launch_pdl(relpos_bw_loop<T, 32>, dim3(grid), dim3(256),
                          8 * relpos_sums_bytes(p.R), st, dinp, part, dout, y, mask, p);
    }
    const unsigned grid = relpos_cut(p, kRelposBwBlocks, 1);
    return launch_pdl(relpos_bw_loop<T, 256>, dim3(grid), dim3(256), relpos_sums_bytes(p.R), st,
                      dinp, part, dout, y, mask, p);
}

template <typename T>
cudaError_t launch_relpos_bw(T *dinp, float *dtable, const T *dout, const T *y, const T *mask,
                             const int32_t *bucket, RelposShape p, float *part,
                             cudaStream_t st) {
    p.per = 1;
    if (p.rows > 0) {
        const cudaError_t e = launch_relpos_bw_rows<T>(dinp, dout, y, mask, p, part, st);
        if (e != cudaSuccess) return e;
    }  // else rows_per_head is 0 too and the gradient becomes zero
    const dim3 grid((unsigned)p.H, (unsigned)ceil_div(p.num_buckets, kRelposFoldBuckets));
    return launch_pdl(relpos_fold, grid, dim3(256), relpos_sums_bytes(p.R), st, dtable,
                      (const float *)part, bucket, p);
}

#define LSR_RELPOS_INSTANTIATE(T)                                                              \
    template cudaError_t launch_relpos_fw<T>(T *, const T *, const T *, const T *,             \
                                             const int32_t *, RelposShape, cudaStream_t);      \
    template cudaError_t launch_relpos_bw<T>(T *, float *, const T *, const T *, const T *,    \
                                             const int32_t *, RelposShape, float *,            \
                                             cudaStream_t);

}  // namespace lsr
