// relpos_dispatch.cuh -- launchers of the softmax with a relative position
// bias (instantiated per direction and storage dtype in relpos_fw_f32.cu ...
// relpos_bw_bf16.cu, so that the build compiles them in parallel).
#pragma once

#include "dispatch.cuh"
#include "relpos.cuh"

namespace lsr {

// Most blocks of the backward.  A constant, not the device's SM count, so that
// the cut of the rows, and with it the order of the table gradient's sums,
// depends only on the problem.
constexpr int64_t kRelposSms = 152;
constexpr int64_t kRelposBwBlocks = 4 * kRelposSms;
// Shared memory of an SM that the blocks can have.
constexpr size_t kRelposSmSmem = 220 * 1024;

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

// Threads per row and chunks per thread of the backward (those of
// LSR_DENSE4_BUCKETS with at least four threads).
#define LSR_RELPOS_BW_BUCKETS(X)                                                        \
    X(4, 1) X(4, 2) X(4, 3) X(4, 4) X(8, 3) X(8, 4) X(16, 3) X(16, 4) X(32, 3) X(32, 4) \
    X(64, 3) X(64, 4) X(128, 3) X(128, 4) X(256, 3) X(256, 4) X(512, 3) X(512, 4)

// Bucket of the register-resident kernels; false: the row is too long
// (or a head's rows pass 32 bits).
// `phase`: elements by which the tensors start past a 16-byte address.
// As many chunks per thread as allowed, so that the row's own costs are shared
// by more elements ([32,16,512,512] bf16 forward: 322 instructions per row and
// warp at one row per warp and two chunks, 92 us at two rows and four).
inline bool pick_relpos_bucket(const RelposShape &p, int V, int phase, int *tpr, int *cpt) {
    if (p.Tk > (int64_t)512 * 4 * V || p.rows_per_head > INT32_MAX - 512) return false;
    const int64_t chunks = p.Tk % V == 0 && phase == 0 ? p.Tk / V : (p.Tk + 2 * V - 2) / V;
    return pick_bucket_dense(chunks, 4, 512, tpr, cpt);
}

template <typename T>
int relpos_phase(const void *p) {
    return (int)(reinterpret_cast<uintptr_t>(p) % 16 / sizeof(T));
}

template <typename T, int TPR, int CPT, bool AL, bool MASKED>
cudaError_t launch_relpos_fw_vec(T *out, const T *inp, const T *mask, const T *table,
                                 const int32_t *bucket, RelposShape p, int mask_vec,
                                 cudaStream_t st) {
    constexpr auto K = relpos_fw_vec<T, TPR, CPT, AL, MASKED>;
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
    if (relpos_phase<T>(out) == phase && pick_relpos_bucket(p, V, phase, &tpr, &cpt)) {
        const bool al = p.Tk % V == 0 && phase == 0;
        const int mask_vec = relpos_phase<T>(mask) == 0;
#define F(TPR_, CPT_, AL_, M_) \
    launch_relpos_fw_vec<T, TPR_, CPT_, AL_, M_>(out, inp, mask, table, bucket, p, mask_vec, st)
#define X(TPR_, CPT_)                                                              \
    if (tpr == TPR_ && cpt == CPT_)                                                \
        return mask ? (al ? F(TPR_, CPT_, true, true) : F(TPR_, CPT_, false, true)) \
                    : (al ? F(TPR_, CPT_, true, false) : F(TPR_, CPT_, false, false));
        LSR_DENSE4_BUCKETS(X)
#undef X
#undef F
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

// Threads of a backward block: as many as let two blocks share an SM, at
// least a warp or a row group.  (The largest arrays, max_distance 2048 with
// two of them in one warp, still fit kRelposSmSmem.)
template <int TPR, int CPT>
int relpos_bw_threads(int band_stride) {
    int n = relpos_block<TPR>();
    while (n / 2 >= (TPR < 32 ? 32 : TPR) &&
           relpos_bw_smem<TPR, CPT>(n, band_stride) > kRelposSmSmem / 2 - 4096)
        n /= 2;
    return n;
}

template <typename T, int TPR, int CPT, bool AL, bool MASKED>
cudaError_t launch_relpos_bw_vec(T *dinp, const T *dout, const T *y, const T *mask,
                                 RelposShape &p, float *part, cudaStream_t st) {
    constexpr auto K = relpos_bw_vec<T, TPR, CPT, AL, MASKED>;
    const cudaError_t e = relpos_allow_smem<K>(kRelposSmSmem);
    if (e != cudaSuccess) return e;
    const int stride = relpos_band<Traits<T>::kVec>(p).stride;
    const int n = relpos_bw_threads<TPR, CPT>(stride);
    const size_t smem = relpos_bw_smem<TPR, CPT>(n, stride);
    int64_t blocks = kRelposSms * relpos_resident(512 / n, smem);
    if (blocks > kRelposBwBlocks) blocks = kRelposBwBlocks;
    const unsigned grid = relpos_cut(p, blocks, n / TPR);
    return launch_pdl(K, dim3(grid), dim3(n), smem, st, dinp, part, dout, y, mask, p);
}

template <typename T>
cudaError_t launch_relpos_bw_rows(T *dinp, const T *dout, const T *y, const T *mask,
                                  RelposShape &p, float *part, cudaStream_t st) {
    constexpr int V = Traits<T>::kVec;
    const int phase = relpos_phase<T>(y);
    int tpr = 0, cpt = 0;
    if (relpos_phase<T>(dout) == phase && relpos_phase<T>(dinp) == phase &&
        pick_relpos_bucket(p, V, phase, &tpr, &cpt)) {
        const bool al = p.Tk % V == 0 && phase == 0 && p.Tq % 4 == 0;
        if (tpr < 4) {  // groups of one or two threads would need too many arrays
            cpt = (int)ceil_div(tpr * cpt, 4);
            tpr = 4;
        }
#define F(TPR_, CPT_, AL_, M_) \
    launch_relpos_bw_vec<T, TPR_, CPT_, AL_, M_>(dinp, dout, y, mask, p, part, st)
#define X(TPR_, CPT_)                                                              \
    if (tpr == TPR_ && cpt == CPT_)                                                \
        return mask ? (al ? F(TPR_, CPT_, true, true) : F(TPR_, CPT_, false, true)) \
                    : (al ? F(TPR_, CPT_, true, false) : F(TPR_, CPT_, false, false));
        LSR_RELPOS_BW_BUCKETS(X)
#undef X
#undef F
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
    return launch_pdl(relpos_fold, grid, dim3(kRelposFoldThreads), relpos_fold_smem(p.R), st,
                      dtable, (const float *)part, bucket, p);
}

#define LSR_RELPOS_FW_INSTANTIATE(T)                                                        \
    template cudaError_t launch_relpos_fw<T>(T *, const T *, const T *, const T *,          \
                                             const int32_t *, RelposShape, cudaStream_t);
#define LSR_RELPOS_BW_INSTANTIATE(T)                                                        \
    template cudaError_t launch_relpos_bw<T>(T *, float *, const T *, const T *, const T *, \
                                             const int32_t *, RelposShape, float *,         \
                                             cudaStream_t);

}  // namespace lsr
