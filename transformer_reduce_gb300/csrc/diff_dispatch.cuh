// diff_dispatch.cuh -- launchers of the difference of two softmax maps
// (instantiated per direction and storage dtype in diff_fw_f32.cu ...
// diff_bw_bf16.cu, so that the build compiles them in parallel).
#pragma once

#include "diff_softmax.cuh"
#include "relpos_dispatch.cuh"  // relpos_allow_smem, relpos_phase

namespace lsr {

// Threads per row and chunks per thread: as many chunks as registers allow for
// most calls, one for calls of few rows.
#define LSR_DIFF_FW_BUCKETS(X)                                                           \
    X(4, 1) X(4, 2) X(4, 4) X(8, 3) X(8, 4) X(16, 3) X(16, 4) X(32, 3) X(32, 4) X(64, 3) \
    X(64, 4) X(128, 3) X(128, 4) X(256, 3) X(256, 4) X(512, 3) X(512, 4)                 \
    X(32, 1) X(64, 1) X(128, 1) X(256, 1) X(512, 1)
// (the backward holds three tensors; four chunks spill and took 135 us where two
// take 120)
#define LSR_DIFF_BW_BUCKETS(X)                                                            \
    X(4, 1) X(4, 2) X(8, 2) X(16, 2) X(32, 2) X(64, 2) X(128, 2) X(256, 2) X(512, 2)      \
    X(512, 4) X(32, 1) X(64, 1) X(128, 1) X(256, 1) X(512, 1)

// Rows up to which a call spreads a row over as many threads as it has chunks
// (a call of so few rows does not fill the GPU with a block per eight rows).
constexpr int64_t kDiffFewRows = 1216;  // eight per SM

// Bucket of the register-resident kernels, at most `most` chunks per thread but
// for the longest rows; false: the row is too long (or a head passes 32 bits).
inline bool pick_diff_bucket(const DiffShape &p, int V, bool al, int most, int *tpr, int *cpt) {
    if (p.Tk > (int64_t)512 * 4 * V || p.Tq > INT32_MAX / p.Tk) return false;
    const int64_t chunks = al ? p.Tk / V : (p.Tk + 2 * V - 2) / V;
    if (p.rows <= kDiffFewRows && chunks > 16 && chunks <= 512) {
        *tpr = next_pow2(chunks);
        *cpt = 1;
        return true;
    }
    const int longest = chunks > 512 * most ? 4 : most;
    if (!pick_bucket_dense(chunks, longest, 512, tpr, cpt)) return false;
    if (*tpr < 4) {
        const int c = (int)ceil_div(*tpr * *cpt, 4);
        *tpr = 4;
        *cpt = c;
    }
    if (*cpt == 3 && (*tpr == 4 || most == 2)) *cpt = 4;  // (the instantiated ones)
    return true;
}

// Phase of a tensor's rows relative to those of dense rows [B, H, Tq, Tk] that
// start `phase` elements past a 16-byte address: whether all agree.
template <typename T, typename P>
bool diff_same_phase(const DiffRows<P> &x, int phase, const DiffShape &p) {
    constexpr int V = Traits<T>::kVec;
    const int64_t dense = p.Tq * p.Tk;
    return relpos_phase<T>(x.p) == phase && (x.head - dense) % V == 0 &&
           (x.batch - p.H * dense) % V == 0;
}

// Whether the rows of a causal call are dealt over the grid, in turns of G rows,
// instead of cut into runs of `per`.  A block that meets every batch entry looks
// through all their masks first, and past kRelposWinMax of them adds the mask
// element by element; a run of half a head or more is balanced by itself.  Dealt
// and in runs, us, forward and backward, bf16 with padding:
//     [64,1,16,1000] 24.3, 27.7 and  9.3,  13.2     [70,6,333,333]   118, 249 and  98, 200
//     [32,8,512,512] 70.1, 118  and 63.9, 116       [8,8,1024,1024] 64.1, 107 and 73.6, 123
//     [64,8,256,256] 42.6, 74.2 and 35.1, 62.7      [4,8,2048,2048]  125, 194 and  150, 229
template <bool MASKED>
bool diff_dealt(const DiffShape &p, int G) {
    if (!p.causal || p.Tq == 1) return false;
    return !MASKED || (p.per * 2 < p.Tq && p.B <= p.per / G && p.B <= kRelposWinMax);
}

template <auto K, int TPR, int CPT, bool AL, bool MASKED, typename... Args>
cudaError_t launch_diff_rows(int tensors, int resident, int mask_vec, DiffShape p, cudaStream_t st, Args... args) {
    const size_t smem = diff_smem<TPR, CPT, AL>(tensors);
    const cudaError_t e = relpos_allow_smem<K>(smem);
    if (e != cudaSuccess) return e;
    const int G = diff_block<TPR>() / TPR;
    const int64_t blocks =
        (int64_t)device_sm_count() * relpos_resident(resident, smem);
    p.per = ceil_div(ceil_div(p.rows, blocks), G) * G;
    const unsigned grid = (unsigned)ceil_div(p.rows, p.per);
    if (diff_dealt<MASKED>(p, G)) p.per = 0;
    return launch_pdl(K, dim3(grid), dim3(diff_block<TPR>()), smem, st, args..., p, mask_vec);
}

template <typename T>
cudaError_t launch_diff_fw(T *out, float4 *stats, DiffRows<const T> x1, DiffRows<const T> x2,
                           const float *lam, const T *mask, DiffShape p, cudaStream_t st) {
    constexpr int V = Traits<T>::kVec;
    const bool al = p.Tk % V == 0 && relpos_phase<T>(out) == 0 && diff_same_phase<T>(x1, 0, p) &&
                    diff_same_phase<T>(x2, 0, p);
    int tpr = 0, cpt = 0;
    const int mask_vec = relpos_phase<T>(mask) == 0;
    if (pick_diff_bucket(p, V, al, 4, &tpr, &cpt)) {
#define F(TPR_, CPT_, AL_, M_)                                                             \
    launch_diff_rows<diff_fw_vec<T, TPR_, CPT_, AL_, M_>, TPR_, CPT_, AL_, M_>(             \
        2, diff_fw_min_blocks<TPR_, CPT_>(), mask_vec, p, st, out, stats, x1, x2, lam, mask)
#define X(TPR_, CPT_)                                                               \
    if (tpr == TPR_ && cpt == CPT_)                                                 \
        return mask ? (al ? F(TPR_, CPT_, true, true) : F(TPR_, CPT_, false, true)) \
                    : (al ? F(TPR_, CPT_, true, false) : F(TPR_, CPT_, false, false));
        LSR_DIFF_FW_BUCKETS(X)
#undef X
#undef F
    }
    if (p.Tk <= kLoopWarpRowMax)
        return launch_persistent<diff_fw_loop<T, 32>>(256, 0, ceil_div(p.rows, 8), st, out, stats,
                                                      x1, x2, lam, mask, p);
    return launch_persistent<diff_fw_loop<T, 256>>(256, 0, p.rows, st, out, stats, x1, x2, lam,
                                                   mask, p);
}

template <typename T>
cudaError_t launch_diff_bw_rows(DiffRows<T> dx1, DiffRows<T> dx2, float *row_dot, const T *dout,
                                DiffRows<const T> x1, DiffRows<const T> x2, const float *lam,
                                const float4 *stats, const T *mask, DiffShape p,
                                cudaStream_t st) {
    constexpr int V = Traits<T>::kVec;
    const int phase = relpos_phase<T>(dout);
    const bool al = p.Tk % V == 0 && phase == 0 && diff_same_phase<T>(x1, 0, p) &&
                    diff_same_phase<T>(x2, 0, p);
    int tpr = 0, cpt = 0;
    const int mask_vec = relpos_phase<T>(mask) == 0;
    if (diff_same_phase<T>(dx1, phase, p) && diff_same_phase<T>(dx2, phase, p) &&
        pick_diff_bucket(p, V, al, 2, &tpr, &cpt)) {
#define F(TPR_, CPT_, AL_, M_)                                                                 \
    launch_diff_rows<diff_bw_vec<T, TPR_, CPT_, AL_, M_>, TPR_, CPT_, AL_, M_>(                 \
        3, diff_bw_min_blocks<TPR_, CPT_>(), mask_vec, p, st, dx1, dx2, row_dot, dout, x1, x2, \
        lam, stats, mask)
#define X(TPR_, CPT_)                                                               \
    if (tpr == TPR_ && cpt == CPT_)                                                 \
        return mask ? (al ? F(TPR_, CPT_, true, true) : F(TPR_, CPT_, false, true)) \
                    : (al ? F(TPR_, CPT_, true, false) : F(TPR_, CPT_, false, false));
        LSR_DIFF_BW_BUCKETS(X)
#undef X
#undef F
    }
    if (p.Tk <= kLoopWarpRowMax)
        return launch_persistent<diff_bw_loop<T, 32>>(256, 0, ceil_div(p.rows, 8), st, dx1, dx2,
                                                      row_dot, dout, x1, x2, lam, stats, mask, p);
    return launch_persistent<diff_bw_loop<T, 256>>(256, 0, p.rows, st, dx1, dx2, row_dot, dout, x1,
                                                   x2, lam, stats, mask, p);
}

template <typename T>
cudaError_t launch_diff_bw(DiffRows<T> dx1, DiffRows<T> dx2, float *dlam, const T *dout,
                           DiffRows<const T> x1, DiffRows<const T> x2, const float *lam,
                           const float4 *stats, const T *mask, DiffShape p, float *row_dot,
                           cudaStream_t st) {
    if (p.rows > 0 && p.Tk > 0) {
        const cudaError_t e = launch_diff_bw_rows<T>(dx1, dx2, row_dot, dout, x1, x2, lam, stats,
                                                     mask, p, st);
        if (e != cudaSuccess) return e;
    } else {
        p.rows = 0;  // the gradient becomes zero
    }
    return launch_pdl(diff_fold, dim3(p.lam_step ? (unsigned)p.H : 1u), dim3(kDiffFoldThreads), 0,
                      st, dlam, (const float *)row_dot, p);
}

#define LSR_DIFF_FW_INSTANTIATE(T)                                                            \
    template cudaError_t launch_diff_fw<T>(T *, float4 *, DiffRows<const T>, DiffRows<const T>, \
                                           const float *, const T *, DiffShape, cudaStream_t);
#define LSR_DIFF_BW_INSTANTIATE(T)                                                              \
    template cudaError_t launch_diff_bw<T>(DiffRows<T>, DiffRows<T>, float *, const T *,        \
                                           DiffRows<const T>, DiffRows<const T>, const float *, \
                                           const float4 *, const T *, DiffShape, float *,       \
                                           cudaStream_t);

}  // namespace lsr
