// block_norm_dispatch.cuh -- launchers of the norms around a block
// (instantiated per storage dtype in block_norm_f32.cu ... block_norm_bf16.cu).
#pragma once

#include "block_norm.cuh"
#include "dispatch.cuh"
#include "relpos_dispatch.cuh"  // relpos_allow_smem

namespace lsr {

// Threads per row and chunks per thread.  Forward: up to four chunks, one where
// there are few rows.  Backward: two (of the sums of 16 columns, 64 registers
// for LayerNorm).
#define LSR_BN_FW_BUCKETS(X)                                                               \
    X(32, 1) X(32, 2) X(32, 4) X(64, 4) X(128, 4) X(256, 4) X(512, 4) X(1024, 4) X(64, 1) \
    X(128, 1) X(256, 1) X(512, 1) X(1024, 1)
#define LSR_BN_BW_BUCKETS(X) \
    X(32, 1) X(32, 2) X(64, 2) X(128, 2) X(256, 2) X(512, 2) X(1024, 2) X(1024, 4)

// Rows up to which the forward gives every chunk a thread of its own.
constexpr int64_t kBnFewRows = 608;  // four per SM
// Blocks of the backward: a constant, not the device's SM count, so that the
// order of the column sums depends only on the problem.
constexpr int64_t kBnSms = 152;

inline void pick_bn_bucket(int64_t chunks, int most, int *tpr, int *cpt) {
    int t = 32;
    while (t < 1024 && (int64_t)t * most < chunks) t *= 2;
    *tpr = t;
    const int64_t c = ceil_div(chunks, t);
    *cpt = c <= 1 ? 1 : c <= 2 ? 2 : 4;
    if (t > 32) *cpt = *cpt < most ? most : *cpt;
}

// (16-bit rows end at 2048 chunks)
template <typename T, int TPR, int CPT>
constexpr bool bn_reached() { return TPR * CPT <= 2048 || Traits<T>::kVec == 4; }

template <typename T>
bool bn_aligned(int64_t hidden, std::initializer_list<const void *> ptrs) {
    if (hidden % Traits<T>::kVec) return false;
    for (const void *p : ptrs)
        if (reinterpret_cast<uintptr_t>(p) % 16) return false;
    return true;
}

template <typename T>
cudaError_t launch_block_norm_fw(const BlockNorm<T> &a, cudaStream_t st) {
    const bool al = bn_aligned<T>(a.hidden, {a.x, a.r, a.gate, a.gamma_post, a.beta_post,
                                             a.gamma_pre, a.beta_pre, a.h, a.y});
    const int64_t chunks = ceil_div(a.hidden, Traits<T>::kVec);
    int tpr = 0, cpt = 0;
    pick_bn_bucket(chunks, a.rows <= kBnFewRows && chunks <= 1024 ? 1 : 4, &tpr, &cpt);
    auto go = [&](auto kernel, int per_sm, int block, int groups) {
        const int64_t workers = (int64_t)device_sm_count() * per_sm * groups;
        const int64_t per = ceil_div(a.rows, workers);
        return launch_pdl(kernel, dim3((unsigned)ceil_div(ceil_div(a.rows, per), groups)),
                          dim3(block), 0, st, a, per);
    };
#define F(TPR_, CPT_, AL_, L_)                                                                  \
    go(bn_fw<T, TPR_, CPT_, AL_, L_>,                                                           \
       occupancy_per_sm<bn_fw<T, TPR_, CPT_, AL_, L_>>(bn_block<TPR_>(), 0), bn_block<TPR_>(), \
       bn_block<TPR_>() / TPR_)
#define X(TPR_, CPT_)                                                                    \
    if constexpr (bn_reached<T, TPR_, CPT_>())                                           \
        if (tpr == TPR_ && cpt == CPT_)                                                  \
        return a.layer ? (al ? F(TPR_, CPT_, true, true) : F(TPR_, CPT_, false, true))   \
                       : (al ? F(TPR_, CPT_, true, false) : F(TPR_, CPT_, false, false));
    LSR_BN_FW_BUCKETS(X)
#undef X
#undef F
    return cudaErrorInvalidValue;  // (the buckets cover every size)
}

// The backward's bucket and cut.
struct BnPlan {
    int tpr, cpt, groups;
    BnCut cut;
};
template <typename T>
BnPlan bn_plan(int64_t rows, int64_t hidden, int64_t gates) {
    BnPlan p = {};
    const int64_t chunks = ceil_div(hidden, Traits<T>::kVec);
    pick_bn_bucket(chunks, 2, &p.tpr, &p.cpt);
    const int block = p.tpr < 256 ? 256 : p.tpr;
    p.groups = block / p.tpr;
    if (rows <= 0) return p;
    const int64_t most = kBnSms * (block <= 512 ? 512 / block : 1) * p.groups;
    const int64_t count = gates < 1 ? 1 : gates;
    const int64_t share = rows / count;  // rows of a gate
    const int64_t per = ceil_div(rows, most);
    if (gates > 1 && share <= per) {  // whole gates' rows
        p.cut.per = ceil_div(per, share) * share;
        p.cut.parts = 0;
        p.cut.workers = ceil_div(rows, p.cut.per);
    } else {
        int64_t parts = most / count;
        parts = parts < 1 ? 1 : parts;
        p.cut.per = ceil_div(share, parts);
        p.cut.parts = ceil_div(share, p.cut.per);
        p.cut.workers = count * p.cut.parts;
    }
    p.cut.blocks = ceil_div(p.cut.workers, p.groups);
    p.cut.single = gates <= 1;
    return p;
}

template <typename T>
size_t block_norm_workspace(int64_t rows, int64_t hidden, int64_t gates, bool layer) {
    const BnPlan p = bn_plan<T>(rows, hidden, gates);
    const int64_t gate_parts = gates > 1 && p.cut.parts > 1 ? p.cut.workers : 0;
    return (size_t)(p.cut.blocks * (layer ? 4 : 2) + gate_parts) * hidden * sizeof(float);
}

template <typename T>
cudaError_t launch_block_norm_bw(const BlockNorm<T> &a, float *part, cudaStream_t st) {
    const int64_t gates = a.gate ? a.gates : 0;
    const BnPlan p = bn_plan<T>(a.rows, a.hidden, gates);
    const int sums = a.layer ? 4 : 2;
    if (a.rows == 0 && gates > 0) {
        const cudaError_t z = cudaMemsetAsync(a.dgate, 0, (size_t)(gates * a.hidden) * 4, st);
        if (z != cudaSuccess) return z;
    }
    float *gate_part = part + p.cut.blocks * sums * a.hidden;
    cudaError_t e = cudaSuccess;
    if (a.rows > 0) {
        const bool al = bn_aligned<T>(a.hidden, {a.x, a.dy, a.dh, a.h_in, a.gate, a.gamma_post,
                                                 a.beta_post, a.gamma_pre, a.dx, a.dr, a.dgate});
        const bool multi = p.cut.parts == 0;
        const int form = !a.gamma_pre || !a.dh           ? kBnAny
                         : a.gamma_post                  ? (a.gate ? kBnGate : kBnPost)
                         : a.gate                        ? kBnAny
                                                         : kBnPlain;
        const int tpr = p.tpr, cpt = p.cpt;
        auto go = [&](auto kernel, int block, size_t smem) {
            return launch_pdl(kernel, dim3((unsigned)p.cut.blocks), dim3(block), smem, st, a, p.cut,
                              part, gate_part);
        };
        e = cudaErrorInvalidValue;  // (the buckets cover every size)
#define F(TPR_, CPT_, AL_, L_, M_, FORM_)                                                   \
    (e = relpos_allow_smem<bn_bw<T, TPR_, CPT_, AL_, L_, M_, FORM_>>(                       \
         bn_bw_smem<TPR_, CPT_, AL_>(Traits<T>::kVec)),                                     \
     e == cudaSuccess ? go(bn_bw<T, TPR_, CPT_, AL_, L_, M_, FORM_>, bn_block<TPR_>(),      \
                           bn_bw_smem<TPR_, CPT_, AL_>(Traits<T>::kVec))                    \
                      : e)
#define M(TPR_, CPT_, L_)                                                              \
    (!al ? (multi ? F(TPR_, CPT_, false, L_, true, kBnAny)                             \
                  : F(TPR_, CPT_, false, L_, false, kBnAny))                           \
     : multi ? (form == kBnGate ? F(TPR_, CPT_, true, L_, true, kBnGate)               \
                                : F(TPR_, CPT_, true, L_, true, kBnAny))               \
     : form == kBnGate  ? F(TPR_, CPT_, true, L_, false, kBnGate)                      \
     : form == kBnPost  ? F(TPR_, CPT_, true, L_, false, kBnPost)                      \
     : form == kBnPlain ? F(TPR_, CPT_, true, L_, false, kBnPlain)                     \
                        : F(TPR_, CPT_, true, L_, false, kBnAny))
#define X(TPR_, CPT_)                                          \
    if constexpr (bn_reached<T, TPR_, CPT_>())                 \
        if (tpr == TPR_ && cpt == CPT_)                        \
            e = a.layer ? M(TPR_, CPT_, true) : M(TPR_, CPT_, false);
        LSR_BN_BW_BUCKETS(X)
#undef X
#undef M
#undef F
        if (e != cudaSuccess) return e;
    }
    BnFold<T> f = {};
    f.part = part;
    f.gate_part = gate_part;
    f.out[0] = a.dgamma_pre;
    f.out[1] = a.dgamma_post;
    f.out[2] = a.dbeta_pre;
    f.out[3] = a.dbeta_post;
    f.dgate = a.dgate;
    f.hidden = a.hidden;
    f.blocks = p.cut.blocks;
    f.parts = p.cut.parts;
    f.sums = sums;
    f.single = p.cut.single;
    f.gate = a.gate;
    f.gamma_post = a.gamma_post;
    f.beta_post = a.beta_post;
    const int64_t vectors = sums + (gates > 1 && p.cut.parts > 1 ? gates : 0);
    const bool wide = a.hidden % 4 == 0 && reinterpret_cast<uintptr_t>(a.dgate) % 16 == 0 &&
                      reinterpret_cast<uintptr_t>(a.dgamma_pre) % 16 == 0 &&
                      reinterpret_cast<uintptr_t>(a.dgamma_post) % 16 == 0 &&
                      reinterpret_cast<uintptr_t>(a.dbeta_pre) % 16 == 0 &&
                      reinterpret_cast<uintptr_t>(a.dbeta_post) % 16 == 0;
    return launch_pdl(wide ? bn_fold<T, 4> : bn_fold<T, 1>,
                      dim3((unsigned)ceil_div(a.hidden, wide ? 128 : 32), (unsigned)vectors),
                      dim3(32 * kBnFoldWarps), 0, st, f);
}

#define LSR_BN_FW_INSTANTIATE(T) \
    template cudaError_t launch_block_norm_fw<T>(const BlockNorm<T> &, cudaStream_t);
#define LSR_BN_BW_INSTANTIATE(T)                                                               \
    template cudaError_t launch_block_norm_bw<T>(const BlockNorm<T> &, float *, cudaStream_t); \
    template size_t block_norm_workspace<T>(int64_t, int64_t, int64_t, bool);

}  // namespace lsr
