// qk_dispatch.cuh -- launchers of the per-head query / key norm with the
// position rotation (instantiated per storage dtype in qk_norm_rope_f32.cu,
// qk_norm_rope_f16.cu and qk_norm_rope_bf16.cu).
#pragma once

#include <type_traits>

#include "dispatch.cuh"
#include "qk_norm_rope.cuh"

namespace lsr {

// Most blocks of the backward.
constexpr int64_t kQkBwBlocks = 4 * 152;

// Blocks of the query and key sides of the backward: `blocks` (a constant, not
// the device's SM count, so that the order of the gamma gradient's sums depends
// only on the problem) in proportion to the sides' work, each side with at most
// one block per eight tokens.
inline void qk_bw_split(int64_t tokens, int64_t blocks, int64_t wq, int64_t wk, int64_t &nq,
                        int64_t &nk) {
    nq = blocks * wq / (wq + wk);
    if (wq > 0 && nq < 1) nq = 1;
    if (wk > 0 && nq > blocks - 1) nq = blocks - 1;
    nk = wk > 0 ? blocks - nq : 0;
    const int64_t most = ceil_div(tokens, 8);
    if (nq > most) nq = most;
    if (nk > most) nk = most;
}

// Whether a side's heads are whole vectors of V elements at their alignment.
template <typename T>
bool qk_side_vec(const QkSide<T> &s, int V) {
    const auto bits = reinterpret_cast<uintptr_t>(s.out) | reinterpret_cast<uintptr_t>(s.x) |
                      reinterpret_cast<uintptr_t>(s.dout) | reinterpret_cast<uintptr_t>(s.gamma);
    const int64_t strides = s.x_stride | s.out_stride | s.dout_stride;
    return s.heads == 0 || (bits % (V * sizeof(T)) == 0 && strides % V == 0);
}
// Lanes per head (a power of two) of the kernel with vectors of V elements; 0:
// it cannot take this call.
template <typename T>
int qk_lanes_vec(const QkSide<T> &q, const QkSide<T> &k, const QkRope &r, int V, int least) {
    const auto angles = reinterpret_cast<uintptr_t>(r.cos) | reinterpret_cast<uintptr_t>(r.sin);
    if (r.D % V || r.rot % (r.interleaved ? V : 2 * V) || angles % 8 || !qk_side_vec(q, V) ||
        !qk_side_vec(k, V) || q.heads + k.heads > (1 << 20))  // (a token's elements fit 31 bits)
        return 0;
    int lanes = least;
    while (lanes < qk_lanes(r.D, r.rot, V, r.interleaved)) lanes *= 2;
    return lanes <= 32 ? lanes : 0;
}

template <typename T, int V, int LPR, bool INTER>
cudaError_t launch_qk_fw_vec(const QkSide<T> &q, const QkSide<T> &k, const QkRope &r,
                             cudaStream_t st) {
    constexpr int RPW = 32 / LPR;
    const int ngq = (int)ceil_div(q.heads, RPW), ngk = (int)ceil_div(k.heads, RPW);
    // as many groups of a token per warp as leave a warp for every warp slot
    // (two blocks of eight on each SM)
    const int64_t slots = (int64_t)device_sm_count() * 16;
    int64_t per_item = r.tokens * (ngq + ngk) / slots;
    per_item = per_item < 1 ? 1 : (per_item > ngq + ngk ? ngq + ngk : per_item);
    const int64_t items = r.tokens * ceil_div(ngq + ngk, per_item);
    return launch_persistent<qk_fw_vec<T, V, LPR, INTER>>(256, 0, ceil_div(items, 8), st, q, k, r,
                                                          ngq, ngk, (int)per_item);
}

// Calls f(V, LPR) as integral constants for the widest vectors that the call's
// sizes and addresses allow; false if none do.  Forward / backward of 8192
// tokens of 16 + 16 heads, bf16, against one warp per head (qk_fw_slots): 84
// features in 8-byte vectors 29 / 41 us, 72 / 92; 36 features in 4-byte vectors
// 23 / 33, 56 / 61.
// Vectors of two elements on 32 lanes (66 to 128 features) are for the forward
// alone.  The same call in vectors / by one warp per head, forward and
// backward: bf16 66 features 43 / 71 and 98 / 87 us, 100 features 44 / 72 and
// 99 / 92, 126 features 44 / 73 and 99 / 98; fp32 66 features 44 / 66 and 103 /
// 84, 100 features 49 / 68 and 112 / 91, 126 features 56 / 72 and 113 / 97.
// (Only 128 features of bf16 4 bytes off a boundary lose by it: 96 / 98.)
template <typename T, bool BACK, typename F>
bool qk_pick(const QkSide<T> &q, const QkSide<T> &k, const QkRope &r, F f) {
    constexpr int W = Traits<T>::kVec;  // 16 bytes
    int lanes = qk_lanes_vec(q, k, r, W, 2);
#define X(V_, L_)                                                                    \
    if constexpr (!(BACK && (V_) == 2 && L_ == 32)) {                                \
        if (lanes == L_) {                                                           \
            f(std::integral_constant<int, V_>(), std::integral_constant<int, L_>()); \
            return true;                                                             \
        }                                                                            \
    }
    X(W, 2) X(W, 4) X(W, 8) X(W, 16) X(W, 32)
    lanes = qk_lanes_vec(q, k, r, W / 2, 8);  // 8 bytes
    X(W / 2, 8) X(W / 2, 16) X(W / 2, 32)
    if constexpr (W / 4 >= 2) {
        lanes = qk_lanes_vec(q, k, r, W / 4, 8);  // 4 bytes
        X(W / 4, 8) X(W / 4, 16) X(W / 4, 32)
    }
#undef X
    return false;
}

template <typename T, int NS>
cudaError_t launch_qk_fw_slots(const QkSide<T> &q, const QkSide<T> &k, const QkRope &r,
                               cudaStream_t st) {
    // (heads as the groups of the vector kernel, one per warp at a time)
    const int64_t heads = q.heads + k.heads, slots = (int64_t)device_sm_count() * 16;
    int64_t per_item = r.tokens > 0 ? r.tokens * heads / slots : 1;
    per_item = per_item < 1 ? 1 : (per_item > heads ? heads : per_item);
    const int64_t items = r.tokens * ceil_div(heads, per_item);
    return launch_persistent<qk_fw_slots<T, NS>>(256, 0, ceil_div(items, 8), st, q, k, r,
                                                 (int)per_item);
}

template <typename T>
cudaError_t launch_qk_fw(QkSide<T> q, QkSide<T> k, QkRope r, cudaStream_t st) {
    cudaError_t e = cudaSuccess;
    if (qk_pick<T, false>(q, k, r, [&](auto v, auto lanes) {
            constexpr int V = decltype(v)::value, L = decltype(lanes)::value;
            e = r.interleaved ? launch_qk_fw_vec<T, V, L, true>(q, k, r, st)
                              : launch_qk_fw_vec<T, V, L, false>(q, k, r, st);
        }))
        return e;
#define X(NS_) \
    if (r.D <= 64 * NS_) return launch_qk_fw_slots<T, NS_>(q, k, r, st);
    X(1) X(2) X(4) X(8) X(16)
#undef X
    return cudaErrorInvalidValue;  // not reachable: D <= kQkMaxHeadDim
}

template <typename T, int V, int LPR, bool INTER>
cudaError_t launch_qk_bw_vec(const QkSide<T> &q, const QkSide<T> &k, const QkRope &r, float *part,
                             int64_t &nq, int64_t &nk, cudaStream_t st) {
    constexpr int RPW = 32 / LPR;
    // two blocks on each SM; a side's work goes by its groups of heads
    qk_bw_split(r.tokens, 2 * 152, ceil_div(q.heads, RPW), ceil_div(k.heads, RPW), nq, nk);
    ensure_dynamic_smem<qk_bw_vec<T, V, LPR, INTER>>(qk_bw_smem<T, V>());
    return launch_pdl(qk_bw_vec<T, V, LPR, INTER>, dim3((unsigned)(nq + nk)), dim3(256),
                      qk_bw_smem<T, V>(), st, q, k, r, part, (int)nq);
}

template <typename T>
cudaError_t launch_qk_bw_rows(const QkSide<T> &q, const QkSide<T> &k, const QkRope &r, float *part,
                              int64_t &nq, int64_t &nk, cudaStream_t st) {
    cudaError_t e = cudaSuccess;
    if (qk_pick<T, true>(q, k, r, [&](auto v, auto lanes) {
            constexpr int V = decltype(v)::value, L = decltype(lanes)::value;
            e = r.interleaved ? launch_qk_bw_vec<T, V, L, true>(q, k, r, part, nq, nk, st)
                              : launch_qk_bw_vec<T, V, L, false>(q, k, r, part, nq, nk, st);
        }))
        return e;
    qk_bw_split(r.tokens, kQkBwBlocks, q.heads, k.heads, nq, nk);
#define X(NS_)                                                                          \
    if (r.D <= 64 * NS_)                                                                \
        return launch_pdl(qk_bw_slots<T, NS_>, dim3((unsigned)(nq + nk)), dim3(256),    \
                          (size_t)8 * r.D * 4, st, q, k, r, part, (int)nq);
    X(1) X(2) X(4) X(8) X(16)
#undef X
    return cudaErrorInvalidValue;  // not reachable: D <= kQkMaxHeadDim
}

template <typename T>
cudaError_t launch_qk_bw(QkSide<T> q, QkSide<T> k, QkRope r, float *part, cudaStream_t st) {
    int64_t nq = 0, nk = 0;
    if (r.tokens > 0) {
        const cudaError_t e = launch_qk_bw_rows(q, k, r, part, nq, nk, st);
        if (e != cudaSuccess) return e;
    }
    return launch_pdl(qk_fold, dim3((unsigned)ceil_div(r.D, 32), 2), dim3(1024), 0, st, q.dgamma,
                      k.dgamma, (const float *)part, r.D, (int)nq, (int)(nq + nk));
}

#define LSR_QK_INSTANTIATE(T)                                                              \
    template cudaError_t launch_qk_fw<T>(QkSide<T>, QkSide<T>, QkRope, cudaStream_t);       \
    template cudaError_t launch_qk_bw<T>(QkSide<T>, QkSide<T>, QkRope, float *, cudaStream_t);

}  // namespace lsr
