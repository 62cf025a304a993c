// qk_norm_rope.cu -- launchers and instantiations of the per-head query / key
// norm with the position rotation, for every storage dtype.
#include "qk_norm_rope.cuh"
#include "dispatch.cuh"

namespace lsr {

// Blocks of the backward, a constant (not the device's SM count), so that the
// order of the gamma gradient's sums depends only on the problem.
constexpr int64_t kQkBwBlocks = 4 * 152;

// Blocks of the query and key sides, in proportion to their rows, each side
// with at most one block per row.
static void qk_bw_split(int64_t tokens, int64_t Hq, int64_t Hk, int64_t &nq, int64_t &nk) {
    const int64_t heads = Hq + Hk;
    nq = heads ? kQkBwBlocks * Hq / heads : 0;
    nk = heads ? kQkBwBlocks - nq : 0;
    if (Hq > 0 && nq < 1) nq = 1;
    if (Hk > 0 && nk < 1) nk = 1;
    if (nq > tokens * Hq) nq = tokens * Hq;
    if (nk > tokens * Hk) nk = tokens * Hk;
}

int64_t qk_bw_parts(int64_t tokens, int64_t Hq, int64_t Hk) {
    if (tokens <= 0) return 0;
    int64_t nq, nk;
    qk_bw_split(tokens, Hq, Hk, nq, nk);
    return nq + nk;
}

template <typename T>
cudaError_t launch_qk_fw(QkSide<T> q, QkSide<T> k, QkRope r, cudaStream_t st) {
    const int64_t rows = r.tokens * (q.heads + k.heads);
    return launch_persistent<qk_fw_loop<T>>(256, 0, ceil_div(rows, 8), st, q, k, r);
}

template <typename T>
cudaError_t launch_qk_bw(QkSide<T> q, QkSide<T> k, QkRope r, float *part, cudaStream_t st) {
    int64_t nq = 0, nk = 0;
    if (r.tokens > 0) {
        qk_bw_split(r.tokens, q.heads, k.heads, nq, nk);
        const cudaError_t e =
            launch_pdl(qk_bw_loop<T>, dim3((unsigned)(nq + nk)), dim3(256),
                       (size_t)8 * r.D * 4, st, q, k, r, part, (int)nq);
        if (e != cudaSuccess) return e;
    }
    return launch_pdl(qk_fold, dim3((unsigned)ceil_div(r.D, 32), 2), dim3(256), 0, st, q.dgamma,
                      k.dgamma, (const float *)part, r.D, (int)nq, (int)(nq + nk));
}

#define LSR_QK_INSTANTIATE(T)                                                              \
    template cudaError_t launch_qk_fw<T>(QkSide<T>, QkSide<T>, QkRope, cudaStream_t);       \
    template cudaError_t launch_qk_bw<T>(QkSide<T>, QkSide<T>, QkRope, float *, cudaStream_t);
LSR_QK_INSTANTIATE(float)
LSR_QK_INSTANTIATE(__half)
LSR_QK_INSTANTIATE(__nv_bfloat16)
#undef LSR_QK_INSTANTIATE

}  // namespace lsr
