// launch.h -- internal C++ launchers behind the C ABI (one instantiation per
// storage dtype, compiled in its own translation unit).  Arguments have been
// validated by the ABI layer; `vec` says whether every tensor of the call is
// 16-byte aligned with a row length in bytes that is a multiple of 16.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace lsr {

// Rows per partial-sum chunk of the gamma/beta reduction, and the chunk count.
// Chosen so that column tiles x chunks gives roughly 1024 blocks; depends only
// on (rows, hidden), never on the GPU, so the summation order is fixed.
int64_t dgdb_rows_per_chunk(int64_t rows, int64_t hidden);
int64_t dgdb_num_chunks(int64_t rows, int64_t hidden);

// Number of SMs of the current device (cached per device).
int device_sm_count();

// qoff = Tk - Tq: a causal row sees keys j <= (query index) + qoff.  scale
// (> 0) multiplies the scores before the mask is added (1 for plain softmax).
template <typename T>
cudaError_t launch_softmax_fw(T *out, const T *inp, const T *mask, int64_t rows,
                              int64_t rows_per_batch, int64_t Tq, int64_t Tk,
                              int causal, int64_t qoff, float scale, bool vec, cudaStream_t st);
template <typename T>
cudaError_t launch_softmax_bw_masked(T *dinp, const T *dout, const T *y, const T *mask,
                                     int64_t rows, int64_t rows_per_batch, int64_t Tq,
                                     int64_t Tk, int causal, int64_t qoff, float scale, bool vec,
                                     cudaStream_t st);
template <typename T>
cudaError_t launch_softmax_bw(T *dinp, const T *dout, const T *y, int64_t rows,
                              int64_t Tk, bool vec, cudaStream_t st);
template <typename T>
cudaError_t launch_ln_fw(T *y, float *mean, float *rstd, const T *x, const T *gamma,
                         const T *beta, int64_t rows, int64_t N, float eps, bool vec,
                         cudaStream_t st);
template <typename T>
cudaError_t launch_ln_dinp(T *dx, const T *dy, const T *x, const T *gamma,
                           const float *mean, const float *rstd, int64_t rows,
                           int64_t N, bool vec, cudaStream_t st);
template <typename T>
cudaError_t launch_ln_dgdb(float *dgamma, float *dbeta, const T *dy, const T *x,
                           const float *mean, const float *rstd, int64_t rows,
                           int64_t N, float *part, bool vec, cudaStream_t st);

// Partial-sum slots the fused LayerNorm backward may use for `rows` rows:
// one per row chunk, at most 456.
int64_t ln_bw_fused_max_parts(int64_t rows);

// Fused LayerNorm backward: dx, dgamma, dbeta from one read of dy and x.
template <typename T>
cudaError_t launch_ln_bw_fused(T *dx, float *dgamma, float *dbeta, const T *dy, const T *x,
                               const T *gamma, const float *mean, const float *rstd,
                               int64_t rows, int64_t N, float *part, bool vec, cudaStream_t st);

// RMSNorm (no mean, no beta): forward, input gradient, gamma gradient.
template <typename T>
cudaError_t launch_rms_fw(T *y, float *rstd, const T *x, const T *gamma, int64_t rows, int64_t N,
                          float eps, bool vec, cudaStream_t st);
template <typename T>
cudaError_t launch_rms_dinp(T *dx, const T *dy, const T *x, const T *gamma, const float *rstd,
                            int64_t rows, int64_t N, bool vec, cudaStream_t st);
template <typename T>
cudaError_t launch_rms_dgamma(float *dgamma, const T *dy, const T *x, const float *rstd,
                              int64_t rows, int64_t N, float *part, bool vec, cudaStream_t st);

// Softmax cross entropy over a vocabulary (forward: loss and log-sum-exp per
// row; backward: dz from the saved log-sum-exp).  vec: take 16-byte vectors
// for the aligned middle of each row (the backward needs z and dz at the same
// offset modulo 16 bytes).
template <typename T>
cudaError_t launch_ce_fw(float *loss, float *lse, const T *z, const int32_t *target, int64_t rows,
                         int64_t V, bool vec, cudaStream_t st);
template <typename T>
cudaError_t launch_ce_bw(T *dz, const T *z, const int32_t *target, const float *lse,
                         const float *dloss, int64_t rows, int64_t V, bool vec, cudaStream_t st);

// Softmax with a relative position bias: the problem and its cut into runs of
// `per` rows in head-major order (h, b, i), one run per block.
struct RelposShape {
    int64_t rows_per_head;  // B * Tq
    int64_t rows;           // H * B * Tq
    int64_t per;            // rows of a block's run
    int64_t H, Tq, Tk, qoff;
    int64_t num_buckets;
    int R;
    int causal;
    float scale;
};

constexpr int kRelposMaxDistance = 2048;
// Workspace slots of 2R + 1 floats that the backward may use.
int64_t relpos_bw_slots(int64_t H);
template <typename T>
cudaError_t launch_relpos_fw(T *out, const T *inp, const T *mask, const T *table,
                             const int32_t *bucket, RelposShape p, cudaStream_t st);
template <typename T>
cudaError_t launch_relpos_bw(T *dinp, float *dtable, const T *dout, const T *y, const T *mask,
                             const int32_t *bucket, RelposShape p, float *part,
                             cudaStream_t st);

// Per-head norm of queries and keys with the position rotation.  One side
// (queries or keys) of a call: x and out are [tokens, heads, D] with a stride
// between tokens.
template <typename T>
struct QkSide {
    T *out;            // forward: the rotated norm; backward: dx
    const T *x;        // forward input
    const T *dout;     // backward only
    const T *gamma;    // [D]
    float *rstd_out;   // forward: written unless NULL
    const float *rstd;  // backward: as saved
    float *dgamma;     // backward
    int64_t heads, x_stride, out_stride, dout_stride;
};
struct QkRope {
    const float *cos, *sin;    // [max_pos, rot / 2]
    const int32_t *positions;  // [tokens]
    int64_t tokens, max_pos;
    int D, rot, interleaved;
    float eps;
};
constexpr int kQkMaxHeadDim = 1024;
// Blocks of the backward, each with one partial gamma gradient of D floats.
int64_t qk_bw_parts(int64_t tokens, int64_t Hq, int64_t Hk);
template <typename T>
cudaError_t launch_qk_fw(QkSide<T> q, QkSide<T> k, QkRope r, cudaStream_t st);
template <typename T>
cudaError_t launch_qk_bw(QkSide<T> q, QkSide<T> k, QkRope r, float *part, cudaStream_t st);

// Global norm of many tensors, and the tensors times min(1, max_norm / (norm
// + eps)); host arrays of `count` entries; dts holds ls_dtype codes.
int64_t grad_parts(int64_t count);
cudaError_t launch_grad_norm(float *norm, const void *const *grads, const int64_t *sizes,
                             const int32_t *dts, int64_t count, double *part, cudaStream_t st);
cudaError_t launch_grad_clip(float *norm, void *const *out, const void *const *grads,
                             const int64_t *sizes, const int32_t *dts, int64_t count,
                             float max_norm, float eps, double *part, cudaStream_t st);

// Difference of two attention softmax maps with a learned weight.
struct DiffShape {
    int64_t rows;  // B * H * Tq, in the order (b, h, i)
    int64_t per;   // rows of a block's run
    int64_t B, H, Tq, Tk, qoff;
    int lam_step;  // 1: a weight per head, 0: one for all
    int causal;
    float scale;
};
// Where a tensor's rows lie: element offset b * batch + h * head + i * Tk.
template <typename T>
struct DiffRows {
    T *p;
    int64_t batch, head;
    int64_t extent;  // elements from the first to past the last
    __device__ __forceinline__ int64_t at(int64_t b, int64_t h, int64_t i, int64_t Tk) const {
        return b * batch + h * head + i * Tk;
    }
};
template <typename T>
cudaError_t launch_diff_fw(T *out, float4 *stats, DiffRows<const T> x1, DiffRows<const T> x2,
                           const float *lam, const T *mask, DiffShape p, cudaStream_t st);
// row_dot: workspace of a float per row.
template <typename T>
cudaError_t launch_diff_bw(DiffRows<T> dx1, DiffRows<T> dx2, float *dlam, const T *dout,
                           DiffRows<const T> x1, DiffRows<const T> x2, const float *lam,
                           const float4 *stats, const T *mask, DiffShape p, float *row_dot,
                           cudaStream_t st);

// Norms after and before a block with its gate and residual scale.
template <typename T>
struct BlockNorm {
    int64_t rows, hidden, gates, gate_rows;  // gate_rows: rows that share a gate
    float residual_scale, eps;
    int layer;  // LayerNorm, else RMSNorm
    const T *x, *r, *gate, *gamma_post, *beta_post, *gamma_pre, *beta_pre;
    float *stats;  // [4][rows]: mean and rstd after, mean and rstd before the next block
    T *h, *y;      // forward
    // backward
    const T *dy, *dh, *h_in;
    const float *stats_in;
    T *dx, *dr;
    float *dgate, *dgamma_post, *dbeta_post, *dgamma_pre, *dbeta_pre;
};
constexpr int kBlockNormMaxHidden = 16384;
template <typename T>
cudaError_t launch_block_norm_fw(const BlockNorm<T> &a, cudaStream_t st);
template <typename T>
cudaError_t launch_block_norm_bw(const BlockNorm<T> &a, float *part, cudaStream_t st);
// Bytes of the backward's workspace (gates: 0 without a gate).
template <typename T>
size_t block_norm_workspace(int64_t rows, int64_t hidden, int64_t gates, bool layer);

// Softmax cross entropy from hidden states x [rows, D] and a vocabulary matrix
// w [V, D] (es: bytes of an element), and its gradients (dw may be NULL).
size_t linear_ce_workspace(bool backward, int64_t rows, int64_t D, int64_t V, size_t es);
template <typename T>
cudaError_t launch_linear_ce_fw(float *loss, float *lse, const T *x, const T *w,
                                const int32_t *target, int64_t rows, int64_t D, int64_t V,
                                void *workspace, cudaStream_t st);
template <typename T>
cudaError_t launch_linear_ce_bw(T *dx, T *dw, const T *x, const T *w, const int32_t *target,
                                const float *lse, const float *dloss, int64_t rows, int64_t D,
                                int64_t V, void *workspace, cudaStream_t st);

}  // namespace lsr
