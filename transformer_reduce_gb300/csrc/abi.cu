// abi.cu -- the extern "C" entry points of libls_reduce.so (declared and
// documented in include/ls_reduce.h).  This layer validates every argument on
// the host, picks the storage dtype and the vector/scalar path, and enqueues
// the kernels on the caller's stream.  It never allocates, frees or
// synchronises.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cmath>

#include "launch.h"
#include "ls_reduce.h"

namespace lsr {

int64_t dgdb_rows_per_chunk(int64_t rows, int64_t hidden) {
    // At most about 456 blocks (256-column tiles x row chunks): three
    // resident blocks on each of a GB300's 152 SMs, one wave with no partial
    // second wave.  A constant, not the device's SM count, so the summation
    // order depends only on (rows, hidden).
    if (rows <= 0 || hidden <= 0) return 1;
    const int64_t tiles = (hidden + 255) / 256;
    const int64_t target_chunks = tiles < 456 ? 456 / tiles : 1;
    int64_t rpc = (rows + target_chunks - 1) / target_chunks;
    if (rpc < 16) rpc = 16;
    while ((rows + rpc - 1) / rpc > 65535) rpc *= 2;
    return rpc;
}

int64_t dgdb_num_chunks(int64_t rows, int64_t hidden) {
    if (rows <= 0 || hidden <= 0) return 0;
    const int64_t rpc = dgdb_rows_per_chunk(rows, hidden);
    return (rows + rpc - 1) / rpc;
}

int64_t ln_bw_fused_max_parts(int64_t rows) {
    // 456 chunks is the most any bucket uses (fewer chunks of more rows never
    // need more slots); one slot per chunk
    if (rows <= 0) return 0;
    const int64_t rpc = (rows + 455) / 456;
    return (rows + rpc - 1) / rpc;
}

int device_sm_count() {
    constexpr int kMaxDev = 64;
    static std::atomic<int> cache[kMaxDev];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0) return 1;
    if (dev < kMaxDev) {
        int v = cache[dev].load(std::memory_order_relaxed);
        if (v > 0) return v;
    }
    int n = 1;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n < 1)
        n = 1;
    if (dev < kMaxDev) cache[dev].store(n, std::memory_order_relaxed);
    return n;
}

}  // namespace lsr

namespace {

size_t elem_size(ls_dtype dt) {
    switch (dt) {
        case LS_F32: return 4;
        case LS_F16: return 2;
        case LS_BF16: return 2;
    }
    return 0;
}

bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// 16-byte vector path: every tensor 16-byte aligned and rows a whole number of
// 16-byte chunks (so every row starts on a 16-byte boundary too).
bool vec_ok(int64_t row_len, size_t es, std::initializer_list<const void *> ptrs) {
    if ((row_len * (int64_t)es) % 16 != 0) return false;
    for (const void *p : ptrs)
        if (p && !aligned(p, 16)) return false;
    return true;
}

ls_status from_cuda(cudaError_t e) { return e == cudaSuccess ? LS_OK : LS_ERR_CUDA; }

// One side (queries or keys) of the per-head norm with its typed pointers.
template <typename T>
lsr::QkSide<T> qk_side(void *out, const void *x, const void *dout, const void *gamma,
                              float *rstd_out, const float *rstd, float *dgamma, int64_t heads,
                              int64_t x_stride, int64_t out_stride, int64_t dout_stride) {
    lsr::QkSide<T> s = {};
    s.out = static_cast<T *>(out);
    s.x = static_cast<const T *>(x);
    s.dout = static_cast<const T *>(dout);
    s.gamma = static_cast<const T *>(gamma);
    s.rstd_out = rstd_out;
    s.rstd = rstd;
    s.dgamma = dgamma;
    s.heads = heads;
    s.x_stride = x_stride;
    s.out_stride = out_stride;
    s.dout_stride = dout_stride;
    return s;
}

}  // namespace

extern "C" {

const char *ls_status_string(ls_status s) {
    switch (s) {
        case LS_OK: return "LS_OK";
        case LS_ERR_INVALID_ARG: return "LS_ERR_INVALID_ARG: null pointer, negative size, inconsistent shape or overlapping outputs";
        case LS_ERR_UNSUPPORTED: return "LS_ERR_UNSUPPORTED: unknown dtype or size beyond the library limits";
        case LS_ERR_MISALIGNED: return "LS_ERR_MISALIGNED: pointer not aligned to its element size";
        case LS_ERR_WORKSPACE: return "LS_ERR_WORKSPACE: workspace missing, too small or not 16-byte aligned";
        case LS_ERR_CUDA: return "LS_ERR_CUDA: the CUDA runtime rejected a launch";
    }
    return "unknown ls_status";
}

static ls_status softmax_fw_impl(void *out, const void *inp, const void *mask, int64_t B,
                                 int64_t H, int64_t Tq, int64_t Tk, int causal, float scale,
                                 ls_dtype dt, void *stream) {
    const size_t es = elem_size(dt);
    if (es == 0) return LS_ERR_UNSUPPORTED;
    if (B < 0 || H < 0 || Tq < 0 || Tk < 0) return LS_ERR_INVALID_ARG;
    if (causal && Tq > Tk) return LS_ERR_INVALID_ARG;
    if (Tk > LS_MAX_ROW_LENGTH) return LS_ERR_UNSUPPORTED;
    if (B == 0 || H == 0 || Tq == 0 || Tk == 0) return LS_OK;
    if (!out || !inp) return LS_ERR_INVALID_ARG;
    if (H > INT64_MAX / B || Tq > INT64_MAX / (B * H) || Tk > INT64_MAX / (B * H * Tq))
        return LS_ERR_UNSUPPORTED;
    if (!aligned(out, es) || !aligned(inp, es) || (mask && !aligned(mask, es)))
        return LS_ERR_MISALIGNED;
    const int64_t rows = B * H * Tq;
    const bool vec = vec_ok(Tk, es, {out, inp, mask});
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    switch (dt) {
        case LS_F32:
            return from_cuda(lsr::launch_softmax_fw<float>(
                (float *)out, (const float *)inp, (const float *)mask, rows, H * Tq, Tq, Tk,
                causal ? 1 : 0, Tk - Tq, scale, vec, st));
        case LS_F16:
            return from_cuda(lsr::launch_softmax_fw<__half>(
                (__half *)out, (const __half *)inp, (const __half *)mask, rows, H * Tq, Tq, Tk,
                causal ? 1 : 0, Tk - Tq, scale, vec, st));
        case LS_BF16:
            return from_cuda(lsr::launch_softmax_fw<__nv_bfloat16>(
                (__nv_bfloat16 *)out, (const __nv_bfloat16 *)inp, (const __nv_bfloat16 *)mask,
                rows, H * Tq, Tq, Tk, causal ? 1 : 0, Tk - Tq, scale, vec, st));
    }
    return LS_ERR_UNSUPPORTED;
}

static bool scale_ok(float scale) { return std::isfinite(scale) && scale > 0.f; }

ls_status ls_softmax_fw(void *out, const void *inp, const void *mask, int64_t B, int64_t H,
                        int64_t Tq, int64_t Tk, int causal, ls_dtype dt, void *stream) {
    return softmax_fw_impl(out, inp, mask, B, H, Tq, Tk, causal, 1.0f, dt, stream);
}

ls_status ls_softmax_fw_scaled(void *out, const void *inp, const void *mask, int64_t B,
                               int64_t H, int64_t Tq, int64_t Tk, int causal, float scale,
                               ls_dtype dt, void *stream) {
    if (elem_size(dt) == 0) return LS_ERR_UNSUPPORTED;
    if (!scale_ok(scale)) return LS_ERR_INVALID_ARG;
    return softmax_fw_impl(out, inp, mask, B, H, Tq, Tk, causal, scale, dt, stream);
}

ls_status ls_softmax_bw(void *dinp, const void *dout, const void *out_fw, int64_t B, int64_t H,
                        int64_t Tq, int64_t Tk, ls_dtype dt, void *stream) {
    const size_t es = elem_size(dt);
    if (es == 0) return LS_ERR_UNSUPPORTED;
    if (B < 0 || H < 0 || Tq < 0 || Tk < 0) return LS_ERR_INVALID_ARG;
    if (Tk > LS_MAX_ROW_LENGTH) return LS_ERR_UNSUPPORTED;
    if (B == 0 || H == 0 || Tq == 0 || Tk == 0) return LS_OK;
    if (!dinp || !dout || !out_fw) return LS_ERR_INVALID_ARG;
    if (H > INT64_MAX / B || Tq > INT64_MAX / (B * H) || Tk > INT64_MAX / (B * H * Tq))
        return LS_ERR_UNSUPPORTED;
    if (!aligned(dinp, es) || !aligned(dout, es) || !aligned(out_fw, es))
        return LS_ERR_MISALIGNED;
    const int64_t rows = B * H * Tq;
    const bool vec = vec_ok(Tk, es, {dinp, dout, out_fw});
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    switch (dt) {
        case LS_F32:
            return from_cuda(lsr::launch_softmax_bw<float>(
                (float *)dinp, (const float *)dout, (const float *)out_fw, rows, Tk, vec, st));
        case LS_F16:
            return from_cuda(lsr::launch_softmax_bw<__half>(
                (__half *)dinp, (const __half *)dout, (const __half *)out_fw, rows, Tk, vec, st));
        case LS_BF16:
            return from_cuda(lsr::launch_softmax_bw<__nv_bfloat16>(
                (__nv_bfloat16 *)dinp, (const __nv_bfloat16 *)dout,
                (const __nv_bfloat16 *)out_fw, rows, Tk, vec, st));
    }
    return LS_ERR_UNSUPPORTED;
}

static ls_status softmax_bw_masked_impl(void *dinp, const void *dout, const void *out_fw,
                                        const void *mask, int64_t B, int64_t H, int64_t Tq,
                                        int64_t Tk, int causal, float scale, ls_dtype dt,
                                        void *stream) {
    const size_t es = elem_size(dt);
    if (es == 0) return LS_ERR_UNSUPPORTED;
    if (B < 0 || H < 0 || Tq < 0 || Tk < 0) return LS_ERR_INVALID_ARG;
    if (causal && Tq > Tk) return LS_ERR_INVALID_ARG;
    if (Tk > LS_MAX_ROW_LENGTH) return LS_ERR_UNSUPPORTED;
    if (B == 0 || H == 0 || Tq == 0 || Tk == 0) return LS_OK;
    if (!dinp || !dout || !out_fw) return LS_ERR_INVALID_ARG;
    if (H > INT64_MAX / B || Tq > INT64_MAX / (B * H) || Tk > INT64_MAX / (B * H * Tq))
        return LS_ERR_UNSUPPORTED;
    if (!aligned(dinp, es) || !aligned(dout, es) || !aligned(out_fw, es) ||
        (mask && !aligned(mask, es)))
        return LS_ERR_MISALIGNED;
    const int64_t rows = B * H * Tq;
    const bool vec = vec_ok(Tk, es, {dinp, dout, out_fw, mask});
    const int c = causal ? 1 : 0;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    switch (dt) {
        case LS_F32:
            return from_cuda(lsr::launch_softmax_bw_masked<float>(
                (float *)dinp, (const float *)dout, (const float *)out_fw, (const float *)mask,
                rows, H * Tq, Tq, Tk, c, Tk - Tq, scale, vec, st));
        case LS_F16:
            return from_cuda(lsr::launch_softmax_bw_masked<__half>(
                (__half *)dinp, (const __half *)dout, (const __half *)out_fw,
                (const __half *)mask, rows, H * Tq, Tq, Tk, c, Tk - Tq, scale, vec, st));
        case LS_BF16:
            return from_cuda(lsr::launch_softmax_bw_masked<__nv_bfloat16>(
                (__nv_bfloat16 *)dinp, (const __nv_bfloat16 *)dout,
                (const __nv_bfloat16 *)out_fw, (const __nv_bfloat16 *)mask, rows, H * Tq, Tq,
                Tk, c, Tk - Tq, scale, vec, st));
    }
    return LS_ERR_UNSUPPORTED;
}

ls_status ls_softmax_bw_masked(void *dinp, const void *dout, const void *out_fw,
                               const void *mask, int64_t B, int64_t H, int64_t Tq, int64_t Tk,
                               int causal, ls_dtype dt, void *stream) {
    return softmax_bw_masked_impl(dinp, dout, out_fw, mask, B, H, Tq, Tk, causal, 1.0f, dt,
                                  stream);
}

ls_status ls_softmax_bw_masked_scaled(void *dinp, const void *dout, const void *out_fw,
                                      const void *mask, int64_t B, int64_t H, int64_t Tq,
                                      int64_t Tk, int causal, float scale, ls_dtype dt,
                                      void *stream) {
    if (elem_size(dt) == 0) return LS_ERR_UNSUPPORTED;
    if (!scale_ok(scale)) return LS_ERR_INVALID_ARG;
    return softmax_bw_masked_impl(dinp, dout, out_fw, mask, B, H, Tq, Tk, causal, scale, dt,
                                  stream);
}

// Shared checks of the LayerNorm entry points.
static ls_status ln_check(int64_t rows, int64_t hidden, size_t es) {
    if (es == 0) return LS_ERR_UNSUPPORTED;
    if (rows < 0 || hidden < 1) return LS_ERR_INVALID_ARG;
    if (hidden > LS_MAX_ROW_LENGTH) return LS_ERR_UNSUPPORTED;
    if (rows > 0 && hidden > INT64_MAX / rows) return LS_ERR_UNSUPPORTED;
    return LS_OK;
}

ls_status ls_layernorm_fw(void *y, float *mean, float *rstd, const void *x, const void *gamma,
                          const void *beta, int64_t rows, int64_t hidden, float eps,
                          ls_dtype dt, void *stream) {
    const size_t es = elem_size(dt);
    ls_status s = ln_check(rows, hidden, es);
    if (s != LS_OK) return s;
    if (!(eps >= 0.f) || !std::isfinite(eps)) return LS_ERR_INVALID_ARG;
    if (rows == 0) return LS_OK;
    if (!y || !mean || !rstd || !x || !gamma || !beta) return LS_ERR_INVALID_ARG;
    if (!aligned(y, es) || !aligned(x, es) || !aligned(gamma, es) || !aligned(beta, es) ||
        !aligned(mean, 4) || !aligned(rstd, 4))
        return LS_ERR_MISALIGNED;
    const bool vec = vec_ok(hidden, es, {y, x, gamma, beta});
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    switch (dt) {
        case LS_F32:
            return from_cuda(lsr::launch_ln_fw<float>((float *)y, mean, rstd, (const float *)x,
                                                      (const float *)gamma, (const float *)beta,
                                                      rows, hidden, eps, vec, st));
        case LS_F16:
            return from_cuda(lsr::launch_ln_fw<__half>(
                (__half *)y, mean, rstd, (const __half *)x, (const __half *)gamma,
                (const __half *)beta, rows, hidden, eps, vec, st));
        case LS_BF16:
            return from_cuda(lsr::launch_ln_fw<__nv_bfloat16>(
                (__nv_bfloat16 *)y, mean, rstd, (const __nv_bfloat16 *)x,
                (const __nv_bfloat16 *)gamma, (const __nv_bfloat16 *)beta, rows, hidden, eps,
                vec, st));
    }
    return LS_ERR_UNSUPPORTED;
}

ls_status ls_layernorm_bw_dinp(void *dx, const void *dy, const void *x, const void *gamma,
                               const float *mean, const float *rstd, int64_t rows,
                               int64_t hidden, ls_dtype dt, void *stream) {
    const size_t es = elem_size(dt);
    ls_status s = ln_check(rows, hidden, es);
    if (s != LS_OK) return s;
    if (rows == 0) return LS_OK;
    if (!dx || !dy || !x || !gamma || !mean || !rstd) return LS_ERR_INVALID_ARG;
    if (!aligned(dx, es) || !aligned(dy, es) || !aligned(x, es) || !aligned(gamma, es) ||
        !aligned(mean, 4) || !aligned(rstd, 4))
        return LS_ERR_MISALIGNED;
    const bool vec = vec_ok(hidden, es, {dx, dy, x, gamma});
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    switch (dt) {
        case LS_F32:
            return from_cuda(lsr::launch_ln_dinp<float>((float *)dx, (const float *)dy,
                                                        (const float *)x, (const float *)gamma,
                                                        mean, rstd, rows, hidden, vec, st));
        case LS_F16:
            return from_cuda(lsr::launch_ln_dinp<__half>((__half *)dx, (const __half *)dy,
                                                         (const __half *)x,
                                                         (const __half *)gamma, mean, rstd,
                                                         rows, hidden, vec, st));
        case LS_BF16:
            return from_cuda(lsr::launch_ln_dinp<__nv_bfloat16>(
                (__nv_bfloat16 *)dx, (const __nv_bfloat16 *)dy, (const __nv_bfloat16 *)x,
                (const __nv_bfloat16 *)gamma, mean, rstd, rows, hidden, vec, st));
    }
    return LS_ERR_UNSUPPORTED;
}

ls_status ls_rmsnorm_fw(void *y, float *rstd, const void *x, const void *gamma, int64_t rows,
                        int64_t hidden, float eps, ls_dtype dt, void *stream) {
    const size_t es = elem_size(dt);
    ls_status s = ln_check(rows, hidden, es);
    if (s != LS_OK) return s;
    if (!(eps >= 0.f) || !std::isfinite(eps)) return LS_ERR_INVALID_ARG;
    if (rows == 0) return LS_OK;
    if (!y || !rstd || !x || !gamma) return LS_ERR_INVALID_ARG;
    if (!aligned(y, es) || !aligned(x, es) || !aligned(gamma, es) || !aligned(rstd, 4))
        return LS_ERR_MISALIGNED;
    const bool vec = vec_ok(hidden, es, {y, x, gamma});
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    switch (dt) {
        case LS_F32:
            return from_cuda(lsr::launch_rms_fw<float>((float *)y, rstd, (const float *)x,
                                                       (const float *)gamma, rows, hidden, eps,
                                                       vec, st));
        case LS_F16:
            return from_cuda(lsr::launch_rms_fw<__half>((__half *)y, rstd, (const __half *)x,
                                                        (const __half *)gamma, rows, hidden, eps,
                                                        vec, st));
        case LS_BF16:
            return from_cuda(lsr::launch_rms_fw<__nv_bfloat16>(
                (__nv_bfloat16 *)y, rstd, (const __nv_bfloat16 *)x, (const __nv_bfloat16 *)gamma,
                rows, hidden, eps, vec, st));
    }
    return LS_ERR_UNSUPPORTED;
}

ls_status ls_rmsnorm_bw_dinp(void *dx, const void *dy, const void *x, const void *gamma,
                             const float *rstd, int64_t rows, int64_t hidden, ls_dtype dt,
                             void *stream) {
    const size_t es = elem_size(dt);
    ls_status s = ln_check(rows, hidden, es);
    if (s != LS_OK) return s;
    if (rows == 0) return LS_OK;
    if (!dx || !dy || !x || !gamma || !rstd) return LS_ERR_INVALID_ARG;
    if (!aligned(dx, es) || !aligned(dy, es) || !aligned(x, es) || !aligned(gamma, es) ||
        !aligned(rstd, 4))
        return LS_ERR_MISALIGNED;
    const bool vec = vec_ok(hidden, es, {dx, dy, x, gamma});
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    switch (dt) {
        case LS_F32:
            return from_cuda(lsr::launch_rms_dinp<float>((float *)dx, (const float *)dy,
                                                         (const float *)x, (const float *)gamma,
                                                         rstd, rows, hidden, vec, st));
        case LS_F16:
            return from_cuda(lsr::launch_rms_dinp<__half>((__half *)dx, (const __half *)dy,
                                                          (const __half *)x,
                                                          (const __half *)gamma, rstd, rows,
                                                          hidden, vec, st));
        case LS_BF16:
            return from_cuda(lsr::launch_rms_dinp<__nv_bfloat16>(
                (__nv_bfloat16 *)dx, (const __nv_bfloat16 *)dy, (const __nv_bfloat16 *)x,
                (const __nv_bfloat16 *)gamma, rstd, rows, hidden, vec, st));
    }
    return LS_ERR_UNSUPPORTED;
}

ls_status ls_rmsnorm_bw_dgamma(float *dgamma, const void *dy, const void *x, const float *rstd,
                               int64_t rows, int64_t hidden, void *workspace,
                               size_t workspace_bytes, ls_dtype dt, void *stream) {
    const size_t es = elem_size(dt);
    ls_status s = ln_check(rows, hidden, es);
    if (s != LS_OK) return s;
    if (!dgamma) return LS_ERR_INVALID_ARG;
    if (rows > 0 && (!dy || !x || !rstd)) return LS_ERR_INVALID_ARG;
    if (!aligned(dgamma, 4) || (dy && !aligned(dy, es)) || (x && !aligned(x, es)) ||
        (rstd && !aligned(rstd, 4)))
        return LS_ERR_MISALIGNED;
    const size_t need = ls_layernorm_bw_dgamma_dbeta_workspace_size(rows, hidden);
    if (need > 0 && (!workspace || workspace_bytes < need || !aligned(workspace, 16)))
        return LS_ERR_WORKSPACE;
    const bool vec = vec_ok(hidden, es, {dy, x});
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    float *part = static_cast<float *>(workspace);
    switch (dt) {
        case LS_F32:
            return from_cuda(lsr::launch_rms_dgamma<float>(dgamma, (const float *)dy,
                                                           (const float *)x, rstd, rows, hidden,
                                                           part, vec, st));
        case LS_F16:
            return from_cuda(lsr::launch_rms_dgamma<__half>(dgamma, (const __half *)dy,
                                                            (const __half *)x, rstd, rows, hidden,
                                                            part, vec, st));
        case LS_BF16:
            return from_cuda(lsr::launch_rms_dgamma<__nv_bfloat16>(
                dgamma, (const __nv_bfloat16 *)dy, (const __nv_bfloat16 *)x, rstd, rows, hidden,
                part, vec, st));
    }
    return LS_ERR_UNSUPPORTED;
}

size_t ls_layernorm_bw_workspace_size(int64_t rows, int64_t hidden) {
    if (rows <= 0 || hidden <= 0) return 0;
    const size_t fused = (size_t)lsr::ln_bw_fused_max_parts(rows) * 2u * (size_t)hidden * 4u;
    const size_t split = ls_layernorm_bw_dgamma_dbeta_workspace_size(rows, hidden);
    return fused > split ? fused : split;
}

ls_status ls_layernorm_bw(void *dx, float *dgamma, float *dbeta, const void *dy, const void *x,
                          const void *gamma, const float *mean, const float *rstd, int64_t rows,
                          int64_t hidden, void *workspace, size_t workspace_bytes, ls_dtype dt,
                          void *stream) {
    const size_t es = elem_size(dt);
    ls_status s = ln_check(rows, hidden, es);
    if (s != LS_OK) return s;
    if (!dgamma || !dbeta) return LS_ERR_INVALID_ARG;
    if (rows > 0 && (!dx || !dy || !x || !gamma || !mean || !rstd)) return LS_ERR_INVALID_ARG;
    if (!aligned(dgamma, 4) || !aligned(dbeta, 4) || (dx && !aligned(dx, es)) ||
        (dy && !aligned(dy, es)) || (x && !aligned(x, es)) || (gamma && !aligned(gamma, es)) ||
        (mean && !aligned(mean, 4)) || (rstd && !aligned(rstd, 4)))
        return LS_ERR_MISALIGNED;
    const size_t need = ls_layernorm_bw_workspace_size(rows, hidden);
    if (need > 0 && (!workspace || workspace_bytes < need || !aligned(workspace, 16)))
        return LS_ERR_WORKSPACE;
    const bool vec = vec_ok(hidden, es, {dx, dy, x, gamma});
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    float *part = static_cast<float *>(workspace);
    switch (dt) {
        case LS_F32:
            return from_cuda(lsr::launch_ln_bw_fused<float>(
                (float *)dx, dgamma, dbeta, (const float *)dy, (const float *)x,
                (const float *)gamma, mean, rstd, rows, hidden, part, vec, st));
        case LS_F16:
            return from_cuda(lsr::launch_ln_bw_fused<__half>(
                (__half *)dx, dgamma, dbeta, (const __half *)dy, (const __half *)x,
                (const __half *)gamma, mean, rstd, rows, hidden, part, vec, st));
        case LS_BF16:
            return from_cuda(lsr::launch_ln_bw_fused<__nv_bfloat16>(
                (__nv_bfloat16 *)dx, dgamma, dbeta, (const __nv_bfloat16 *)dy,
                (const __nv_bfloat16 *)x, (const __nv_bfloat16 *)gamma, mean, rstd, rows, hidden,
                part, vec, st));
    }
    return LS_ERR_UNSUPPORTED;
}

size_t ls_layernorm_bw_dgamma_dbeta_workspace_size(int64_t rows, int64_t hidden) {
    if (rows <= 0 || hidden <= 0) return 0;
    const int64_t nchunks = lsr::dgdb_num_chunks(rows, hidden);
    return (size_t)nchunks * 2u * (size_t)hidden * sizeof(float);
}

ls_status ls_layernorm_bw_dgamma_dbeta(float *dgamma, float *dbeta, const void *dy, const void *x,
                                       const float *mean, const float *rstd, int64_t rows,
                                       int64_t hidden, void *workspace, size_t workspace_bytes,
                                       ls_dtype dt, void *stream) {
    const size_t es = elem_size(dt);
    ls_status s = ln_check(rows, hidden, es);
    if (s != LS_OK) return s;
    if (!dgamma || !dbeta) return LS_ERR_INVALID_ARG;
    if (rows > 0 && (!dy || !x || !mean || !rstd)) return LS_ERR_INVALID_ARG;
    if (!aligned(dgamma, 4) || !aligned(dbeta, 4) || (dy && !aligned(dy, es)) ||
        (x && !aligned(x, es)) || (mean && !aligned(mean, 4)) || (rstd && !aligned(rstd, 4)))
        return LS_ERR_MISALIGNED;
    const size_t need = ls_layernorm_bw_dgamma_dbeta_workspace_size(rows, hidden);
    if (need > 0 && (!workspace || workspace_bytes < need || !aligned(workspace, 16)))
        return LS_ERR_WORKSPACE;
    const bool vec = vec_ok(hidden, es, {dy, x});
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    float *part = static_cast<float *>(workspace);
    switch (dt) {
        case LS_F32:
            return from_cuda(lsr::launch_ln_dgdb<float>(dgamma, dbeta, (const float *)dy,
                                                        (const float *)x, mean, rstd, rows,
                                                        hidden, part, vec, st));
        case LS_F16:
            return from_cuda(lsr::launch_ln_dgdb<__half>(dgamma, dbeta, (const __half *)dy,
                                                         (const __half *)x, mean, rstd, rows,
                                                         hidden, part, vec, st));
        case LS_BF16:
            return from_cuda(lsr::launch_ln_dgdb<__nv_bfloat16>(
                dgamma, dbeta, (const __nv_bfloat16 *)dy, (const __nv_bfloat16 *)x, mean, rstd,
                rows, hidden, part, vec, st));
    }
    return LS_ERR_UNSUPPORTED;
}

// ----------------------------------------------------------------------------
// cross entropy over a vocabulary
// ----------------------------------------------------------------------------
ls_status ls_cross_entropy_fw(float *loss, float *lse, const void *logits, const int32_t *target,
                              int64_t rows, int64_t vocab, ls_dtype dt, void *stream) {
    const size_t es = elem_size(dt);
    ls_status s = ln_check(rows, vocab, es);
    if (s != LS_OK) return s;
    if (rows > 0 && (!loss || !lse || !logits || !target)) return LS_ERR_INVALID_ARG;
    if ((loss && !aligned(loss, 4)) || (lse && !aligned(lse, 4)) ||
        (logits && !aligned(logits, es)) || (target && !aligned(target, 4)))
        return LS_ERR_MISALIGNED;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    // the aligned middle of every row is read in 16-byte vectors whatever the
    // row's start offset
    switch (dt) {
        case LS_F32:
            return from_cuda(lsr::launch_ce_fw<float>(loss, lse, (const float *)logits, target,
                                                      rows, vocab, true, st));
        case LS_F16:
            return from_cuda(lsr::launch_ce_fw<__half>(loss, lse, (const __half *)logits, target,
                                                       rows, vocab, true, st));
        case LS_BF16:
            return from_cuda(lsr::launch_ce_fw<__nv_bfloat16>(
                loss, lse, (const __nv_bfloat16 *)logits, target, rows, vocab, true, st));
    }
    return LS_ERR_UNSUPPORTED;
}

ls_status ls_cross_entropy_bw(void *dlogits, const void *logits, const int32_t *target,
                              const float *lse, const float *dloss, int64_t rows, int64_t vocab,
                              ls_dtype dt, void *stream) {
    const size_t es = elem_size(dt);
    ls_status s = ln_check(rows, vocab, es);
    if (s != LS_OK) return s;
    if (rows > 0 && (!dlogits || !logits || !target || !lse || !dloss)) return LS_ERR_INVALID_ARG;
    if ((dlogits && !aligned(dlogits, es)) || (logits && !aligned(logits, es)) ||
        (target && !aligned(target, 4)) || (lse && !aligned(lse, 4)) ||
        (dloss && !aligned(dloss, 4)))
        return LS_ERR_MISALIGNED;
    // vectors need logits and dlogits at the same offset within 16 bytes
    const bool vec =
        ((reinterpret_cast<uintptr_t>(dlogits) ^ reinterpret_cast<uintptr_t>(logits)) & 15u) == 0;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    switch (dt) {
        case LS_F32:
            return from_cuda(lsr::launch_ce_bw<float>((float *)dlogits, (const float *)logits,
                                                      target, lse, dloss, rows, vocab, vec, st));
        case LS_F16:
            return from_cuda(lsr::launch_ce_bw<__half>((__half *)dlogits, (const __half *)logits,
                                                       target, lse, dloss, rows, vocab, vec, st));
        case LS_BF16:
            return from_cuda(lsr::launch_ce_bw<__nv_bfloat16>(
                (__nv_bfloat16 *)dlogits, (const __nv_bfloat16 *)logits, target, lse, dloss, rows,
                vocab, vec, st));
    }
    return LS_ERR_UNSUPPORTED;
}

// ----------------------------------------------------------------------------
// softmax with a relative position bias
// ----------------------------------------------------------------------------
// Shared checks; sets `empty` when there is no score at all.
static ls_status relpos_check(int64_t B, int64_t H, int64_t Tq, int64_t Tk, int64_t num_buckets,
                              int64_t max_distance, int causal, float scale, bool *empty) {
    if (B < 0 || H < 0 || Tq < 0 || Tk < 0 || num_buckets < 1 || max_distance < 1)
        return LS_ERR_INVALID_ARG;
    if (!scale_ok(scale) || (causal && Tq > Tk)) return LS_ERR_INVALID_ARG;
    if (Tk > LS_MAX_ROW_LENGTH || Tq > LS_MAX_ROW_LENGTH ||
        max_distance > LS_MAX_RELPOS_DISTANCE || num_buckets > LS_MAX_RELPOS_BUCKETS ||
        H > INT32_MAX || H > INT64_MAX / 8 / num_buckets)
        return LS_ERR_UNSUPPORTED;
    *empty = B == 0 || H == 0 || Tq == 0 || Tk == 0;
    if (!*empty && (H > INT64_MAX / B || Tq > INT64_MAX / (B * H) || Tk > INT64_MAX / (B * H * Tq)))
        return LS_ERR_UNSUPPORTED;
    return LS_OK;
}

static lsr::RelposShape relpos_shape(int64_t B, int64_t H, int64_t Tq, int64_t Tk,
                                     int64_t num_buckets, int64_t max_distance, int causal,
                                     float scale, bool empty) {
    lsr::RelposShape p = {};
    p.rows_per_head = empty ? 0 : B * Tq;
    p.rows = empty ? 0 : B * Tq * H;
    p.per = 1;
    p.H = H;
    p.Tq = Tq;
    p.Tk = Tk;
    p.qoff = Tk - Tq;
    p.num_buckets = num_buckets;
    p.R = (int)max_distance;
    p.causal = causal ? 1 : 0;
    p.scale = scale;
    return p;
}

ls_status ls_softmax_fw_relpos(void *out, const void *inp, const void *mask, const void *table,
                               const int32_t *bucket, int64_t B, int64_t H, int64_t Tq,
                               int64_t Tk, int64_t num_buckets, int64_t max_distance, int causal,
                               float scale, ls_dtype dt, void *stream) {
    const size_t es = elem_size(dt);
    if (es == 0) return LS_ERR_UNSUPPORTED;
    bool empty = false;
    const ls_status s =
        relpos_check(B, H, Tq, Tk, num_buckets, max_distance, causal, scale, &empty);
    if (s != LS_OK) return s;
    if (empty) return LS_OK;
    if (!out || !inp || !table || !bucket) return LS_ERR_INVALID_ARG;
    if (!aligned(out, es) || !aligned(inp, es) || !aligned(table, es) || !aligned(bucket, 4) ||
        (mask && !aligned(mask, es)))
        return LS_ERR_MISALIGNED;
    const lsr::RelposShape p =
        relpos_shape(B, H, Tq, Tk, num_buckets, max_distance, causal, scale, empty);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    switch (dt) {
        case LS_F32:
            return from_cuda(lsr::launch_relpos_fw<float>((float *)out, (const float *)inp,
                                                          (const float *)mask,
                                                          (const float *)table, bucket, p, st));
        case LS_F16:
            return from_cuda(lsr::launch_relpos_fw<__half>((__half *)out, (const __half *)inp,
                                                           (const __half *)mask,
                                                           (const __half *)table, bucket, p, st));
        case LS_BF16:
            return from_cuda(lsr::launch_relpos_fw<__nv_bfloat16>(
                (__nv_bfloat16 *)out, (const __nv_bfloat16 *)inp, (const __nv_bfloat16 *)mask,
                (const __nv_bfloat16 *)table, bucket, p, st));
    }
    return LS_ERR_UNSUPPORTED;
}

size_t ls_softmax_bw_relpos_workspace_size(int64_t H, int64_t max_distance) {
    if (H <= 0 || max_distance <= 0 || max_distance > LS_MAX_RELPOS_DISTANCE || H > INT32_MAX)
        return 0;
    return (size_t)lsr::relpos_bw_slots(H) * (size_t)(2 * max_distance + 1) * sizeof(float);
}

ls_status ls_softmax_bw_relpos(void *dinp, float *dtable, const void *dout, const void *out_fw,
                               const void *mask, const int32_t *bucket, int64_t B, int64_t H,
                               int64_t Tq, int64_t Tk, int64_t num_buckets, int64_t max_distance,
                               int causal, float scale, void *workspace, size_t workspace_bytes,
                               ls_dtype dt, void *stream) {
    const size_t es = elem_size(dt);
    if (es == 0) return LS_ERR_UNSUPPORTED;
    bool empty = false;
    const ls_status s =
        relpos_check(B, H, Tq, Tk, num_buckets, max_distance, causal, scale, &empty);
    if (s != LS_OK) return s;
    if (H == 0) return LS_OK;
    if (!dtable || !bucket || (!empty && (!dinp || !dout || !out_fw))) return LS_ERR_INVALID_ARG;
    if ((dinp && !aligned(dinp, es)) || (dout && !aligned(dout, es)) ||
        (out_fw && !aligned(out_fw, es)) || (mask && !aligned(mask, es)) || !aligned(dtable, 4) ||
        !aligned(bucket, 4))
        return LS_ERR_MISALIGNED;
    const size_t need = ls_softmax_bw_relpos_workspace_size(H, max_distance);
    if (!empty && (!workspace || workspace_bytes < need || !aligned(workspace, 16)))
        return LS_ERR_WORKSPACE;
    const lsr::RelposShape p =
        relpos_shape(B, H, Tq, Tk, num_buckets, max_distance, causal, scale, empty);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    float *part = static_cast<float *>(workspace);
    switch (dt) {
        case LS_F32:
            return from_cuda(lsr::launch_relpos_bw<float>((float *)dinp, dtable,
                                                          (const float *)dout,
                                                          (const float *)out_fw,
                                                          (const float *)mask, bucket, p, part,
                                                          st));
        case LS_F16:
            return from_cuda(lsr::launch_relpos_bw<__half>(
                (__half *)dinp, dtable, (const __half *)dout, (const __half *)out_fw,
                (const __half *)mask, bucket, p, part, st));
        case LS_BF16:
            return from_cuda(lsr::launch_relpos_bw<__nv_bfloat16>(
                (__nv_bfloat16 *)dinp, dtable, (const __nv_bfloat16 *)dout,
                (const __nv_bfloat16 *)out_fw, (const __nv_bfloat16 *)mask, bucket, p, part, st));
    }
    return LS_ERR_UNSUPPORTED;
}

// ----------------------------------------------------------------------------
// per-head norm of queries and keys with the position rotation
// ----------------------------------------------------------------------------
static ls_status qk_check(int64_t tokens, int64_t Hq, int64_t Hk, int64_t D, int64_t rot,
                          int64_t max_pos, const float *cos, const float *sin,
                          const int32_t *positions) {
    if (tokens < 0 || Hq < 0 || Hk < 0 || D < 1 || rot < 0 || rot > D || rot % 2 != 0)
        return LS_ERR_INVALID_ARG;
    if (D > LS_MAX_HEAD_DIM || Hq > LS_MAX_HEADS || Hk > LS_MAX_HEADS) return LS_ERR_UNSUPPORTED;
    if (tokens > 0 && (Hq + Hk + 1) * D > INT64_MAX / tokens) return LS_ERR_UNSUPPORTED;
    if (rot > 0 && tokens > 0 && Hq + Hk > 0) {
        if (!cos || !sin || !positions || max_pos < 1) return LS_ERR_INVALID_ARG;
        if (max_pos > INT64_MAX / rot) return LS_ERR_UNSUPPORTED;
        if (!aligned(cos, 4) || !aligned(sin, 4) || !aligned(positions, 4))
            return LS_ERR_MISALIGNED;
    }
    return LS_OK;
}

// A tensor of one side: dense heads, tokens `stride` elements apart.
static ls_status qk_tensor(const void *p, int64_t tokens, int64_t heads, int64_t D,
                           int64_t stride, size_t es) {
    if (tokens == 0 || heads == 0) return LS_OK;
    if (!p || stride < heads * D) return LS_ERR_INVALID_ARG;
    if (stride > INT64_MAX / tokens) return LS_ERR_UNSUPPORTED;
    return aligned(p, es) ? LS_OK : LS_ERR_MISALIGNED;
}

// A tensor of `tokens` rows of `row` bytes, `stride` bytes apart.
struct QkSpan {
    uintptr_t at;
    int64_t row, stride;
};
static QkSpan qk_span(const void *p, int64_t heads, int64_t D, int64_t stride, size_t es) {
    return QkSpan{reinterpret_cast<uintptr_t>(p), heads * D * (int64_t)es, stride * (int64_t)es};
}

// Whether two of them share a byte.  (Of tensors with different strides whose
// ranges meet, only those that begin within a row of each other are found.)
static bool qk_meet(const QkSpan &a, const QkSpan &b, int64_t tokens) {
    if (a.row == 0 || b.row == 0) return false;
    const int64_t d = (int64_t)(b.at - a.at), last = tokens - 1;
    if (tokens == 1 || a.stride != b.stride) return d < a.row && -d < b.row;
    // row j of b begins (j - i) * stride + d bytes past row i of a
    int64_t k = d / a.stride, rest = d % a.stride;
    if (rest < 0) {
        rest += a.stride;
        --k;
    }
    return (rest < a.row && k >= -last && k <= last) ||
           (a.stride - rest < b.row && k + 1 >= -last && k + 1 <= last);
}
static bool qk_same(const QkSpan &a, const QkSpan &b, int64_t tokens) {
    return a.at == b.at && (tokens == 1 || a.stride == b.stride);
}

static lsr::QkRope qk_rope(const float *cos, const float *sin, const int32_t *positions,
                           int64_t tokens, int64_t max_pos, int64_t D, int64_t rot,
                           int interleaved, float eps) {
    lsr::QkRope r = {};
    r.cos = cos;
    r.sin = sin;
    r.positions = positions;
    r.tokens = tokens;
    r.max_pos = max_pos;
    r.D = (int)D;
    r.rot = (int)rot;
    r.interleaved = interleaved ? 1 : 0;
    r.eps = eps;
    return r;
}

ls_status ls_qk_norm_rope_fw(void *q_out, void *k_out, float *q_rstd, float *k_rstd,
                             const void *q, const void *k, const void *gamma_q,
                             const void *gamma_k, const float *cos, const float *sin,
                             const int32_t *positions, int64_t tokens, int64_t Hq, int64_t Hk,
                             int64_t D, int64_t rot, int64_t max_pos, int64_t q_out_stride,
                             int64_t k_out_stride, int64_t q_stride, int64_t k_stride,
                             int interleaved, float eps, ls_dtype dt, void *stream) {
    const size_t es = elem_size(dt);
    if (es == 0) return LS_ERR_UNSUPPORTED;
    ls_status s = qk_check(tokens, Hq, Hk, D, rot, max_pos, cos, sin, positions);
    if (s != LS_OK) return s;
    if (!(eps >= 0.f) || !std::isfinite(eps)) return LS_ERR_INVALID_ARG;
    if (tokens == 0 || Hq + Hk == 0) return LS_OK;
    if ((s = qk_tensor(q_out, tokens, Hq, D, q_out_stride, es)) != LS_OK ||
        (s = qk_tensor(k_out, tokens, Hk, D, k_out_stride, es)) != LS_OK ||
        (s = qk_tensor(q, tokens, Hq, D, q_stride, es)) != LS_OK ||
        (s = qk_tensor(k, tokens, Hk, D, k_stride, es)) != LS_OK)
        return s;
    if ((Hq > 0 && !gamma_q) || (Hk > 0 && !gamma_k)) return LS_ERR_INVALID_ARG;
    if ((gamma_q && !aligned(gamma_q, es)) || (gamma_k && !aligned(gamma_k, es)) ||
        (q_rstd && !aligned(q_rstd, 4)) || (k_rstd && !aligned(k_rstd, 4)))
        return LS_ERR_MISALIGNED;
    // each side reads and writes on its own: no output may touch the other
    // side's tensors, nor its own input other than in place
    const QkSpan so[2] = {qk_span(q_out, Hq, D, q_out_stride, es),
                          qk_span(k_out, Hk, D, k_out_stride, es)};
    const QkSpan si[2] = {qk_span(q, Hq, D, q_stride, es), qk_span(k, Hk, D, k_stride, es)};
    if (qk_meet(so[0], so[1], tokens)) return LS_ERR_INVALID_ARG;
    for (int i = 0; i < 2; ++i)
        if (qk_meet(so[i], si[1 - i], tokens) ||
            (!qk_same(so[i], si[i], tokens) && qk_meet(so[i], si[i], tokens)))
            return LS_ERR_INVALID_ARG;
    const lsr::QkRope r =
        qk_rope(cos, sin, positions, tokens, max_pos, D, rot, interleaved, eps);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    auto launch = [&](auto zero) {
        using T = decltype(zero);
        return from_cuda(lsr::launch_qk_fw<T>(
            qk_side<T>(q_out, q, nullptr, gamma_q, q_rstd, nullptr, nullptr, Hq, q_stride,
                       q_out_stride, 0),
            qk_side<T>(k_out, k, nullptr, gamma_k, k_rstd, nullptr, nullptr, Hk, k_stride,
                       k_out_stride, 0),
            r, st));
    };
    switch (dt) {
        case LS_F32: return launch(float());
        case LS_F16: return launch(__half());
        case LS_BF16: return launch(__nv_bfloat16());
    }
    return LS_ERR_UNSUPPORTED;
}

size_t ls_qk_norm_rope_bw_workspace_size(int64_t tokens, int64_t Hq, int64_t Hk, int64_t D) {
    if (tokens <= 0 || Hq < 0 || Hk < 0 || Hq > LS_MAX_HEADS || Hk > LS_MAX_HEADS || D <= 0 ||
        D > LS_MAX_HEAD_DIM)
        return 0;
    return (size_t)lsr::qk_bw_parts(tokens, Hq, Hk) * (size_t)D * sizeof(float);
}

ls_status ls_qk_norm_rope_bw(void *dq, void *dk, float *dgamma_q, float *dgamma_k,
                             const void *dq_out, const void *dk_out, const void *q, const void *k,
                             const void *gamma_q, const void *gamma_k, const float *q_rstd,
                             const float *k_rstd, const float *cos, const float *sin,
                             const int32_t *positions, int64_t tokens, int64_t Hq, int64_t Hk,
                             int64_t D, int64_t rot, int64_t max_pos, int64_t dq_stride,
                             int64_t dk_stride, int64_t dq_out_stride, int64_t dk_out_stride,
                             int64_t q_stride, int64_t k_stride, int interleaved, void *workspace,
                             size_t workspace_bytes, ls_dtype dt, void *stream) {
    const size_t es = elem_size(dt);
    if (es == 0) return LS_ERR_UNSUPPORTED;
    ls_status s = qk_check(tokens, Hq, Hk, D, rot, max_pos, cos, sin, positions);
    if (s != LS_OK) return s;
    if ((Hq > 0 && !dgamma_q) || (Hk > 0 && !dgamma_k)) return LS_ERR_INVALID_ARG;
    if (Hq + Hk == 0) return LS_OK;
    if ((s = qk_tensor(dq, tokens, Hq, D, dq_stride, es)) != LS_OK ||
        (s = qk_tensor(dk, tokens, Hk, D, dk_stride, es)) != LS_OK ||
        (s = qk_tensor(dq_out, tokens, Hq, D, dq_out_stride, es)) != LS_OK ||
        (s = qk_tensor(dk_out, tokens, Hk, D, dk_out_stride, es)) != LS_OK ||
        (s = qk_tensor(q, tokens, Hq, D, q_stride, es)) != LS_OK ||
        (s = qk_tensor(k, tokens, Hk, D, k_stride, es)) != LS_OK)
        return s;
    if (tokens > 0 && ((Hq > 0 && (!gamma_q || !q_rstd)) || (Hk > 0 && (!gamma_k || !k_rstd))))
        return LS_ERR_INVALID_ARG;
    if ((gamma_q && !aligned(gamma_q, es)) || (gamma_k && !aligned(gamma_k, es)) ||
        (q_rstd && !aligned(q_rstd, 4)) || (k_rstd && !aligned(k_rstd, 4)) ||
        (dgamma_q && !aligned(dgamma_q, 4)) || (dgamma_k && !aligned(dgamma_k, 4)))
        return LS_ERR_MISALIGNED;
    const size_t need = ls_qk_norm_rope_bw_workspace_size(tokens, Hq, Hk, D);
    if (need > 0 && (!workspace || workspace_bytes < need || !aligned(workspace, 16)))
        return LS_ERR_WORKSPACE;
    if (tokens > 0) {  // as in the forward
        const QkSpan so[2] = {qk_span(dq, Hq, D, dq_stride, es), qk_span(dk, Hk, D, dk_stride, es)};
        const QkSpan sd[2] = {qk_span(dq_out, Hq, D, dq_out_stride, es),
                              qk_span(dk_out, Hk, D, dk_out_stride, es)};
        const QkSpan si[2] = {qk_span(q, Hq, D, q_stride, es), qk_span(k, Hk, D, k_stride, es)};
        if (qk_meet(so[0], so[1], tokens)) return LS_ERR_INVALID_ARG;
        for (int i = 0; i < 2; ++i)
            if (qk_meet(so[i], sd[1 - i], tokens) || qk_meet(so[i], si[1 - i], tokens) ||
                (!qk_same(so[i], sd[i], tokens) && qk_meet(so[i], sd[i], tokens)) ||
                (!qk_same(so[i], si[i], tokens) && qk_meet(so[i], si[i], tokens)))
                return LS_ERR_INVALID_ARG;
    }
    const lsr::QkRope r =
        qk_rope(cos, sin, positions, tokens, max_pos, D, rot, interleaved, 0.f);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    float *part = static_cast<float *>(workspace);
    auto launch = [&](auto zero) {
        using T = decltype(zero);
        return from_cuda(lsr::launch_qk_bw<T>(
            qk_side<T>(dq, q, dq_out, gamma_q, nullptr, q_rstd, Hq > 0 ? dgamma_q : nullptr, Hq,
                       q_stride, dq_stride, dq_out_stride),
            qk_side<T>(dk, k, dk_out, gamma_k, nullptr, k_rstd, Hk > 0 ? dgamma_k : nullptr, Hk,
                       k_stride, dk_stride, dk_out_stride),
            r, part, st));
    };
    switch (dt) {
        case LS_F32: return launch(float());
        case LS_F16: return launch(__half());
        case LS_BF16: return launch(__nv_bfloat16());
    }
    return LS_ERR_UNSUPPORTED;
}

// ----------------------------------------------------------------------------
// global gradient norm and clipping
// ----------------------------------------------------------------------------
// Checks the host lists (out NULL: a norm alone).
static ls_status grad_check(const float *norm, void *const *out, bool clip,
                            const void *const *grads, const int64_t *sizes,
                            const int32_t *dtypes, int64_t count, const void *workspace,
                            size_t workspace_bytes) {
    if (count < 0 || !norm) return LS_ERR_INVALID_ARG;
    if (count > 0 && (!grads || !sizes || !dtypes || (clip && !out))) return LS_ERR_INVALID_ARG;
    if (!aligned(norm, 4)) return LS_ERR_MISALIGNED;
    int64_t total = 0;
    for (int64_t i = 0; i < count; ++i) {
        const size_t es = elem_size((ls_dtype)dtypes[i]);
        if (es == 0) return LS_ERR_UNSUPPORTED;
        if (sizes[i] < 0) return LS_ERR_INVALID_ARG;
        if (sizes[i] == 0) continue;
        if (!grads[i] || (clip && !out[i])) return LS_ERR_INVALID_ARG;
        if (!aligned(grads[i], es) || (clip && !aligned(out[i], es))) return LS_ERR_MISALIGNED;
        if (sizes[i] > LS_MAX_GRAD_ELEMENTS - total) return LS_ERR_UNSUPPORTED;
        total += sizes[i];
    }
    const size_t need = ls_grad_norm_workspace_size(count);
    if (need > 0 && (!workspace || workspace_bytes < need || !aligned(workspace, 16)))
        return LS_ERR_WORKSPACE;
    return LS_OK;
}

// Whether an output overlaps another output, or a gradient that is not its own
// in place.  (A list's outputs are taken kBlock at a time and sorted; the
// spans of a block that do not overlap are in order by their ends too, so the
// last one that begins before an address range ends decides.)
static bool grad_overlaps(void *const *out, const void *const *grads, const int64_t *sizes,
                          const int32_t *dtypes, int64_t count) {
    struct Span {
        uintptr_t beg, end;
    };
    auto span = [&](const void *p, int64_t i) {
        const uintptr_t a = reinterpret_cast<uintptr_t>(p);
        return Span{a, a + (uintptr_t)sizes[i] * elem_size((ls_dtype)dtypes[i])};
    };
    constexpr int64_t kBlock = 512;
    Span held[kBlock];
    for (int64_t i0 = 0; i0 < count; i0 += kBlock) {
        const int64_t i1 = std::min(count, i0 + kBlock);
        int n = 0;
        for (int64_t i = i0; i < i1; ++i)
            if (sizes[i] > 0) held[n++] = span(out[i], i);
        if (n == 0) continue;
        std::sort(held, held + n, [](const Span &a, const Span &b) { return a.beg < b.beg; });
        for (int k = 1; k < n; ++k)
            if (held[k].beg < held[k - 1].end) return true;
        auto meets = [&](const Span &s) {
            if (s.end <= held[0].beg || s.beg >= held[n - 1].end) return false;
            const Span *past = std::partition_point(
                held, held + n, [&](const Span &a) { return a.beg < s.end; });
            return past[-1].end > s.beg;
        };
        for (int64_t j = 0; j < count; ++j) {
            if (sizes[j] == 0) continue;
            if (out[j] != grads[j] && meets(span(grads[j], j))) return true;
            if (j >= i1 && meets(span(out[j], j))) return true;
        }
    }
    return false;
}

size_t ls_grad_norm_workspace_size(int64_t count) {
    return (size_t)lsr::grad_parts(count) * sizeof(double);
}

ls_status ls_grad_norm(float *norm, const void *const *grads, const int64_t *sizes,
                       const int32_t *dtypes, int64_t count, void *workspace,
                       size_t workspace_bytes, void *stream) {
    const ls_status s = grad_check(norm, nullptr, false, grads, sizes, dtypes, count, workspace,
                                   workspace_bytes);
    if (s != LS_OK) return s;
    return from_cuda(lsr::launch_grad_norm(norm, grads, sizes, dtypes, count,
                                           static_cast<double *>(workspace),
                                           static_cast<cudaStream_t>(stream)));
}

ls_status ls_grad_clip(float *norm, void *const *out, const void *const *grads,
                       const int64_t *sizes, const int32_t *dtypes, int64_t count, float max_norm,
                       float eps, void *workspace, size_t workspace_bytes, void *stream) {
    if (!std::isfinite(max_norm) || !(max_norm > 0.f) || !std::isfinite(eps) || !(eps >= 0.f))
        return LS_ERR_INVALID_ARG;
    const ls_status s = grad_check(norm, out, true, grads, sizes, dtypes, count, workspace,
                                   workspace_bytes);
    if (s != LS_OK) return s;
    if (grad_overlaps(out, grads, sizes, dtypes, count)) return LS_ERR_INVALID_ARG;
    return from_cuda(lsr::launch_grad_clip(norm, out, grads, sizes, dtypes, count, max_norm, eps,
                                           static_cast<double *>(workspace),
                                           static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
