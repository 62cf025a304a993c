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

// A tensor of heads with its typed pointer.
template <typename T>
lsr::DiffRows<T> diff_rows(void *p, int64_t B, int64_t H, int64_t len, int64_t batch,
                                  int64_t head) {
    // (the stride of a single entry does not matter, and may be anything)
    const int64_t sb = B > 1 ? batch : H * len, sh = H > 1 ? head : len;
    return lsr::DiffRows<T>{static_cast<T *>(p), sb, sh, (B - 1) * sb + (H - 1) * sh + len};
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

// ----------------------------------------------------------------------------
// cross entropy from hidden states
// ----------------------------------------------------------------------------
// Bytes [at, at + n) of a tensor.
struct Span {
    uintptr_t at;
    uint64_t n;
};
static Span span_of(const void *p, int64_t elements, size_t es) {
    return Span{reinterpret_cast<uintptr_t>(p), p ? (uint64_t)elements * es : 0};
}
static bool spans_meet(const Span &a, const Span &b) {
    return a.n > 0 && b.n > 0 && a.at < b.at + b.n && b.at < a.at + a.n;
}
// Whether an output shares memory with another output or an input.
static bool outputs_overlap(std::initializer_list<Span> outs, std::initializer_list<Span> ins) {
    for (auto o = outs.begin(); o != outs.end(); ++o) {
        for (auto q = o + 1; q != outs.end(); ++q)
            if (spans_meet(*o, *q)) return true;
        for (const Span &i : ins)
            if (spans_meet(*o, i)) return true;
    }
    return false;
}

static ls_status linear_ce_sizes(int64_t rows, int64_t hidden, int64_t vocab) {
    if (rows < 0 || hidden < 1 || vocab < 1) return LS_ERR_INVALID_ARG;
    if (rows > LS_MAX_LINEAR_ROWS || hidden > LS_MAX_LINEAR_HIDDEN || vocab > LS_MAX_LINEAR_VOCAB ||
        (rows + vocab) * hidden > ((int64_t)1 << 38))
        return LS_ERR_UNSUPPORTED;
    return LS_OK;
}

static size_t linear_ce_size(bool backward, int64_t rows, int64_t hidden, int64_t vocab,
                             ls_dtype dt) {
    const size_t es = elem_size(dt);
    if (es == 0 || linear_ce_sizes(rows, hidden, vocab) != LS_OK) return 0;
    return lsr::linear_ce_workspace(backward, rows, hidden, vocab, es);
}

size_t ls_linear_cross_entropy_fw_workspace_size(int64_t rows, int64_t hidden, int64_t vocab,
                                                 ls_dtype dt) {
    return rows == 0 ? 0 : linear_ce_size(false, rows, hidden, vocab, dt);
}

size_t ls_linear_cross_entropy_bw_workspace_size(int64_t rows, int64_t hidden, int64_t vocab,
                                                 ls_dtype dt) {
    return linear_ce_size(true, rows, hidden, vocab, dt);
}

// What both directions want of x, w and the targets.
static ls_status linear_ce_check(const void *x, const void *w, const int32_t *target, int64_t rows,
                                 int64_t hidden, size_t es) {
    if (!w || (rows > 0 && (!x || !target))) return LS_ERR_INVALID_ARG;
    // 16-bit rows of whole 16 bytes are read where they lie
    const size_t wa = es == 2 && hidden % 8 == 0 ? 16 : es;
    if (!aligned(x, es) || !aligned(w, wa) || !aligned(target, 4)) return LS_ERR_MISALIGNED;
    return LS_OK;
}

ls_status ls_linear_cross_entropy_fw(float *loss, float *lse, const void *x, const void *w,
                                     const int32_t *target, int64_t rows, int64_t hidden,
                                     int64_t vocab, void *workspace, size_t workspace_bytes,
                                     ls_dtype dt, void *stream) {
    const size_t es = elem_size(dt);
    if (es == 0) return LS_ERR_UNSUPPORTED;
    ls_status s = linear_ce_sizes(rows, hidden, vocab);
    if (s != LS_OK) return s;
    if (rows == 0) return LS_OK;
    if (!loss || !lse) return LS_ERR_INVALID_ARG;
    if ((s = linear_ce_check(x, w, target, rows, hidden, es)) != LS_OK) return s;
    if (!aligned(loss, 4) || !aligned(lse, 4)) return LS_ERR_MISALIGNED;
    const size_t need = ls_linear_cross_entropy_fw_workspace_size(rows, hidden, vocab, dt);
    if (!workspace || workspace_bytes < need || !aligned(workspace, 16)) return LS_ERR_WORKSPACE;
    if (outputs_overlap({span_of(loss, rows, 4), span_of(lse, rows, 4), span_of(workspace, need, 1)},
                        {span_of(x, rows * hidden, es), span_of(w, vocab * hidden, es),
                         span_of(target, rows, 4)}))
        return LS_ERR_INVALID_ARG;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    auto launch = [&](auto zero) {
        using T = decltype(zero);
        return from_cuda(lsr::launch_linear_ce_fw<T>(loss, lse, static_cast<const T *>(x),
                                                     static_cast<const T *>(w), target, rows,
                                                     hidden, vocab, workspace, st));
    };
    switch (dt) {
        case LS_F32: return launch(float());
        case LS_F16: return launch(__half());
        case LS_BF16: return launch(__nv_bfloat16());
    }
    return LS_ERR_UNSUPPORTED;
}

ls_status ls_linear_cross_entropy_bw(void *dx, void *dw, const void *x, const void *w,
                                     const int32_t *target, const float *lse, const float *dloss,
                                     int64_t rows, int64_t hidden, int64_t vocab, void *workspace,
                                     size_t workspace_bytes, ls_dtype dt, void *stream) {
    const size_t es = elem_size(dt);
    if (es == 0) return LS_ERR_UNSUPPORTED;
    ls_status s = linear_ce_sizes(rows, hidden, vocab);
    if (s != LS_OK) return s;
    if (rows > 0 && (!dx || !lse || !dloss)) return LS_ERR_INVALID_ARG;
    if (rows == 0 && !dw) return LS_OK;
    if ((s = linear_ce_check(x, w, target, rows, hidden, es)) != LS_OK) return s;
    if (!aligned(dx, es) || !aligned(dw, es) || !aligned(lse, 4) || !aligned(dloss, 4))
        return LS_ERR_MISALIGNED;
    const size_t need = ls_linear_cross_entropy_bw_workspace_size(rows, hidden, vocab, dt);
    if (!workspace || workspace_bytes < need || !aligned(workspace, 16)) return LS_ERR_WORKSPACE;
    if (outputs_overlap({span_of(dx, rows * hidden, es), span_of(dw, vocab * hidden, es),
                         span_of(workspace, need, 1)},
                        {span_of(x, rows * hidden, es), span_of(w, vocab * hidden, es),
                         span_of(target, rows, 4), span_of(lse, rows, 4), span_of(dloss, rows, 4)}))
        return LS_ERR_INVALID_ARG;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    auto launch = [&](auto zero) {
        using T = decltype(zero);
        return from_cuda(lsr::launch_linear_ce_bw<T>(
            static_cast<T *>(dx), static_cast<T *>(dw), static_cast<const T *>(x),
            static_cast<const T *>(w), target, lse, dloss, rows, hidden, vocab, workspace, st));
    };
    switch (dt) {
        case LS_F32: return launch(float());
        case LS_F16: return launch(__half());
        case LS_BF16: return launch(__nv_bfloat16());
    }
    return LS_ERR_UNSUPPORTED;
}

// ----------------------------------------------------------------------------
// difference of two softmax maps
// ----------------------------------------------------------------------------
// B batch entries of H heads of `len` dense elements each.
struct HeadSpan {
    uintptr_t at;
    int64_t len, batch, head;  // bytes
};
// Whether a tensor may be written: no two of its heads share memory.
static bool heads_apart(int64_t B, int64_t H, int64_t len, int64_t batch, int64_t head) {
    if (batch < 0 || head < 0) return false;
    const bool outer = (H == 1 || head >= len) && (B == 1 || batch >= (H - 1) * head + len);
    const bool inner = (B == 1 || batch >= len) && (H == 1 || head >= (B - 1) * batch + len);
    return outer || inner;
}
// Whether two tensors share a byte.  (Of tensors with different strides:
// whether their ranges meet.)
static bool heads_meet(const HeadSpan &a, const HeadSpan &b, int64_t B, int64_t H) {
    const int64_t sb = B > 1 ? a.batch : 0, sh = H > 1 ? a.head : 0;
    const int64_t tb = B > 1 ? b.batch : 0, th = H > 1 ? b.head : 0;
    const uintptr_t a_end = a.at + (uintptr_t)((B - 1) * sb + (H - 1) * sh + a.len);
    const uintptr_t b_end = b.at + (uintptr_t)((B - 1) * tb + (H - 1) * th + b.len);
    if (a.len == 0 || b.len == 0 || a_end <= b.at || b_end <= a.at) return false;
    if (sb != tb || sh != th) return true;
    // -len_b < d + x * sb + y * sh < len_a for some |x| < B, |y| < H: for every step of
    // the shorter axis, the nearest step of the other
    const int64_t d = (int64_t)(b.at - a.at);
    const int64_t n = B < H ? B : H, m = B < H ? H : B;
    const int64_t sn = B < H ? sb : sh, sm = B < H ? sh : sb;
    for (int64_t y = 1 - n; y < n; ++y) {
        const int64_t v = d + y * sn;
        int64_t x = sm > 0 ? -v / sm : 0;
        for (int64_t k = x - 1; k <= x + 1; ++k) {
            const int64_t c = k < 1 - m ? 1 - m : (k > m - 1 ? m - 1 : k);
            const int64_t gap = v + c * sm;
            if (gap < a.len && -gap < b.len) return true;
        }
    }
    return false;
}
static bool heads_same(const HeadSpan &a, const HeadSpan &b, int64_t B, int64_t H) {
    return a.at == b.at && (B == 1 || a.batch == b.batch) && (H == 1 || a.head == b.head);
}

// Sizes of both directions.
static ls_status diff_check(int64_t B, int64_t H, int64_t Tq, int64_t Tk, int64_t lam_count,
                            int causal, float scale) {
    if (B < 0 || H < 0 || Tq < 0 || Tk < 0) return LS_ERR_INVALID_ARG;
    if (causal && Tq > Tk) return LS_ERR_INVALID_ARG;
    if (!std::isfinite(scale) || !(scale > 0.f)) return LS_ERR_INVALID_ARG;
    if (lam_count != 1 && lam_count != H) return LS_ERR_INVALID_ARG;
    const int64_t most = (int64_t)1 << 30;
    if (B > most || H > LS_MAX_HEADS || Tq > LS_MAX_ROW_LENGTH || Tk > LS_MAX_ROW_LENGTH)
        return LS_ERR_UNSUPPORTED;
    if (B > 0 && H > 0 && Tq > 0 && Tk > 0 &&
        (B * H > ((int64_t)1 << 44) / Tq || B * H * Tq > ((int64_t)1 << 58) / Tk))
        return LS_ERR_UNSUPPORTED;
    return LS_OK;
}
// A tensor of heads: [B, H, Tq, Tk] with strides of elements.
static ls_status diff_tensor(const void *p, int64_t B, int64_t H, int64_t len, int64_t batch,
                             int64_t head, size_t es) {
    if (!p || batch < 0 || head < 0) return LS_ERR_INVALID_ARG;
    const int64_t most = (int64_t)1 << 58;
    if ((B > 1 && batch > most / B) || (H > 1 && head > most / H)) return LS_ERR_UNSUPPORTED;
    (void)len;
    return aligned(p, es) ? LS_OK : LS_ERR_MISALIGNED;
}
static HeadSpan head_span(const void *p, int64_t len, int64_t batch, int64_t head, size_t es) {
    return HeadSpan{reinterpret_cast<uintptr_t>(p), len * (int64_t)es, batch * (int64_t)es,
                    head * (int64_t)es};
}
// A tensor that lies in one piece.
static HeadSpan flat_span(const void *p, int64_t elements, size_t es) {
    return HeadSpan{reinterpret_cast<uintptr_t>(p), p ? elements * (int64_t)es : 0, 0, 0};
}
static lsr::DiffShape diff_shape(int64_t B, int64_t H, int64_t Tq, int64_t Tk, int64_t lam_count,
                                 int causal, float scale) {
    lsr::DiffShape p = {};
    p.rows = B * H * Tq;
    p.B = B;
    p.H = H;
    p.Tq = Tq;
    p.Tk = Tk;
    p.qoff = Tk - Tq;
    p.lam_step = lam_count == 1 ? 0 : 1;
    p.causal = causal ? 1 : 0;
    p.scale = scale;
    return p;
}

ls_status ls_softmax_fw_diff(void *out, float *stats, const void *x1, const void *x2,
                             const float *lam, const void *mask, int64_t B, int64_t H, int64_t Tq,
                             int64_t Tk, int64_t x1_batch, int64_t x1_head, int64_t x2_batch,
                             int64_t x2_head, int64_t lam_count, int causal, float scale,
                             ls_dtype dt, void *stream) {
    const size_t es = elem_size(dt);
    if (es == 0) return LS_ERR_UNSUPPORTED;
    ls_status s = diff_check(B, H, Tq, Tk, lam_count, causal, scale);
    if (s != LS_OK) return s;
    const int64_t len = Tq * Tk;
    if (B == 0 || H == 0 || len == 0) return LS_OK;
    if (!out || !lam) return LS_ERR_INVALID_ARG;
    if ((s = diff_tensor(x1, B, H, len, x1_batch, x1_head, es)) != LS_OK ||
        (s = diff_tensor(x2, B, H, len, x2_batch, x2_head, es)) != LS_OK)
        return s;
    if (!aligned(out, es) || !aligned(mask, es) || !aligned(lam, 4) || !aligned(stats, 16))
        return LS_ERR_MISALIGNED;
    const HeadSpan so = head_span(out, len, H * len, len, es);
    const HeadSpan i1 = head_span(x1, len, x1_batch, x1_head, es);
    const HeadSpan i2 = head_span(x2, len, x2_batch, x2_head, es);
    if ((heads_meet(so, i1, B, H) && !heads_same(so, i1, B, H)) || heads_meet(so, i2, B, H))
        return LS_ERR_INVALID_ARG;
    if (outputs_overlap({span_of(out, B * H * len, es), span_of(stats, 4 * B * H * Tq, 4)},
                        {span_of(lam, lam_count, 4), span_of(mask, B * Tk, es)}))
        return LS_ERR_INVALID_ARG;
    const HeadSpan ss = flat_span(stats, 4 * B * H * Tq, 4);
    if (stats && (heads_meet(ss, i1, B, H) || heads_meet(ss, i2, B, H))) return LS_ERR_INVALID_ARG;
    const lsr::DiffShape p = diff_shape(B, H, Tq, Tk, lam_count, causal, scale);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    auto launch = [&](auto zero) {
        using T = decltype(zero);
        return from_cuda(lsr::launch_diff_fw<T>(
            static_cast<T *>(out), reinterpret_cast<float4 *>(stats),
            diff_rows<const T>(const_cast<void *>(x1), B, H, len, x1_batch, x1_head),
            diff_rows<const T>(const_cast<void *>(x2), B, H, len, x2_batch, x2_head), lam,
            static_cast<const T *>(mask), p, st));
    };
    switch (dt) {
        case LS_F32: return launch(float());
        case LS_F16: return launch(__half());
        case LS_BF16: return launch(__nv_bfloat16());
    }
    return LS_ERR_UNSUPPORTED;
}

size_t ls_softmax_bw_diff_workspace_size(int64_t B, int64_t H, int64_t Tq) {
    if (B <= 0 || H <= 0 || Tq <= 0 || diff_check(B, H, Tq, 1, H, 0, 1.f) != LS_OK) return 0;
    return (size_t)(B * H * Tq) * sizeof(float);
}

ls_status ls_softmax_bw_diff(void *dx1, void *dx2, float *dlam, const void *dout, const void *x1,
                             const void *x2, const float *lam, const float *stats,
                             const void *mask, int64_t B, int64_t H, int64_t Tq, int64_t Tk,
                             int64_t dx1_batch, int64_t dx1_head, int64_t dx2_batch,
                             int64_t dx2_head, int64_t x1_batch, int64_t x1_head, int64_t x2_batch,
                             int64_t x2_head, int64_t lam_count, int causal, float scale,
                             void *workspace, size_t workspace_bytes, ls_dtype dt, void *stream) {
    const size_t es = elem_size(dt);
    if (es == 0) return LS_ERR_UNSUPPORTED;
    ls_status s = diff_check(B, H, Tq, Tk, lam_count, causal, scale);
    if (s != LS_OK) return s;
    if (lam_count == 0) return LS_OK;
    if (!dlam) return LS_ERR_INVALID_ARG;
    if (!aligned(dlam, 4)) return LS_ERR_MISALIGNED;
    const int64_t len = Tq * Tk;
    const lsr::DiffShape p = diff_shape(B, H, Tq, Tk, lam_count, causal, scale);
    if (p.rows > 0 && Tk > 0) {
        if (!dout || !lam || !stats) return LS_ERR_INVALID_ARG;
        if ((s = diff_tensor(dx1, B, H, len, dx1_batch, dx1_head, es)) != LS_OK ||
            (s = diff_tensor(dx2, B, H, len, dx2_batch, dx2_head, es)) != LS_OK ||
            (s = diff_tensor(x1, B, H, len, x1_batch, x1_head, es)) != LS_OK ||
            (s = diff_tensor(x2, B, H, len, x2_batch, x2_head, es)) != LS_OK)
            return s;
        if (!heads_apart(B, H, len, dx1_batch, dx1_head) ||
            !heads_apart(B, H, len, dx2_batch, dx2_head))
            return LS_ERR_INVALID_ARG;
        if (!aligned(dout, es) || !aligned(mask, es) || !aligned(lam, 4) || !aligned(stats, 16))
            return LS_ERR_MISALIGNED;
        const size_t need = ls_softmax_bw_diff_workspace_size(B, H, Tq);
        if (!workspace || workspace_bytes < need || !aligned(workspace, 16))
            return LS_ERR_WORKSPACE;
        const HeadSpan o1 = head_span(dx1, len, dx1_batch, dx1_head, es);
        const HeadSpan o2 = head_span(dx2, len, dx2_batch, dx2_head, es);
        const HeadSpan i1 = head_span(x1, len, x1_batch, x1_head, es);
        const HeadSpan i2 = head_span(x2, len, x2_batch, x2_head, es);
        const HeadSpan g = head_span(dout, len, H * len, len, es);
        const HeadSpan flat[] = {flat_span(stats, 4 * p.rows, 4), flat_span(workspace, p.rows, 4),
                                 flat_span(mask, B * Tk, es), flat_span(lam, lam_count, 4),
                                 flat_span(dlam, lam_count, 4)};
        if (heads_meet(o1, o2, B, H)) return LS_ERR_INVALID_ARG;
        if (outputs_overlap({span_of(dlam, lam_count, 4), span_of(workspace, p.rows, 4)},
                            {span_of(dout, p.rows * Tk, es), span_of(stats, 4 * p.rows, 4),
                             span_of(mask, B * Tk, es), span_of(lam, lam_count, 4)}))
            return LS_ERR_INVALID_ARG;
        for (const HeadSpan &f : {flat[1], flat[4]})  // the workspace and dlam
            if (heads_meet(i1, f, B, H) || heads_meet(i2, f, B, H)) return LS_ERR_INVALID_ARG;
        for (const HeadSpan *o : {&o1, &o2}) {
            const HeadSpan &own = o == &o1 ? i1 : i2, &other = o == &o1 ? i2 : i1;
            if ((heads_meet(*o, own, B, H) && !heads_same(*o, own, B, H)) ||
                heads_meet(*o, other, B, H) || heads_meet(*o, g, B, H))
                return LS_ERR_INVALID_ARG;
            for (const HeadSpan &f : flat)
                if (heads_meet(*o, f, B, H)) return LS_ERR_INVALID_ARG;
        }
    }
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    auto launch = [&](auto zero) {
        using T = decltype(zero);
        return from_cuda(lsr::launch_diff_bw<T>(
            diff_rows<T>(dx1, B, H, len, dx1_batch, dx1_head),
            diff_rows<T>(dx2, B, H, len, dx2_batch, dx2_head), dlam, static_cast<const T *>(dout),
            diff_rows<const T>(const_cast<void *>(x1), B, H, len, x1_batch, x1_head),
            diff_rows<const T>(const_cast<void *>(x2), B, H, len, x2_batch, x2_head), lam,
            reinterpret_cast<const float4 *>(stats), static_cast<const T *>(mask), p,
            static_cast<float *>(workspace), st));
    };
    switch (dt) {
        case LS_F32: return launch(float());
        case LS_F16: return launch(__half());
        case LS_BF16: return launch(__nv_bfloat16());
    }
    return LS_ERR_UNSUPPORTED;
}

// ----------------------------------------------------------------------------
// norms around a block
// ----------------------------------------------------------------------------
static ls_status block_norm_check(int64_t rows, int64_t hidden, int64_t gates, bool has_gate,
                                  float residual_scale) {
    if (rows < 0 || hidden < 1 || !std::isfinite(residual_scale)) return LS_ERR_INVALID_ARG;
    if (has_gate && (gates < 1 || rows % gates != 0)) return LS_ERR_INVALID_ARG;
    if (hidden > LS_MAX_BLOCK_HIDDEN || rows > ((int64_t)1 << 40)) return LS_ERR_UNSUPPORTED;
    return LS_OK;
}

ls_status ls_block_norm_fw(void *h, void *y, float *stats, const void *x, const void *r,
                           const void *gate, const void *gamma_post, const void *beta_post,
                           const void *gamma_pre, const void *beta_pre, int64_t rows,
                           int64_t hidden, int64_t gates, float residual_scale, float eps,
                           int layer, ls_dtype dt, void *stream) {
    const size_t es = elem_size(dt);
    if (es == 0) return LS_ERR_UNSUPPORTED;
    const ls_status s = block_norm_check(rows, hidden, gates, gate != nullptr, residual_scale);
    if (s != LS_OK) return s;
    if (!(eps >= 0.f) || !std::isfinite(eps)) return LS_ERR_INVALID_ARG;
    if ((beta_post && (!layer || !gamma_post)) || (beta_pre && (!layer || !gamma_pre)))
        return LS_ERR_INVALID_ARG;
    if (rows == 0) return LS_OK;
    if (!h || !stats || !x || !r || (gamma_pre && !y)) return LS_ERR_INVALID_ARG;
    for (const void *p : {(const void *)h, (const void *)y, x, r, gate, gamma_post, beta_post,
                          gamma_pre, beta_pre})
        if (!aligned(p, es)) return LS_ERR_MISALIGNED;
    if (!aligned(stats, 4)) return LS_ERR_MISALIGNED;
    const int64_t n = rows * hidden;
    if (!gamma_pre) y = nullptr;  // not written
    // h and y may be x or r itself; nothing else may meet them
    const Span small[] = {span_of(gate, gate ? gates * hidden : 0, es),
                          span_of(gamma_post, hidden, es), span_of(beta_post, hidden, es),
                          span_of(gamma_pre, hidden, es), span_of(beta_pre, hidden, es)};
    const Span outs[] = {span_of(h, n, es), span_of(y, n, es), span_of(stats, 4 * rows, 4)};
    const Span rows_in[] = {span_of(x, n, es), span_of(r, n, es)};
    for (int i = 0; i < 3; ++i) {
        for (int j = i + 1; j < 3; ++j)
            if (spans_meet(outs[i], outs[j])) return LS_ERR_INVALID_ARG;
        for (const Span &q : small)
            if (spans_meet(outs[i], q)) return LS_ERR_INVALID_ARG;
        for (const Span &q : rows_in)
            if (spans_meet(outs[i], q) && (i == 2 || outs[i].at != q.at)) return LS_ERR_INVALID_ARG;
    }
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    auto launch = [&](auto zero) {
        using T = decltype(zero);
        lsr::BlockNorm<T> a = {};
        a.rows = rows;
        a.hidden = hidden;
        a.gates = gates;
        a.gate_rows = gate ? rows / gates : rows;
        a.residual_scale = residual_scale;
        a.eps = eps;
        a.layer = layer ? 1 : 0;
        a.x = static_cast<const T *>(x);
        a.r = static_cast<const T *>(r);
        a.gate = static_cast<const T *>(gate);
        a.gamma_post = static_cast<const T *>(gamma_post);
        a.beta_post = static_cast<const T *>(beta_post);
        a.gamma_pre = static_cast<const T *>(gamma_pre);
        a.beta_pre = static_cast<const T *>(beta_pre);
        a.stats = stats;
        a.h = static_cast<T *>(h);
        a.y = static_cast<T *>(y);
        return from_cuda(lsr::launch_block_norm_fw<T>(a, st));
    };
    switch (dt) {
        case LS_F32: return launch(float());
        case LS_F16: return launch(__half());
        case LS_BF16: return launch(__nv_bfloat16());
    }
    return LS_ERR_UNSUPPORTED;
}

size_t ls_block_norm_bw_workspace_size(int64_t rows, int64_t hidden, int64_t gates, int layer,
                                       ls_dtype dt) {
    if (rows <= 0 || gates < 0 || block_norm_check(rows, hidden, gates, gates > 0, 1.f) != LS_OK)
        return 0;
    switch (dt) {
        case LS_F32: return lsr::block_norm_workspace<float>(rows, hidden, gates, layer != 0);
        case LS_F16: return lsr::block_norm_workspace<__half>(rows, hidden, gates, layer != 0);
        case LS_BF16:
            return lsr::block_norm_workspace<__nv_bfloat16>(rows, hidden, gates, layer != 0);
    }
    return 0;
}

ls_status ls_block_norm_bw(void *dx, void *dr, float *dgate, float *dgamma_post, float *dbeta_post,
                           float *dgamma_pre, float *dbeta_pre, const void *dy, const void *dh,
                           const void *x, const void *h, const float *stats, const void *gate,
                           const void *gamma_post, const void *beta_post, const void *gamma_pre,
                           int64_t rows, int64_t hidden, int64_t gates, float residual_scale,
                           int layer, void *workspace, size_t workspace_bytes, ls_dtype dt,
                           void *stream) {
    const size_t es = elem_size(dt);
    if (es == 0) return LS_ERR_UNSUPPORTED;
    const ls_status s = block_norm_check(rows, hidden, gates, gate != nullptr, residual_scale);
    if (s != LS_OK) return s;
    if (!gate) gates = 0;
    const bool post = gamma_post != nullptr, pre = gamma_pre != nullptr;
    if ((beta_post && (!layer || !post)) || (dbeta_post && (!layer || !post)) ||
        (dbeta_pre && (!layer || !pre)))
        return LS_ERR_INVALID_ARG;
    if ((post && !dgamma_post) || (pre && !dgamma_pre) || (gate && !dgate))
        return LS_ERR_INVALID_ARG;
    if (!post) dgamma_post = nullptr;
    if (!pre) dgamma_pre = nullptr;
    if (!gate) dgate = nullptr;
    if (rows > 0 && (!dx || !dr || !stats || (pre && (!dy || !h)) || (!pre && !dh) ||
                     ((post || gate) && !x)))
        return LS_ERR_INVALID_ARG;
    if (!pre) dy = h = nullptr;  // not read
    if (!post && !gate) x = nullptr;
    for (const void *p : {(const void *)dx, (const void *)dr, dy, dh, x, h, gate, gamma_post,
                          beta_post, gamma_pre})
        if (!aligned(p, es)) return LS_ERR_MISALIGNED;
    for (const float *p : {(const float *)dgate, (const float *)dgamma_post,
                           (const float *)dbeta_post, (const float *)dgamma_pre,
                           (const float *)dbeta_pre, stats})
        if (!aligned(p, 4)) return LS_ERR_MISALIGNED;
    const size_t need = ls_block_norm_bw_workspace_size(rows, hidden, gates, layer, dt);
    if (need > 0 && (!workspace || workspace_bytes < need || !aligned(workspace, 16)))
        return LS_ERR_WORKSPACE;
    const int64_t n = rows * hidden;
    // dx may be dy, dh, x or h itself and dr dy, dh or h; nothing else may meet
    // them or the sums
    const Span outs[] = {span_of(dx, n, es), span_of(dr, n, es),
                         span_of(dgate, gates * hidden, 4), span_of(dgamma_post, hidden, 4),
                         span_of(dbeta_post, hidden, 4), span_of(dgamma_pre, hidden, 4),
                         span_of(dbeta_pre, hidden, 4), span_of(workspace, need, 1)};
    const Span small[] = {span_of(gate, gates * hidden, es), span_of(gamma_post, hidden, es),
                          span_of(beta_post, hidden, es), span_of(gamma_pre, hidden, es),
                          span_of(stats, 4 * rows, 4)};
    const Span rows_in[] = {span_of(x, n, es), span_of(dy, n, es), span_of(dh, n, es),
                            span_of(h, n, es)};
    for (int i = 0; i < 8; ++i) {
        for (int j = i + 1; j < 8; ++j)
            if (spans_meet(outs[i], outs[j])) return LS_ERR_INVALID_ARG;
        for (const Span &q : small)
            if (spans_meet(outs[i], q)) return LS_ERR_INVALID_ARG;
        for (int j = 0; j < 4; ++j)
            if (spans_meet(outs[i], rows_in[j]) &&
                (i > 1 || (i == 1 && j == 0) || outs[i].at != rows_in[j].at))
                return LS_ERR_INVALID_ARG;
    }
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    auto launch = [&](auto zero) {
        using T = decltype(zero);
        lsr::BlockNorm<T> a = {};
        a.rows = rows;
        a.hidden = hidden;
        a.gates = gates;
        a.gate_rows = gate ? rows / gates : rows;
        a.residual_scale = residual_scale;
        a.layer = layer ? 1 : 0;
        a.x = static_cast<const T *>(x);
        a.gate = static_cast<const T *>(gate);
        a.gamma_post = static_cast<const T *>(gamma_post);
        a.beta_post = static_cast<const T *>(beta_post);
        a.gamma_pre = static_cast<const T *>(gamma_pre);
        a.dy = static_cast<const T *>(dy);
        a.dh = static_cast<const T *>(dh);
        a.h_in = static_cast<const T *>(h);
        a.stats_in = stats;
        a.dx = static_cast<T *>(dx);
        a.dr = static_cast<T *>(dr);
        a.dgate = dgate;
        a.dgamma_post = dgamma_post;
        a.dbeta_post = dbeta_post;
        a.dgamma_pre = dgamma_pre;
        a.dbeta_pre = dbeta_pre;
        return from_cuda(lsr::launch_block_norm_bw<T>(a, static_cast<float *>(workspace), st));
    };
    switch (dt) {
        case LS_F32: return launch(float());
        case LS_F16: return launch(__half());
        case LS_BF16: return launch(__nv_bfloat16());
    }
    return LS_ERR_UNSUPPORTED;
}

}  // extern "C"
