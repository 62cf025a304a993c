// grad_clip.cu -- global gradient norm over many tensors of mixed storage
// types, and clipping by it (sm_103a).
//
//     norm = sqrt(sum over all tensors and elements of g^2)
//     out  = g * min(1, max_norm / (norm + eps))
//
// The list of tensors travels in the kernel's parameters (40 bytes a tensor,
// up to kGradCap of them a launch), so nothing is copied to the device and a
// captured graph carries its list.  Tensors are cut into chunks of 2048
// 16-byte slots; a block of 256 threads takes a chunk at a time, eight slots
// per thread in flight together, and finds the chunk's tensor by bisection.
// Slots lie on 16-byte addresses whatever the tensor's own alignment; the
// first and last slot of a tensor are taken element by element.
//
// Every block leaves one FP64 partial sum.  The clipping kernel needs no third
// launch for the total: each of its blocks adds the (at most 608 per launch)
// partials itself, in the same fixed order, and takes the chunks from the end
// of the list, which the norm's pass read last and L2 still holds.  The cut
// depends only on the list, so the norm is bitwise reproducible.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "dispatch.cuh"
#include "launch.h"
#include "ls_device.cuh"
#include "ls_reduce.h"

namespace lsr {
namespace {

constexpr int kGradBlock = 256;
constexpr int kGradSlots = 8;                              // 16-byte slots per thread
constexpr int64_t kGradChunk = kGradBlock * kGradSlots;    // slots per chunk
constexpr int64_t kGradBlocks = 4 * 152;  // partial sums of a launch, a constant of the library
constexpr int kGradCap = 512;             // tensors of a launch
constexpr int kGradSmallCap = 48;         // a shorter list has a parameter block of its own

struct GradSpan {
    const void *g;
    void *o;
    int64_t n;
    int64_t chunk0;  // first chunk of the tensor
    int32_t dt;
};
template <int CAP>
struct GradList {
    GradSpan s[CAP];
    int64_t chunks;
    int32_t count;
};

// Element at the 16-byte address at or below p, relative to p.
template <typename T>
__device__ __forceinline__ int64_t grad_first_element(const void *p) {
    return -(int64_t)((reinterpret_cast<uintptr_t>(p) & 15u) / sizeof(T));
}

int64_t grad_chunks(const void *p, int64_t n, int es) {
    const int64_t bytes = n * es + (int64_t)(reinterpret_cast<uintptr_t>(p) & 15u);
    return n > 0 ? ceil_div(ceil_div(bytes, 16), kGradChunk) : 0;
}

int grad_es(int dt) { return dt == LS_F32 ? 4 : 2; }

template <int CAP>
__device__ __forceinline__ int grad_find(const GradList<CAP> &L, int64_t chunk) {
    int lo = 0, hi = L.count;  // the last tensor whose chunk0 <= chunk
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (L.s[mid].chunk0 <= chunk)
            lo = mid;
        else
            hi = mid;
    }
    return lo;
}

// The slot whose first element is e0 (elements outside [0, n) read as 0).
template <typename T>
__device__ __forceinline__ uint4 grad_load(const T *g, int64_t e0, int64_t n) {
    constexpr int V = Traits<T>::kVec;
    if (e0 >= 0 && e0 + V <= n) return ld_cached16(g + e0);
    float f[V];
#pragma unroll
    for (int e = 0; e < V; ++e)
        f[e] = e0 + e >= 0 && e0 + e < n ? Traits<T>::load1(g + e0 + e) : 0.f;
    return Traits<T>::pack(f);
}

// Sum of squares of a thread's slots of one chunk.  In FP32 unless the squares
// leave the range where that is exact enough (a sum below 2^-90 may have lost
// denormal squares, one that overflowed may be finite), and then in FP64;
// slots of zeros, which a sparse gradient is full of, never take that path.
template <typename T>
__device__ __forceinline__ double grad_chunk_squares(const GradSpan &sp, int64_t chunk) {
    constexpr int V = Traits<T>::kVec;
    const T *g = static_cast<const T *>(sp.g);
    const int64_t e0 =
        grad_first_element<T>(sp.g) +
        ((chunk - sp.chunk0) * kGradChunk + threadIdx.x) * V;
    uint4 raw[kGradSlots];
#pragma unroll
    for (int u = 0; u < kGradSlots; ++u) {
        const int64_t e = e0 + (int64_t)u * kGradBlock * V;
        raw[u] = e < sp.n ? grad_load<T>(g, e, sp.n) : make_uint4(0u, 0u, 0u, 0u);
    }
    float2 s2 = f2(0.f);
#pragma unroll
    for (int u = 0; u < kGradSlots; ++u) {
        float2 v[V / 2];
        unpack2<T>(raw[u], v);
#pragma unroll
        for (int h = 0; h < V / 2; ++h) s2 = fma2(v[h], v[h], s2);
    }
    const float s = s2.x + s2.y;
    if (s > 0x1p-90f && s < INFINITY) return (double)s;
    uint32_t any = 0u;
#pragma unroll
    for (int u = 0; u < kGradSlots; ++u) any |= raw[u].x | raw[u].y | raw[u].z | raw[u].w;
    if (any == 0u) return 0.0;
    double d = 0.0;
#pragma unroll 1
    for (int u = 0; u < kGradSlots; ++u) {
        const int64_t e = e0 + (int64_t)u * kGradBlock * V;
        for (int i = 0; i < V; ++i)
            if (e + i >= 0 && e + i < sp.n) {
                const double x = (double)Traits<T>::load1(g + e + i);
                d = fma(x, x, d);
            }
    }
    return d;
}

__device__ __forceinline__ double grad_block_sum(double v) {
    __shared__ double red[kGradBlock / 32];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    v = red[0];
#pragma unroll
    for (int w = 1; w < kGradBlock / 32; ++w) v += red[w];
    return v;
}

template <int CAP>
__global__ void __launch_bounds__(kGradBlock)
grad_squares(double *part, const __grid_constant__ GradList<CAP> L) {
    pdl_begin();
    double d = 0.0;
    for (int64_t c = blockIdx.x; c < L.chunks; c += gridDim.x) {
        const GradSpan &sp = L.s[grad_find(L, c)];
        if (sp.dt == LS_F32)
            d += grad_chunk_squares<float>(sp, c);
        else if (sp.dt == LS_F16)
            d += grad_chunk_squares<__half>(sp, c);
        else
            d += grad_chunk_squares<__nv_bfloat16>(sp, c);
    }
    d = grad_block_sum(d);
    if (threadIdx.x == 0) part[blockIdx.x] = d;
}

// The norm from all partials, the same in every block that asks.
__device__ __forceinline__ float grad_total_norm(const double *part, int parts) {
    double d = 0.0;
    for (int i = threadIdx.x; i < parts; i += kGradBlock) d += part[i];
    return (float)sqrt(grad_block_sum(d));
}

__global__ void __launch_bounds__(kGradBlock)
grad_norm_final(float *norm, const double *part, int parts) {
    pdl_begin();
    const float v = grad_total_norm(part, parts);
    if (threadIdx.x == 0) *norm = v;
}

template <typename T>
__device__ __forceinline__ void grad_chunk_scale(const GradSpan &sp, int64_t chunk, float coef) {
    constexpr int V = Traits<T>::kVec;
    const T *g = static_cast<const T *>(sp.g);
    T *o = static_cast<T *>(sp.o);
    const bool same =
        ((reinterpret_cast<uintptr_t>(g) ^ reinterpret_cast<uintptr_t>(o)) & 15u) == 0;
    const int64_t e0 =
        grad_first_element<T>(sp.g) +
        ((chunk - sp.chunk0) * kGradChunk + threadIdx.x) * V;
    uint4 raw[kGradSlots];
#pragma unroll
    for (int u = 0; u < kGradSlots; ++u) {
        const int64_t e = e0 + (int64_t)u * kGradBlock * V;
        if (e < sp.n) {
            if (e >= 0 && e + V <= sp.n)
                raw[u] = *reinterpret_cast<const uint4 *>(g + e);
            else
                raw[u] = grad_load<T>(g, e, sp.n);
        }
    }
#pragma unroll
    for (int u = 0; u < kGradSlots; ++u) {
        const int64_t e = e0 + (int64_t)u * kGradBlock * V;
        if (e >= sp.n) continue;
        float f[V];
        Traits<T>::unpack(raw[u], f);
#pragma unroll
        for (int i = 0; i < V; ++i) f[i] *= coef;
        if (same && e >= 0 && e + V <= sp.n) {
            st_stream16(o + e, Traits<T>::pack(f));
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (e + i >= 0 && e + i < sp.n) Traits<T>::store1(o + e + i, f[i]);
        }
    }
}

template <int CAP>
__global__ void __launch_bounds__(kGradBlock)
grad_scale(float *norm, const double *part, int parts, float max_norm, float eps,
           const __grid_constant__ GradList<CAP> L) {
    pdl_begin();
    const float total = grad_total_norm(part, parts);
    if (blockIdx.x == 0 && threadIdx.x == 0) *norm = total;
    const float ratio = max_norm / (total + eps);
    const float coef = ratio >= 1.f ? 1.f : ratio;  // a NaN norm gives NaN
    for (int64_t k = blockIdx.x; k < L.chunks; k += gridDim.x) {
        const int64_t c = L.chunks - 1 - k;
        const GradSpan &sp = L.s[grad_find(L, c)];
        if (coef == 1.f && sp.o == sp.g) continue;  // in place and nothing to clip
        if (sp.dt == LS_F32)
            grad_chunk_scale<float>(sp, c, coef);
        else if (sp.dt == LS_F16)
            grad_chunk_scale<__half>(sp, c, coef);
        else
            grad_chunk_scale<__nv_bfloat16>(sp, c, coef);
    }
}

// One launch's list from tensors [beg, end) of the caller's arrays.
template <int CAP>
void grad_fill(GradList<CAP> &L, void *const *out, const void *const *grads, const int64_t *sizes,
               const int32_t *dts, int64_t beg, int64_t end) {
    L.count = (int)(end - beg);
    int64_t chunks = 0;
    for (int64_t i = beg; i < end; ++i) {
        GradSpan &s = L.s[i - beg];
        s.g = grads[i];
        s.o = out ? out[i] : nullptr;
        s.n = sizes[i];
        s.dt = dts[i];
        s.chunk0 = chunks;
        chunks += grad_chunks(s.g, s.n, grad_es(s.dt));
    }
    L.chunks = chunks;
}

template <int CAP>
cudaError_t grad_squares_launch(double *part, const void *const *grads, const int64_t *sizes,
                                const int32_t *dts, int64_t beg, int64_t end, int *parts,
                                cudaStream_t st) {
    GradList<CAP> L;
    grad_fill<CAP>(L, nullptr, grads, sizes, dts, beg, end);
    *parts = (int)(L.chunks < kGradBlocks ? L.chunks : kGradBlocks);
    if (*parts == 0) return cudaSuccess;
    return launch_pdl(grad_squares<CAP>, dim3((unsigned)*parts), dim3(kGradBlock), 0, st, part, L);
}

template <int CAP>
cudaError_t grad_scale_launch(float *norm, const double *part, int parts, float max_norm,
                              float eps, void *const *out, const void *const *grads,
                              const int64_t *sizes, const int32_t *dts, int64_t beg, int64_t end,
                              cudaStream_t st) {
    GradList<CAP> L;
    grad_fill<CAP>(L, out, grads, sizes, dts, beg, end);
    return launch_persistent<grad_scale<CAP>>(kGradBlock, 0, L.chunks, st, norm, part, parts,
                                              max_norm, eps, L);
}

// Partials of every tensor; *parts: how many were left at `part`.
cudaError_t grad_all_squares(const void *const *grads, const int64_t *sizes, const int32_t *dts,
                             int64_t count, double *part, int *parts, cudaStream_t st) {
    *parts = 0;
    for (int64_t beg = 0; beg < count;) {
        const int64_t end = beg + kGradCap < count ? beg + kGradCap : count;
        int n = 0;
        const cudaError_t e =
            end - beg <= kGradSmallCap
                ? grad_squares_launch<kGradSmallCap>(part + *parts, grads, sizes, dts, beg, end,
                                                     &n, st)
                : grad_squares_launch<kGradCap>(part + *parts, grads, sizes, dts, beg, end, &n, st);
        if (e != cudaSuccess) return e;
        *parts += n;
        beg = end;
    }
    return cudaSuccess;
}

}  // namespace

int64_t grad_parts(int64_t count) {
    return count > 0 ? kGradBlocks * ceil_div(count, kGradCap) : 0;
}

cudaError_t launch_grad_norm(float *norm, const void *const *grads, const int64_t *sizes,
                             const int32_t *dts, int64_t count, double *part, cudaStream_t st) {
    int parts = 0;
    const cudaError_t e = grad_all_squares(grads, sizes, dts, count, part, &parts, st);
    if (e != cudaSuccess) return e;
    return launch_pdl(grad_norm_final, dim3(1), dim3(kGradBlock), 0, st, norm,
                      (const double *)part, parts);
}

cudaError_t launch_grad_clip(float *norm, void *const *out, const void *const *grads,
                             const int64_t *sizes, const int32_t *dts, int64_t count,
                             float max_norm, float eps, double *part, cudaStream_t st) {
    int parts = 0;
    cudaError_t e = grad_all_squares(grads, sizes, dts, count, part, &parts, st);
    if (e != cudaSuccess) return e;
    if (parts == 0)
        return launch_pdl(grad_norm_final, dim3(1), dim3(kGradBlock), 0, st, norm,
                          (const double *)part, 0);
    for (int64_t beg = 0; beg < count;) {
        const int64_t end = beg + kGradCap < count ? beg + kGradCap : count;
        e = end - beg <= kGradSmallCap
                ? grad_scale_launch<kGradSmallCap>(norm, part, parts, max_norm, eps, out, grads,
                                                   sizes, dts, beg, end, st)
                : grad_scale_launch<kGradCap>(norm, part, parts, max_norm, eps, out, grads, sizes,
                                              dts, beg, end, st);
        if (e != cudaSuccess) return e;
        beg = end;
    }
    return cudaSuccess;
}

}  // namespace lsr
