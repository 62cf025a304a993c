// grad_clip.cu -- global gradient norm over many tensors of mixed storage
// types, and clipping by it (sm_103a).
//
//     norm = sqrt(sum over all tensors and elements of g^2)
//     out  = g * min(1, max_norm / (norm + eps))
//
// The list of tensors travels in the kernel's parameters (29 bytes a tensor,
// up to kGradCap of them a launch), so nothing is copied to the device and a
// captured graph carries its list.  Tensors are cut into chunks of 16-byte
// slots; a block of 256 threads takes a chunk at a time, eight slots per
// thread in flight together (four for short lists, which would not fill the GPU
// otherwise), and finds the chunk's tensor by bisection.
// Slots lie on 16-byte addresses whatever the tensor's own alignment; the
// first and last slot of a tensor are taken element by element.
//
// Every block leaves one FP64 partial sum.  The clipping kernel needs no third
// launch for the total: each of its blocks adds the (at most 608 per launch)
// partials itself, in the same fixed order, and takes the chunks from the end
// of the list, which the norm's pass read last and L2 still holds.  The cut
// depends only on the list (its sizes, dtypes and offsets within 16 bytes), so
// the norm of the same call is bitwise reproducible.
//
// Bound by memory: 144 tensors of 151 M bf16 elements, norm 48.7 us (6.2 TB/s),
// norm and scaling 152.8 us (5.9 TB/s); short lists by the two launches (12
// tensors of 0.8 M: 7.2 us).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <type_traits>

#include "dispatch.cuh"
#include "launch.h"
#include "ls_device.cuh"
#include "ls_reduce.h"

namespace lsr {
namespace {

constexpr int kGradBlock = 256;
// 16-byte slots per thread and chunk: eight, so that a thread has 128 bytes in
// flight, or four where eight would leave blocks of the norm without a chunk
// (12 tensors of 0.8 M elements: 7.1 us with four, 8.9 with eight, 10.2 with
// two; 150 tensors of 2.9 M: 16.1, 16.5, 17.5).
constexpr int kGradSlots = 8, kGradFewSlots = 4;
constexpr int64_t kGradBlocks = 4 * 152;  // partial sums of a launch, a constant of the library
constexpr int kGradCap = 512;             // tensors of a launch
constexpr int kGradSmallCap = 48;         // a shorter list has a parameter block of its own

template <int CAP>
struct GradList {
    int32_t count, chunks;
    int32_t chunk0[CAP];  // first chunk of each tensor (read by the bisection: close together)
    uint8_t dt[CAP];
    const void *g[CAP];
    void *o[CAP];
    int64_t n[CAP];
};
// One tensor's part of a list.
struct GradSpan {
    const void *g;
    void *o;
    int64_t n;
    int dt;
    int64_t chunk;  // of the tensor
};

// Element at the 16-byte address at or below p, relative to p.
template <typename T>
__device__ __forceinline__ int64_t grad_first_element(const void *p) {
    return -(int64_t)((reinterpret_cast<uintptr_t>(p) & 15u) / sizeof(T));
}

int64_t grad_slots(const void *p, int64_t n, int es) {
    return n > 0 ? ceil_div(n * es + (int64_t)(reinterpret_cast<uintptr_t>(p) & 15u), 16) : 0;
}

int grad_es(int dt) { return dt == LS_F32 ? 4 : 2; }

// The tensor of a chunk: the last one whose chunk0 <= chunk (tensors without
// elements share their successor's chunk0 and are never the last).
template <int CAP>
__device__ __forceinline__ GradSpan grad_find(const GradList<CAP> &L, int chunk) {
    int lo = 0, hi = L.count;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (L.chunk0[mid] <= chunk)
            lo = mid;
        else
            hi = mid;
    }
    return GradSpan{L.g[lo], L.o[lo], L.n[lo], L.dt[lo], chunk - L.chunk0[lo]};
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
template <typename T, int U>
__device__ __forceinline__ double grad_chunk_squares(const GradSpan &sp) {
    constexpr int V = Traits<T>::kVec;
    const T *g = static_cast<const T *>(sp.g);
    const int64_t e0 =
        grad_first_element<T>(sp.g) +
        (sp.chunk * (kGradBlock * U) + threadIdx.x) * V;
    uint4 raw[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int64_t e = e0 + (int64_t)u * kGradBlock * V;
        raw[u] = e < sp.n ? grad_load<T>(g, e, sp.n) : make_uint4(0u, 0u, 0u, 0u);
    }
    float2 s2 = f2(0.f);
#pragma unroll
    for (int u = 0; u < U; ++u) {
        float2 v[V / 2];
        unpack2<T>(raw[u], v);
#pragma unroll
        for (int h = 0; h < V / 2; ++h) s2 = fma2(v[h], v[h], s2);
    }
    const float s = s2.x + s2.y;
    if (s > 0x1p-90f && s < INFINITY) return (double)s;
    uint32_t any = 0u;
#pragma unroll
    for (int u = 0; u < U; ++u) any |= raw[u].x | raw[u].y | raw[u].z | raw[u].w;
    if (any == 0u) return 0.0;
    double d = 0.0;
#pragma unroll 1
    for (int u = 0; u < U; ++u) {
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

template <int CAP, int U>
__global__ void __launch_bounds__(kGradBlock)
grad_squares(double *part, const __grid_constant__ GradList<CAP> L) {
    pdl_begin();
    double d = 0.0;
    for (int c = blockIdx.x; c < L.chunks; c += gridDim.x) {
        const GradSpan sp = grad_find(L, c);
        if (sp.dt == LS_F32)
            d += grad_chunk_squares<float, U>(sp);
        else if (sp.dt == LS_F16)
            d += grad_chunk_squares<__half, U>(sp);
        else
            d += grad_chunk_squares<__nv_bfloat16, U>(sp);
    }
    d = grad_block_sum(d);
    if (threadIdx.x == 0) part[blockIdx.x] = d;
}

// The norm from all partials, the same in every block that asks.
__device__ __forceinline__ float grad_total_norm(const double *part, int parts) {
    double d = 0.0;
    for (int i = threadIdx.x; i < parts; i += kGradBlock) d += __ldcg(part + i);
    return (float)sqrt(grad_block_sum(d));
}

__global__ void __launch_bounds__(kGradBlock)
grad_norm_final(float *norm, const double *part, int parts) {
    pdl_begin();
    const float v = grad_total_norm(part, parts);
    if (threadIdx.x == 0) *norm = v;
}

template <typename T, int U>
__device__ __forceinline__ void grad_chunk_scale(const GradSpan &sp, float coef) {
    constexpr int V = Traits<T>::kVec;
    const T *g = static_cast<const T *>(sp.g);
    T *o = static_cast<T *>(sp.o);
    const bool same =
        ((reinterpret_cast<uintptr_t>(g) ^ reinterpret_cast<uintptr_t>(o)) & 15u) == 0;
    const int64_t e0 =
        grad_first_element<T>(sp.g) +
        (sp.chunk * (kGradBlock * U) + threadIdx.x) * V;
    uint4 raw[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int64_t e = e0 + (int64_t)u * kGradBlock * V;
        if (e < sp.n) {
            if (e >= 0 && e + V <= sp.n)
                raw[u] = *reinterpret_cast<const uint4 *>(g + e);
            else
                raw[u] = grad_load<T>(g, e, sp.n);
        }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
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

template <int CAP, int U>
__global__ void __launch_bounds__(kGradBlock)
grad_scale(float *norm, const double *part, int parts, float max_norm, float eps,
           const __grid_constant__ GradList<CAP> L) {
    pdl_begin();
    const float total = grad_total_norm(part, parts);
    if (blockIdx.x == 0 && threadIdx.x == 0) *norm = total;
    const float ratio = max_norm / (total + eps);
    const float coef = ratio >= 1.f ? 1.f : ratio;  // a NaN norm gives NaN
    for (int k = blockIdx.x; k < L.chunks; k += gridDim.x) {
        const GradSpan sp = grad_find(L, L.chunks - 1 - k);
        if (coef == 1.f && sp.o == sp.g) continue;  // in place and nothing to clip
        if (sp.dt == LS_F32)
            grad_chunk_scale<float, U>(sp, coef);
        else if (sp.dt == LS_F16)
            grad_chunk_scale<__half, U>(sp, coef);
        else
            grad_chunk_scale<__nv_bfloat16, U>(sp, coef);
    }
}

// A caller's list on the host.
struct GradHost {
    void *const *out;  // NULL: a norm alone
    const void *const *grads;
    const int64_t *sizes;
    const int32_t *dts;
    int64_t count;
};

// One launch's list from tensors [beg, end), cut into chunks of U slots per
// thread.  (The ABI bounds the elements of a list, so chunks fit 31 bits.)
template <int CAP>
void grad_fill(GradList<CAP> &L, const GradHost &a, int64_t beg, int64_t end, int U) {
    L.count = (int)(end - beg);
    int64_t chunks = 0;
    for (int64_t i = beg; i < end; ++i) {
        const int64_t k = i - beg;
        L.g[k] = a.grads[i];
        L.o[k] = a.out ? a.out[i] : nullptr;
        L.n[k] = a.sizes[i];
        L.dt[k] = (uint8_t)a.dts[i];
        L.chunk0[k] = (int32_t)chunks;
        chunks += ceil_div(grad_slots(a.grads[i], a.sizes[i], grad_es(a.dts[i])),
                           (int64_t)kGradBlock * U);
    }
    L.chunks = (int32_t)chunks;
}

template <int CAP, int U>
cudaError_t grad_squares_launch(double *part, const GradHost &a, int64_t beg, int64_t end,
                                int *parts, cudaStream_t st) {
    GradList<CAP> L;
    grad_fill<CAP>(L, a, beg, end, U);
    *parts = (int)(L.chunks < kGradBlocks ? L.chunks : kGradBlocks);
    if (*parts == 0) return cudaSuccess;
    return launch_pdl(grad_squares<CAP, U>, dim3((unsigned)*parts), dim3(kGradBlock), 0, st, part,
                      L);
}

template <int CAP, int U>
cudaError_t grad_scale_launch(float *norm, const double *part, int parts, float max_norm,
                              float eps, const GradHost &a, int64_t beg, int64_t end,
                              cudaStream_t st) {
    GradList<CAP> L;
    grad_fill<CAP>(L, a, beg, end, U);
    return launch_persistent<grad_scale<CAP, U>>(kGradBlock, 0, L.chunks, st, norm, part, parts,
                                                 max_norm, eps, L);
}

// Whether the list is small enough for chunks of few slots.
bool grad_few(const GradHost &a) {
    int64_t slots = 0;
    for (int64_t i = 0; i < a.count; ++i)
        slots += grad_slots(a.grads[i], a.sizes[i], grad_es(a.dts[i]));
    return slots < kGradBlocks * kGradBlock * kGradSlots;
}

// Calls f(beg, end, list capacity, slots per thread) for every launch.
template <typename F>
cudaError_t grad_launches(const GradHost &a, F f) {
    const bool few = grad_few(a);
    using Few = std::integral_constant<int, kGradFewSlots>;
    using Many = std::integral_constant<int, kGradSlots>;
    using Small = std::integral_constant<int, kGradSmallCap>;
    using Full = std::integral_constant<int, kGradCap>;
    for (int64_t beg = 0; beg < a.count; beg += kGradCap) {
        const int64_t end = beg + kGradCap < a.count ? beg + kGradCap : a.count;
        const bool small = end - beg <= kGradSmallCap;
        const cudaError_t e = small ? (few ? f(beg, end, Small(), Few()) : f(beg, end, Small(), Many()))
                                    : (few ? f(beg, end, Full(), Few()) : f(beg, end, Full(), Many()));
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

// Partials of every tensor; *parts: how many were left at `part`.
cudaError_t grad_all_squares(const GradHost &a, double *part, int *parts, cudaStream_t st) {
    *parts = 0;
    return grad_launches(a, [&](int64_t beg, int64_t end, auto cap, auto slots) {
        int n = 0;
        const cudaError_t e = grad_squares_launch<decltype(cap)::value, decltype(slots)::value>(
            part + *parts, a, beg, end, &n, st);
        *parts += n;
        return e;
    });
}

}  // namespace

int64_t grad_parts(int64_t count) {
    return count > 0 ? kGradBlocks * ceil_div(count, kGradCap) : 0;
}

cudaError_t launch_grad_norm(float *norm, const void *const *grads, const int64_t *sizes,
                             const int32_t *dts, int64_t count, double *part, cudaStream_t st) {
    const GradHost a = {nullptr, grads, sizes, dts, count};
    int parts = 0;
    const cudaError_t e = grad_all_squares(a, part, &parts, st);
    if (e != cudaSuccess) return e;
    return launch_pdl(grad_norm_final, dim3(1), dim3(kGradBlock), 0, st, norm,
                      (const double *)part, parts);
}

cudaError_t launch_grad_clip(float *norm, void *const *out, const void *const *grads,
                             const int64_t *sizes, const int32_t *dts, int64_t count,
                             float max_norm, float eps, double *part, cudaStream_t st) {
    const GradHost a = {out, grads, sizes, dts, count};
    int parts = 0;
    const cudaError_t e = grad_all_squares(a, part, &parts, st);
    if (e != cudaSuccess) return e;
    if (parts == 0)
        return launch_pdl(grad_norm_final, dim3(1), dim3(kGradBlock), 0, st, norm,
                          (const double *)part, 0);
    return grad_launches(a, [&](int64_t beg, int64_t end, auto cap, auto slots) {
        return grad_scale_launch<decltype(cap)::value, decltype(slots)::value>(
            norm, part, parts, max_norm, eps, a, beg, end, st);
    });
}

}  // namespace lsr
