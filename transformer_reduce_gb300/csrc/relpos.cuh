// relpos.cuh -- attention softmax with a learned relative position bias by
// buckets, forward and backward (sm_103a).
//
// For query i (the Tq queries are the last Tq of the Tk key positions) and key
// j, with qoff = Tk - Tq and R = max_distance:
//     r    = min(max(j - (i + qoff), -R), R)
//     z_ij = scale * x_ij + table[bucket[r + R], h] + mask[b, j]
//     y    = softmax over the visible j of z_i
// Backward, on visible keys:
//     dz   = y (dy - sum y dy),   dx = scale * dz,
//     dtable[k, h] = sum over every b, i, j with bucket[r + R] == k of dz
//
// The bias of a head depends on j - i alone, so a head's whole bias is 2R + 1
// numbers: a block works on rows of one head at a time and keeps them in
// shared memory, looked up by distance, instead of reading a [H, Tq, Tk] bias
// from memory.  Blocks own contiguous runs of rows in head-major order
// (h, b, i); a run that crosses heads is cut into segments of one head, with
// the bias rebuilt between them, so any number of heads fills the GPU evenly.
//
// The table's gradient needs sums over all rows by distance.  The keys of one
// row have distinct distances, so a row group adds its row into its own array
// of 2R - 1 sums in shared memory without any conflict, each entry touched by
// one thread per row; the two clipped ends (r = -R, r = R), where many keys
// share an entry, are summed in registers.  Each (block, segment) writes its
// 2R + 1 sums to the workspace; a second kernel adds a head's segments in
// order and then the distances of each bucket in order.  No atomics: the
// result depends only on the problem, never on scheduling.
#pragma once

#include "launch.h"
#include "ls_device.cuh"

namespace lsr {

// Bias of head h at clipped distance d - R; an id outside the table adds
// nothing (and its gradient goes nowhere).
template <typename T>
__device__ __forceinline__ float relpos_bias(const T *table, const int32_t *bucket,
                                             const RelposShape &p, int64_t h, int d) {
    const int32_t id = __ldg(bucket + d);
    return id >= 0 && id < p.num_buckets ? Traits<T>::load1_cached(table + id * p.H + h) : 0.f;
}

// Online pair (m, s) standing for s * e^m, merged across a row group.
// Natural units: a row whose every key carries the lowest value of the
// storage type still has a finite maximum, which log2 units would overflow.
__device__ __forceinline__ void natural_merge(float &m, float &s, float m2, float s2) {
    const float mn = fmaxf(m, m2);
    if (mn == -INFINITY) {
        s += s2;  // empty, or NaN sums of rows without a comparable key
        return;
    }
    s = (m == -INFINITY ? s : s * fast_exp2((m - mn) * kLog2e)) +
        (m2 == -INFINITY ? s2 : s2 * fast_exp2((m2 - mn) * kLog2e));
    m = mn;
}
template <int TPR>
__device__ __forceinline__ void group_natural_merge(float &m, float &s, float *smem) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const float m2 = __shfl_xor_sync(0xffffffffu, m, o);
        const float s2 = __shfl_xor_sync(0xffffffffu, s, o);
        natural_merge(m, s, m2, s2);
    }
    if constexpr (TPR > 32) {
        const int warp = threadIdx.x >> 5;
        if ((threadIdx.x & 31) == 0) {
            smem[warp] = m;
            smem[32 + warp] = s;
        }
        __syncthreads();
        m = smem[0];
        s = smem[32];
        for (int w = 1; w < TPR / 32; ++w) natural_merge(m, s, smem[w], smem[32 + w]);
        __syncthreads();
    }
}

// ----------------------------------------------------------------------------
// Forward, any length and alignment: TPR threads per row (a warp, or the whole
// block for long rows), scalar accesses, an online pass and a second pass that
// reads the row again and writes it.
// ----------------------------------------------------------------------------
template <typename T, int TPR>
__global__ void __launch_bounds__(256)
relpos_fw_loop(T *out, const T *inp, const T *mask, const T *table, const int32_t *bucket,
               const RelposShape p) {
    pdl_begin();
    using Tr = Traits<T>;
    constexpr int G = 256 / TPR;
    extern __shared__ float lut[];  // [2R + 1]
    __shared__ float red[64];
    const int lane = threadIdx.x % TPR;
    const int grp = threadIdx.x / TPR;
    const int64_t beg = (int64_t)blockIdx.x * p.per;
    const int64_t end = min(beg + p.per, p.rows);
    for (int64_t t0 = beg; t0 < end;) {
        const int64_t h = t0 / p.rows_per_head;
        const int64_t seg_end = min(end, (h + 1) * p.rows_per_head);
        __syncthreads();
        for (int d = threadIdx.x; d <= 2 * p.R; d += 256)
            lut[d] = relpos_bias<T>(table, bucket, p, h, d);
        __syncthreads();
        for (int64_t t = t0 + grp; t < seg_end; t += G) {
            const int64_t bi = t - h * p.rows_per_head;
            const int64_t b = bi / p.Tq, i = bi - b * p.Tq;
            const int64_t off = ((b * p.H + h) * p.Tq + i) * p.Tk;
            const int64_t q = i + p.qoff;  // the query's key position
            const int64_t jend = p.causal ? min(p.Tk, q + 1) : p.Tk;
            const T *x = inp + off;
            const T *mrow = mask ? mask + b * p.Tk : nullptr;
            auto score = [&](int64_t j, float mv) {
                const int64_t r = min(max(j - q, (int64_t)-p.R), (int64_t)p.R);
                return fmaf(Tr::load1(x + j), p.scale, lut[r + p.R]) + mv;
            };
            float m = -INFINITY, s = 0.f;
            for (int64_t j = lane; j < jend; j += TPR) {
                const float mv = mrow ? Tr::load1_cached(mrow + j) : 0.f;
                if (mv == -INFINITY) continue;
                const float z = score(j, mv);
                if (z > m) {
                    s = (m == -INFINITY ? s : s * fast_exp2((m - z) * kLog2e)) + 1.f;
                    m = z;
                } else if (z != -INFINITY) {
                    s += fast_exp2((z - m) * kLog2e);
                }
            }
            group_natural_merge<TPR>(m, s, red);
            // a score of +inf makes the whole row NaN, as the formula does
            const float inv = m == INFINITY ? __int_as_float(0x7fc00000)
                                            : (s == 0.f ? 0.f : 1.f / s);
            const float mm = m == -INFINITY ? 0.f : m;
            T *o = out + off;
            for (int64_t j = lane; j < p.Tk; j += TPR) {
                float yv = 0.f;
                if (j < jend) {
                    const float mv = mrow ? Tr::load1_cached(mrow + j) : 0.f;
                    if (mv != -INFINITY) yv = fast_exp2((score(j, mv) - mm) * kLog2e) * inv;
                }
                Tr::store1(o + j, yv);
            }
        }
        t0 = seg_end;
    }
}

// ----------------------------------------------------------------------------
// Backward, any length and alignment.
// ----------------------------------------------------------------------------
template <typename T, int TPR>
__global__ void __launch_bounds__(256)
relpos_bw_loop(T *dinp, float *part, const T *dout, const T *y, const T *mask,
               const RelposShape p) {
    pdl_begin();
    using Tr = Traits<T>;
    constexpr int G = 256 / TPR;
    extern __shared__ float acc[];  // [G][2R + 1]
    __shared__ float red[64];
    const int lane = threadIdx.x % TPR;
    const int grp = threadIdx.x / TPR;
    const int W = 2 * p.R + 1;
    float *mine = acc + grp * W;
    const int64_t beg = (int64_t)blockIdx.x * p.per;
    const int64_t end = min(beg + p.per, p.rows);
    for (int64_t t0 = beg; t0 < end;) {
        const int64_t h = t0 / p.rows_per_head;
        const int64_t seg_end = min(end, (h + 1) * p.rows_per_head);
        for (int d = threadIdx.x; d < G * W; d += 256) acc[d] = 0.f;
        __syncthreads();
        float lo_sum = 0.f, hi_sum = 0.f;  // the clipped ends
        for (int64_t t = t0 + grp; t < seg_end; t += G) {
            const int64_t bi = t - h * p.rows_per_head;
            const int64_t b = bi / p.Tq, i = bi - b * p.Tq;
            const int64_t off = ((b * p.H + h) * p.Tq + i) * p.Tk;
            const int64_t q = i + p.qoff;
            const int64_t jend = p.causal ? min(p.Tk, q + 1) : p.Tk;
            const T *mrow = mask ? mask + b * p.Tk : nullptr;
            float s = 0.f;
            for (int64_t j = lane; j < jend; j += TPR) {
                if (mrow && Tr::load1_cached(mrow + j) == -INFINITY) continue;
                s = fmaf(Tr::load1(y + off + j), Tr::load1(dout + off + j), s);
            }
            // for a whole-block row the barriers inside also order this row's
            // additions after the last row's
            s = group_reduce<TPR, OpSum>(s, red);
            for (int64_t j = lane; j < p.Tk; j += TPR) {
                float dz = 0.f;
                if (j < jend && !(mrow && Tr::load1_cached(mrow + j) == -INFINITY)) {
                    dz = Tr::load1(y + off + j) * (Tr::load1(dout + off + j) - s);
                    const int64_t r = j - q;
                    if (r <= -p.R)
                        lo_sum += dz;
                    else if (r >= p.R)
                        hi_sum += dz;
                    else
                        mine[r + p.R] += dz;
                }
                Tr::store1(dinp + off + j, p.scale * dz);
            }
            if constexpr (TPR == 32) __syncwarp();
        }
        lo_sum = group_reduce<TPR, OpSum>(lo_sum, red);
        hi_sum = group_reduce<TPR, OpSum>(hi_sum, red);
        if (lane == 0) {
            mine[0] = lo_sum;
            mine[2 * p.R] = hi_sum;
        }
        __syncthreads();
        float *slot = part + ((int64_t)blockIdx.x + h) * W;
        for (int d = threadIdx.x; d < W; d += 256) {
            float v = acc[d];
            for (int g = 1; g < G; ++g) v += acc[g * W + d];
            slot[d] = v;
        }
        __syncthreads();
        t0 = seg_end;
    }
}

// dtable[k, h] for one head h = blockIdx.x and the buckets of blockIdx.y:
// segment sums of each distance in order, then each bucket's distances.
constexpr int kRelposFoldBuckets = 32;
__global__ void __launch_bounds__(256)
relpos_fold(float *dtable, const float *part, const int32_t *bucket, const RelposShape p) {
    pdl_begin();
    extern __shared__ float dist[];  // [2R + 1]
    const int W = 2 * p.R + 1;
    const int64_t h = blockIdx.x;
    const bool any = p.rows_per_head > 0;
    const int64_t first = any ? h * p.rows_per_head / p.per : 0;
    const int64_t last = any ? ((h + 1) * p.rows_per_head - 1) / p.per : -1;
    for (int d = threadIdx.x; d < W; d += 256) {
        float v = 0.f;
#pragma unroll 8
        for (int64_t k = first; k <= last; ++k) v += __ldg(part + (k + h) * W + d);
        dist[d] = v;
    }
    __syncthreads();
    const int lane = threadIdx.x & 31;
    const int64_t k0 = (int64_t)blockIdx.y * kRelposFoldBuckets;
    for (int64_t k = k0 + (threadIdx.x >> 5); k < min(k0 + kRelposFoldBuckets, p.num_buckets);
         k += 8) {
        float v = 0.f;
        for (int d = lane; d < W; d += 32)
            if (__ldg(bucket + d) == k) v += dist[d];
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
        if (lane == 0) dtable[k * p.H + h] = v;
    }
}

}  // namespace lsr
