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
#include "softmax.cuh"  // keep_elements

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

// ----------------------------------------------------------------------------
// Register-resident rows.  A row is owned by a group of TPR threads (a slice
// of a warp, or TPR / 32 warps) holding CPT 16-byte chunks each; a block of
// relpos_block<TPR>() threads holds several groups that share the head's bias
// and take the rows of a segment in turn.
//
// Chunks lie on 16-byte addresses whatever the row's own start (Tk need not
// be a multiple of the vector): chunk c of a row that starts s elements past
// such an address covers keys c * V - s ... + V - 1, and the first and last
// chunk may reach into the neighbouring rows.  Those elements are read with
// the vector (never past the tensor's ends), ignored, and not written.
//
// Keys outside the window [lo, hi) are invisible: chunks without a visible key
// are not read.  The window of a padding mask (0 and -inf, the keys that are
// not -inf contiguous) is found once per batch entry and block; other masks
// are added element by element.  It is worth finding only when a batch entry
// has several rows of the head in the block (Tq >= kRelposWindowTq): a single
// decoding step would read the whole mask row first and only then the scores.
// ----------------------------------------------------------------------------
constexpr int kRelposWindowTq = 16;
constexpr int kRelposWinMax = 64;  // batch entries of a segment whose windows are kept

template <int TPR>
constexpr int relpos_block() { return TPR < 256 ? 256 : TPR; }

// Window of one mask row, found by one warp; (-1, 0): not a window.  ADDS:
// values other than 0 and -inf matter.
template <typename T, bool ADDS>
__device__ __forceinline__ int2 relpos_mask_window(const T *mrow, int Tk) {
    const int lane = threadIdx.x & 31;
    int first = Tk, last = -1, count = 0, other = 0;
#pragma unroll 4
    for (int j = lane; j < Tk; j += 32) {
        const float v = Traits<T>::load1_cached(mrow + j);
        const bool seen = v != -INFINITY;
        if (ADDS) other |= seen && v != 0.f;
        if (seen) {
            first = min(first, j);
            last = j;
            ++count;
        }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        first = min(first, __shfl_xor_sync(0xffffffffu, first, o));
        last = max(last, __shfl_xor_sync(0xffffffffu, last, o));
        count += __shfl_xor_sync(0xffffffffu, count, o);
        other |= __shfl_xor_sync(0xffffffffu, other, o);
    }
    if (other || (count > 0 && count != last - first + 1)) return make_int2(-1, 0);
    return count == 0 ? make_int2(0, 0) : make_int2(first, last + 1);
}

// Reduction over a row group; one barrier of the group when it has several
// warps.  `red` holds BLOCK / 32 floats that no other reduction in flight uses.
template <int TPR, int BLOCK, typename Op>
__device__ __forceinline__ float relpos_reduce(float v, float *red, int grp) {
    constexpr int W = TPR < 32 ? TPR : 32;
#pragma unroll
    for (int o = W / 2; o > 0; o >>= 1) v = Op::apply(v, __shfl_xor_sync(0xffffffffu, v, o));
    if constexpr (TPR > 32) {
        constexpr int NW = TPR / 32;
        if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
        if constexpr (BLOCK == TPR)
            __syncthreads();
        else
            asm volatile("bar.sync %0, %1;" ::"r"(1 + grp), "r"(TPR) : "memory");
        v = red[grp * NW];
#pragma unroll
        for (int w = 1; w < NW; ++w) v = Op::apply(v, red[grp * NW + w]);
    }
    return v;
}

// Position of a row group in its segment, advanced by G rows without division.
// (The launcher keeps a head's rows below 2^31 - 512, so 32 bits hold them.)
struct RelposCursor {
    int b, i;
    __device__ __forceinline__ RelposCursor(int Tq, int bi) {
        b = bi / Tq;
        i = bi - b * Tq;
    }
    __device__ __forceinline__ void advance(int Tq, int gq, int gr) {
        b += gq;
        i += gr;
        if (i >= Tq) {
            i -= Tq;
            ++b;
        }
    }
};

// Windows of the batch entries of rows [r0, r1) of a head (r0 < r1), into wtab;
// false if there are too many of them or they are not worth finding.
template <typename T, bool ADDS, int BLOCK>
__device__ __forceinline__ bool relpos_find_windows(int2 *wtab, const T *mask, const RelposShape &p,
                                                    int r0, int r1) {
    const int Tq = (int)p.Tq;
    const int b0 = r0 / Tq, nb = (r1 - 1) / Tq - b0 + 1;
    if (!mask || Tq < kRelposWindowTq || nb > kRelposWinMax) return false;
    for (int k = threadIdx.x >> 5; k < nb; k += BLOCK / 32) {
        const int2 w = relpos_mask_window<T, ADDS>(mask + (int64_t)(b0 + k) * p.Tk, (int)p.Tk);
        if ((threadIdx.x & 31) == 0) wtab[k] = w;
    }
    return true;
}

// Chunk of V elements at element offset `at` of a tensor of `total` elements;
// only the elements with bits set are wanted, and at least one of them is.
template <typename T>
__device__ __forceinline__ uint4 relpos_load(const T *base, int64_t at, int64_t total) {
    constexpr int V = Traits<T>::kVec;
    if (at >= 0 && at + V <= total) return ld_stream16(base + at);
    float f[V];
#pragma unroll
    for (int e = 0; e < V; ++e)
        f[e] = at + e >= 0 && at + e < total ? Traits<T>::load1(base + at + e) : 0.f;
    return Traits<T>::pack(f);
}

// Store of a chunk whose first key is j0; keys outside [0, Tk) belong to other
// rows.
template <typename T>
__device__ __forceinline__ void relpos_store(T *row, int j0, int Tk, const uint4 &u) {
    constexpr int V = Traits<T>::kVec;
    if (j0 >= 0 && j0 + V <= Tk) {
        st_stream16(row + j0, u);
        return;
    }
    float f[V];
    Traits<T>::unpack(u, f);
#pragma unroll
    for (int e = 0; e < V; ++e)
        if (j0 + e >= 0 && j0 + e < Tk) Traits<T>::store1(row + j0 + e, f[e]);
}

// Bits of the chunk's visible keys.
template <typename T>
__device__ __forceinline__ uint32_t relpos_bits(const T *mrow, int j0, int lo, int hi) {
    uint32_t bits = 0u;
#pragma unroll
    for (int e = 0; e < Traits<T>::kVec; ++e) {
        bool see = j0 + e >= lo && j0 + e < hi;
        if (mrow && see) see = Traits<T>::load1_cached(mrow + j0 + e) != -INFINITY;
        bits |= (see ? 1u : 0u) << e;
    }
    return bits;
}

// The bias by distance in shared memory: four copies of the 2R + 1 values with
// both ends repeated, copy k shifted by k, so that the V values from any
// distance on start at a 16-byte address of one of them.
template <int V>
__host__ __device__ constexpr int relpos_lut_stride(int R) { return (2 * R + 2 * V + 7) / 4 * 4; }
template <int V>
constexpr size_t relpos_fw_smem(int R) { return (size_t)4 * relpos_lut_stride<V>(R) * 4; }

template <int TPR, int CPT>
constexpr int relpos_fw_min_blocks() {
    return TPR > 256 ? 1 : (CPT <= 1 ? 4 : CPT <= 2 ? 3 : 2);
}

template <typename T, int TPR, int CPT>
__global__ void __launch_bounds__(relpos_block<TPR>(), (relpos_fw_min_blocks<TPR, CPT>()))
relpos_fw_vec(T *out, const T *inp, const T *mask, const T *table, const int32_t *bucket,
              const RelposShape p, int mask_vec) {
    pdl_begin();
    using Tr = Traits<T>;
    constexpr int V = Tr::kVec;
    constexpr int H2 = V / 2;
    constexpr int BLOCK = relpos_block<TPR>();
    constexpr int G = BLOCK / TPR;
    extern __shared__ float4 lut4[];
    float *lut = reinterpret_cast<float *>(lut4);
    __shared__ float red_max[BLOCK / 32], red_sum[BLOCK / 32];
    __shared__ int2 wtab[kRelposWinMax];
    const int lane = threadIdx.x % TPR;
    const int grp = threadIdx.x / TPR;
    const int sub = TPR < 32 ? grp % (32 / (TPR < 32 ? TPR : 32)) : 0;  // group of the warp
    const int Tk = (int)p.Tk, stride = relpos_lut_stride<V>(p.R);
    const int64_t total = p.rows * p.Tk;
    const int Tq = (int)p.Tq, gq = G / Tq, gr = G - gq * Tq;
    const int base_phase = (int)((reinterpret_cast<uintptr_t>(inp) / sizeof(T)) % V);
    const float2 sc = f2(p.scale);

    const int64_t beg = (int64_t)blockIdx.x * p.per;
    const int64_t end = min(beg + p.per, p.rows);
    for (int64_t t0 = beg; t0 < end;) {
        const int64_t h = t0 / p.rows_per_head;
        const int r0 = (int)(t0 - h * p.rows_per_head);
        const int r1 = (int)min(end - h * p.rows_per_head, p.rows_per_head);
        __syncthreads();  // the last segment's bias and windows are no longer read
        for (int x = threadIdx.x; x < stride; x += BLOCK) {
            const float v = relpos_bias<T>(table, bucket, p, h,
                                           min(max(x - V, 0), 2 * p.R));
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (x >= k) lut[k * stride + x - k] = v;
        }
        const bool windows = relpos_find_windows<T, true, BLOCK>(wtab, mask, p, r0, r1);
        const int b0 = r0 / Tq;
        __syncthreads();
        RelposCursor cur(Tq, r0 + grp);
        // groups that share a warp take the same number of turns (shuffles)
        for (int rw = r0 + grp - sub; rw < r1; rw += G, cur.advance(Tq, gq, gr)) {
            const bool valid = rw + sub < r1;
            const int64_t off = (((int64_t)cur.b * p.H + h) * Tq + cur.i) * Tk;
            const int q = cur.i + (int)p.qoff;  // the query's key position
            const int s = (int)((off + base_phase) & (V - 1));
            int lo = 0, hi = valid ? Tk : 0;
            const T *mrow = nullptr;  // set: add the mask element by element
            if (mask && valid) {
                const int2 w = windows ? wtab[cur.b - b0] : make_int2(-1, 0);
                if (w.x < 0) {
                    mrow = mask + (int64_t)cur.b * Tk;
                } else {
                    lo = w.x;
                    hi = w.y;
                }
            }
            if (p.causal) hi = min(hi, q + 1);

            uint4 raw[CPT];
#pragma unroll
            for (int k = 0; k < CPT; ++k) {
                const int j0 = (k * TPR + lane) * V - s;
                if (j0 < hi && j0 + V > lo) raw[k] = relpos_load<T>(inp, off + j0, total);
            }
            float2 v[CPT][H2];
            float m = -INFINITY;
#pragma unroll
            for (int k = 0; k < CPT; ++k) {
                const int j0 = (k * TPR + lane) * V - s;
                if (j0 < hi && j0 + V > lo) {
                    unpack2<T>(raw[k], v[k]);
                    const int u = min(max(j0 - q, -p.R - V), p.R + 1) + p.R + V;
                    const float4 *bias = lut4 + ((u & 3) * stride + (u & ~3)) / 4;
                    float2 bv[H2];
#pragma unroll
                    for (int h2 = 0; h2 < H2; h2 += 2) {
                        const float4 b4 = bias[h2 / 2];
                        bv[h2] = make_float2(b4.x, b4.y);
                        bv[h2 + 1] = make_float2(b4.z, b4.w);
                    }
#pragma unroll
                    for (int h2 = 0; h2 < H2; ++h2) v[k][h2] = fma2(v[k][h2], sc, bv[h2]);
                    if (mrow) {
                        float mv[V];
                        if (mask_vec && j0 >= 0 && j0 + V <= Tk) {
                            Tr::unpack(ld_cached16(mrow + j0), mv);
                        } else {
#pragma unroll
                            for (int e = 0; e < V; ++e)
                                mv[e] = j0 + e >= lo && j0 + e < hi
                                            ? Tr::load1_cached(mrow + j0 + e) : -INFINITY;
                        }
#pragma unroll
                        for (int h2 = 0; h2 < H2; ++h2) {
                            v[k][h2].x = mv[2 * h2] == -INFINITY ? -INFINITY
                                                                 : v[k][h2].x + mv[2 * h2];
                            v[k][h2].y = mv[2 * h2 + 1] == -INFINITY ? -INFINITY
                                                                     : v[k][h2].y + mv[2 * h2 + 1];
                        }
                    }
                    if (j0 < lo || j0 + V > hi) {
#pragma unroll
                        for (int h2 = 0; h2 < H2; ++h2) {
                            const int j = j0 + 2 * h2;
                            if (j < lo || j >= hi) v[k][h2].x = -INFINITY;
                            if (j + 1 < lo || j + 1 >= hi) v[k][h2].y = -INFINITY;
                        }
                    }
#pragma unroll
                    for (int h2 = 0; h2 < H2; ++h2) m = fmax3(m, v[k][h2].x, v[k][h2].y);
                }
            }
            m = relpos_reduce<TPR, BLOCK, OpMax>(m, red_max, grp);
            // e^(z - m): as one fused multiply-add where m * log2 e is finite,
            // else (a row of the type's lowest values) the difference first
            const bool far = !(fabsf(m) < 1e30f);
            const float mm = m == -INFINITY ? 0.f : m;  // nothing visible: all weights 0
            const float2 nmL = f2(-mm * kLog2e), nm = f2(-mm), L2e = f2(kLog2e);
            float2 sum2 = f2(0.f);
#pragma unroll
            for (int k = 0; k < CPT; ++k) {
                const int j0 = (k * TPR + lane) * V - s;
                if (j0 < hi && j0 + V > lo) {
#pragma unroll
                    for (int h2 = 0; h2 < H2; ++h2) {
                        float2 w = far ? mul2(add2(v[k][h2], nm), L2e) : fma2(v[k][h2], L2e, nmL);
                        w.x = fast_exp2(w.x);
                        w.y = fast_exp2(w.y);
                        v[k][h2] = w;
                        sum2 = add2(sum2, w);
                    }
                }
            }
            const float sum =
                relpos_reduce<TPR, BLOCK, OpSum>(sum2.x + sum2.y, red_sum, grp);
            const float inv = sum == 0.f ? 0.f : fast_rcp(sum);
            T *orow = out + off;
#pragma unroll
            for (int k = 0; k < CPT; ++k) {
                const int j0 = (k * TPR + lane) * V - s;
                if (valid && j0 < Tk) {
                    uint4 o = make_uint4(0u, 0u, 0u, 0u);
                    if (j0 < hi && j0 + V > lo) {
                        float2 yv[H2];
#pragma unroll
                        for (int h2 = 0; h2 < H2; ++h2) yv[h2] = mul2(v[k][h2], f2(inv));
                        if (inv != inv) {  // NaN or +inf among the scores: only visible keys
                            const uint32_t bits = relpos_bits<T>(mrow, j0, lo, hi);
#pragma unroll
                            for (int h2 = 0; h2 < H2; ++h2) {
                                if (!((bits >> (2 * h2)) & 1u)) yv[h2].x = 0.f;
                                if (!((bits >> (2 * h2 + 1)) & 1u)) yv[h2].y = 0.f;
                            }
                        }
                        o = pack2<T>(yv);
                    }
                    relpos_store<T>(orow, j0, Tk, o);
                }
            }
        }
        t0 = h * p.rows_per_head + r1;
    }
}

// ----------------------------------------------------------------------------
// Register-resident backward.  Each row group adds its rows' dz by distance
// into its own array of the distances [rmin, rmin + width) that are not
// clipped and can occur, index x stored at x + x / 32: a lane's V keys are
// neighbours, so lanes access with a stride of V, which the gap spreads over
// the banks.
// ----------------------------------------------------------------------------
struct RelposBand {
    int rmin, width, stride;  // stride: floats of a group's array
};
__host__ __device__ inline RelposBand relpos_band(const RelposShape &p) {
    const int64_t last = p.causal ? 0 : p.Tq - 1;  // the largest j - q
    const int rmin = (int)(-p.R + 1 > 1 - p.Tk ? -p.R + 1 : 1 - p.Tk);
    const int rmax = (int)(p.R - 1 < last ? p.R - 1 : last);
    RelposBand b;
    b.rmin = rmin;
    b.width = rmax >= rmin ? rmax - rmin + 1 : 0;
    b.stride = b.width + b.width / 32 + 1;
    return b;
}

template <int TPR, int CPT>
constexpr int relpos_bw_resident() {
    return TPR > 256 ? 1 : (CPT <= 1 ? 4 : CPT <= 2 ? 3 : 2);
}

template <typename T, int TPR, int CPT>
__global__ void __launch_bounds__(relpos_block<TPR>(), (relpos_bw_resident<TPR, CPT>()))
relpos_bw_vec(T *dinp, float *part, const T *dout, const T *y, const T *mask,
              const RelposShape p) {
    pdl_begin();
    using Tr = Traits<T>;
    constexpr int V = Tr::kVec;
    constexpr int H2 = V / 2;
    constexpr int BLOCK = relpos_block<TPR>();
    constexpr int G = BLOCK / TPR;
    extern __shared__ float acc[];  // [G][band.stride]
    __shared__ float red[2][BLOCK / 32];
    __shared__ float ends[2][G];
    __shared__ int2 wtab[kRelposWinMax];
    const int lane = threadIdx.x % TPR;
    const int grp = threadIdx.x / TPR;
    const int sub = TPR < 32 ? grp % (32 / (TPR < 32 ? TPR : 32)) : 0;  // group of the warp
    const int Tk = (int)p.Tk;
    const RelposBand band = relpos_band(p);
    float *mine = acc + grp * band.stride;
    const int64_t total = p.rows * p.Tk;
    const int Tq = (int)p.Tq, gq = G / Tq, gr = G - gq * Tq;
    const int base_phase = (int)((reinterpret_cast<uintptr_t>(y) / sizeof(T)) % V);

    const int64_t beg = (int64_t)blockIdx.x * p.per;
    const int64_t end = min(beg + p.per, p.rows);
    for (int64_t t0 = beg; t0 < end;) {
        const int64_t h = t0 / p.rows_per_head;
        const int r0 = (int)(t0 - h * p.rows_per_head);
        const int r1 = (int)min(end - h * p.rows_per_head, p.rows_per_head);
        for (int x = threadIdx.x; x < G * band.stride; x += BLOCK) acc[x] = 0.f;
        const bool windows = relpos_find_windows<T, false, BLOCK>(wtab, mask, p, r0, r1);
        const int b0 = r0 / Tq;
        __syncthreads();
        float lo_sum = 0.f, hi_sum = 0.f;  // the clipped ends
        int turn = 0;
        RelposCursor cur(Tq, r0 + grp);
        // groups that share a warp take the same number of turns (shuffles)
        for (int rw = r0 + grp - sub; rw < r1; rw += G, cur.advance(Tq, gq, gr)) {
            const bool valid = rw + sub < r1;
            const int64_t off = (((int64_t)cur.b * p.H + h) * Tq + cur.i) * Tk;
            const int q = cur.i + (int)p.qoff;
            const int s0 = (int)((off + base_phase) & (V - 1));
            int lo = 0, hi = valid ? Tk : 0;
            const T *mrow = nullptr;
            if (mask && valid) {
                const int2 w = windows ? wtab[cur.b - b0] : make_int2(-1, 0);
                if (w.x < 0) {
                    mrow = mask + (int64_t)cur.b * Tk;
                } else {
                    lo = w.x;
                    hi = w.y;
                }
            }
            if (p.causal) hi = min(hi, q + 1);

            uint4 yr[CPT], gr4[CPT];
#pragma unroll
            for (int k = 0; k < CPT; ++k) {
                const int j0 = (k * TPR + lane) * V - s0;
                yr[k] = gr4[k] = make_uint4(0u, 0u, 0u, 0u);
                if (j0 < hi && j0 + V > lo) {
                    yr[k] = relpos_load<T>(y, off + j0, total);
                    gr4[k] = relpos_load<T>(dout, off + j0, total);
                }
            }
#pragma unroll
            for (int k = 0; k < CPT; ++k) {
                const int j0 = (k * TPR + lane) * V - s0;
                if (j0 < hi && j0 + V > lo && (mrow || j0 < lo || j0 + V > hi)) {
                    const uint32_t bits = relpos_bits<T>(mrow, j0, lo, hi);
                    keep_elements<T>(yr[k], bits);
                    keep_elements<T>(gr4[k], bits);
                }
            }
            float2 s2 = f2(0.f);
#pragma unroll
            for (int k = 0; k < CPT; ++k) {
                float2 yv[H2], gv[H2];
                unpack2<T>(yr[k], yv);
                unpack2<T>(gr4[k], gv);
#pragma unroll
                for (int h2 = 0; h2 < H2; ++h2) s2 = fma2(yv[h2], gv[h2], s2);
            }
            // the group's barrier also orders this row's additions after the
            // last row's; `red` alternates so that one barrier is enough
            const float s =
                relpos_reduce<TPR, BLOCK, OpSum>(s2.x + s2.y, red[turn], grp);
            turn ^= 1;
#pragma unroll
            for (int k = 0; k < CPT; ++k) {
                const int j0 = (k * TPR + lane) * V - s0;
                if (!valid || j0 >= Tk) continue;
                float2 yv[H2], gv[H2], dz[H2], dx[H2];
                unpack2<T>(yr[k], yv);
                unpack2<T>(gr4[k], gv);
#pragma unroll
                for (int h2 = 0; h2 < H2; ++h2)
                    dz[h2] = mul2(yv[h2], add2(gv[h2], f2(-s)));
                const bool see = j0 < hi && j0 + V > lo;
                if (!(fabsf(s) < INFINITY)) {  // 0 * NaN: invisible keys stay 0
                    const uint32_t bits = see ? relpos_bits<T>(mrow, j0, lo, hi) : 0u;
#pragma unroll
                    for (int h2 = 0; h2 < H2; ++h2) {
                        if (!((bits >> (2 * h2)) & 1u)) dz[h2].x = 0.f;
                        if (!((bits >> (2 * h2 + 1)) & 1u)) dz[h2].y = 0.f;
                    }
                }
#pragma unroll
                for (int h2 = 0; h2 < H2; ++h2) dx[h2] = mul2(dz[h2], f2(p.scale));
                relpos_store<T>(dinp + off, j0, Tk, pack2<T>(dx));
                if (!see) continue;
                const int d0 = j0 - q, x0 = d0 - band.rmin;
                if (x0 >= 0 && x0 + V <= band.width) {
                    float a[V];
#pragma unroll
                    for (int e = 0; e < V; ++e) a[e] = mine[x0 + e + (x0 + e) / 32];
#pragma unroll
                    for (int h2 = 0; h2 < H2; ++h2) {
                        a[2 * h2] += dz[h2].x;
                        a[2 * h2 + 1] += dz[h2].y;
                    }
#pragma unroll
                    for (int e = 0; e < V; ++e) mine[x0 + e + (x0 + e) / 32] = a[e];
                } else if (d0 + V - 1 <= -p.R || d0 >= p.R) {
                    float2 t = dz[0];
#pragma unroll
                    for (int h2 = 1; h2 < H2; ++h2) t = add2(t, dz[h2]);
                    if (d0 < 0)
                        lo_sum += t.x + t.y;
                    else
                        hi_sum += t.x + t.y;
                } else {
#pragma unroll
                    for (int e = 0; e < V; ++e) {
                        const float d = e % 2 ? dz[e / 2].y : dz[e / 2].x;
                        const int x = x0 + e;
                        if (x >= 0 && x < band.width)
                            mine[x + x / 32] += d;
                        else if (d0 + e <= -p.R)
                            lo_sum += d;
                        else if (d0 + e >= p.R)
                            hi_sum += d;
                    }
                }
            }
            if constexpr (TPR <= 32) __syncwarp();
        }
        // the groups' ends: lanes of a group, then its warps
        __shared__ float wends[2][BLOCK / 32];
        constexpr int W = TPR < 32 ? TPR : 32;
        __syncwarp();
#pragma unroll
        for (int o = W / 2; o > 0; o >>= 1) {
            lo_sum += __shfl_xor_sync(0xffffffffu, lo_sum, o);
            hi_sum += __shfl_xor_sync(0xffffffffu, hi_sum, o);
        }
        if constexpr (TPR > 32) {
            if ((threadIdx.x & 31) == 0) {
                wends[0][threadIdx.x >> 5] = lo_sum;
                wends[1][threadIdx.x >> 5] = hi_sum;
            }
            __syncthreads();
            if (lane < 2) {
                float v = 0.f;
                for (int w = 0; w < TPR / 32; ++w) v += wends[lane][grp * (TPR / 32) + w];
                ends[lane][grp] = v;
            }
        } else if (lane == 0) {
            ends[0][grp] = lo_sum;
            ends[1][grp] = hi_sum;
        }
        __syncthreads();
        const int W2 = 2 * p.R + 1;
        float *slot = part + ((int64_t)blockIdx.x + h) * W2;
        for (int d = threadIdx.x; d < W2; d += BLOCK) {
            float v = 0.f;
            const int x = d - p.R - band.rmin;
            if (d == 0 || d == 2 * p.R) {
                for (int g = 0; g < G; ++g) v += ends[d ? 1 : 0][g];
            } else if (x >= 0 && x < band.width) {
                for (int g = 0; g < G; ++g) v += acc[g * band.stride + x + x / 32];
            }
            slot[d] = v;
        }
        __syncthreads();
        t0 = h * p.rows_per_head + r1;
    }
}

// dtable[k, h] for one head h = blockIdx.x and the buckets of blockIdx.y:
// segment sums of each distance in order, then each bucket's distances.
constexpr int kRelposFoldBuckets = 32;
static __global__ void __launch_bounds__(256)
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
