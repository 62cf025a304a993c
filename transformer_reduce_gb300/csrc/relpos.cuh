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
// result depends only on the problem (and on the tensors' offsets within 16
// bytes, which choose the kernel), never on scheduling.
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

// ----------------------------------------------------------------------------
// Forward, any length and alignment: TPR threads per row (a warp, or the whole
// block for long rows), scalar accesses, an online pass and a second pass that
// reads the row again and writes it.  Bound by issue (69 % of the slots, one
// element per instruction): [32,16,512,512] bf16 611 us here, 87 in the kernel
// below, which takes all but the longest rows and tensors at different offsets.
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
// Backward, any length and alignment, as the looped forward ([32,16,512,512]
// bf16: 832 us here, 134 in the kernel below).
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
// With windows / without, forward and backward, 16 heads, 512 keys of bf16,
// 4096 rows per head: Tq = 1 38.8 / 35.7 and 148.9 / 149.3 us; Tq = 4 30.2 /
// 34.1 and 55.7 / 74.7; Tq = 64 25.0 / 30.2 and 46.9 / 66.5.
// ----------------------------------------------------------------------------
constexpr int kRelposWindowTq = 4;
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
struct RelposStep {
    int gq, gr;             // G = gq * Tq + gr
    int64_t step, wrap;     // elements of G rows within the tensor, and of a batch entry's end
    __device__ __forceinline__ RelposStep(const RelposShape &p, int G) {
        const int Tq = (int)p.Tq;
        gq = G / Tq;
        gr = G - gq * Tq;
        step = ((int64_t)gq * p.H * Tq + gr) * p.Tk;
        wrap = (p.H - 1) * Tq * p.Tk;
    }
};
struct RelposCursor {
    int b, i;
    int64_t off;  // element offset of the row
    __device__ __forceinline__ RelposCursor(const RelposShape &p, int64_t h, int bi) {
        b = bi / (int)p.Tq;
        i = bi - b * (int)p.Tq;
        off = (((int64_t)b * p.H + h) * p.Tq + i) * p.Tk;
    }
    __device__ __forceinline__ void advance(int Tq, const RelposStep &g) {
        b += g.gq;
        i += g.gr;
        off += g.step;
        if (i >= Tq) {
            i -= Tq;
            ++b;
            off += g.wrap;
        }
    }
};

// Windows of the batch entries of rows [r0, r1) of a head (r0 < r1), into wtab;
// false if there are too many of them or they are not worth finding.  BLOCK:
// the threads of the block, 0 where the launch decides.
template <typename T, bool ADDS, int BLOCK>
__device__ __forceinline__ bool relpos_find_windows(int2 *wtab, const T *mask, const RelposShape &p,
                                                    int r0, int r1) {
    const int Tq = (int)p.Tq;
    const int b0 = r0 / Tq, nb = (r1 - 1) / Tq - b0 + 1;
    if (!mask || Tq < kRelposWindowTq || nb > kRelposWinMax) return false;
    for (int k = threadIdx.x >> 5; k < nb; k += (BLOCK ? BLOCK : (int)blockDim.x) / 32) {
        const int2 w = relpos_mask_window<T, ADDS>(mask + (int64_t)(b0 + k) * p.Tk, (int)p.Tk);
        if ((threadIdx.x & 31) == 0) wtab[k] = w;
    }
    return true;
}

// Chunk of V elements at element offset `at` of a tensor of `total` elements.
// AL: chunks never leave their row.
template <typename T, bool AL>
__device__ __forceinline__ uint4 relpos_load(const T *base, int64_t at, int64_t total) {
    constexpr int V = Traits<T>::kVec;
    if (AL || (at >= 0 && at + V <= total)) return ld_stream16(base + at);
    float f[V];
#pragma unroll
    for (int e = 0; e < V; ++e)
        f[e] = at + e >= 0 && at + e < total ? Traits<T>::load1(base + at + e) : 0.f;
    return Traits<T>::pack(f);
}

// Store of a chunk whose first key is j0; keys outside [0, Tk) belong to other
// rows: a partial chunk is stored by words, and by halves at its border.
template <typename T, bool AL>
__device__ __forceinline__ void relpos_store(T *row, int j0, int Tk, const uint4 &u) {
    constexpr int V = Traits<T>::kVec;
    if (AL || (j0 >= 0 && j0 + V <= Tk)) {
        st_stream16(row + j0, u);
        return;
    }
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (V == 4) {
            if (j0 + i >= 0 && j0 + i < Tk)
                __stcs(reinterpret_cast<uint32_t *>(row + j0 + i), w[i]);
        } else {
            const int j = j0 + 2 * i;  // (a chunk starts at a 16-byte address)
            if (j >= 0 && j + 1 < Tk)
                __stcs(reinterpret_cast<uint32_t *>(row + j), w[i]);
            else if (j >= 0 && j < Tk)
                __stcs(reinterpret_cast<unsigned short *>(row + j), (unsigned short)w[i]);
            else if (j == -1 && j + 1 < Tk)
                __stcs(reinterpret_cast<unsigned short *>(row + j + 1),
                       (unsigned short)(w[i] >> 16));
        }
    }
}

// The elements [0, n) of a chunk as a mask, for n = 0 ... V, in shared memory.
template <typename T>
__device__ __forceinline__ void relpos_keep_table(uint4 *keep) {
    constexpr int V = Traits<T>::kVec;
    if (threadIdx.x <= V) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int n = (int)threadIdx.x - i * (V / 4);  // elements of word i
            w[i] = n >= V / 4 ? 0xffffffffu : (V == 8 && n == 1 ? 0xffffu : 0u);
        }
        keep[threadIdx.x] = make_uint4(w[0], w[1], w[2], w[3]);
    }
}

// Bits of the chunk's visible keys: inside [lo, hi), and not masked with -inf
// in mrow if that is given.
template <typename T>
__device__ __forceinline__ uint32_t relpos_bits(const T *mrow, int j0, int lo, int hi) {
    constexpr int V = Traits<T>::kVec;
    const int a = min(max(lo - j0, 0), V), b = min(max(hi - j0, 0), V);
    uint32_t bits = ((1u << b) - 1u) & ~((1u << a) - 1u);
    if (mrow) {
#pragma unroll
        for (int e = 0; e < V; ++e)
            if ((bits >> e) & 1u)
                if (Traits<T>::load1_cached(mrow + j0 + e) == -INFINITY) bits &= ~(1u << e);
    }
    return bits;
}

// What a row group needs of one row.
struct RelposRow {
    int64_t off;  // element offset of the row
    int q;        // the query's key position
    int s;        // elements from a 16-byte address to the row's start
    int lo, hi;   // window of visible keys; empty for a row that is not there
    int b;        // batch entry whose mask is added element by element, or -1
};
template <bool AL, int V>
__device__ __forceinline__ RelposRow relpos_row(const RelposShape &p, const RelposCursor &cur,
                                                bool valid, bool masked, const int2 *wtab, int b0,
                                                int phase) {
    RelposRow w;
    w.off = cur.off;
    w.q = cur.i + (int)p.qoff;
    w.s = AL ? 0 : (int)((w.off + phase) & (V - 1));
    w.lo = 0;
    w.hi = valid ? (int)p.Tk : 0;
    w.b = -1;
    if (masked && valid) {
        const int2 win = wtab ? wtab[cur.b - b0] : make_int2(-1, 0);
        if (win.x < 0) {
            w.b = cur.b;
        } else {
            w.lo = win.x;
            w.hi = win.y;
        }
    }
    if (p.causal) w.hi = min(w.hi, w.q + 1);
    if (w.hi <= w.lo) {  // no chunk, not even one that begins before the row, meets it
        w.lo = 0;
        w.hi = -V;
    }
    return w;
}

// The bias by distance in shared memory, as seen by chunks.  A[x] is the bias
// of distance x - R - kLutPad, both ends repeated; copy k (of four) holds A
// shifted by k, so that the values from any distance on start at a 16-byte
// address of the copy of its phase.  All chunks of a row have the same phase,
// and far chunks are clamped by whole 16-byte steps into the repeated ends.
constexpr int kLutPad = 12;  // a chunk clamped at either end lies in it at any phase
__host__ __device__ constexpr int relpos_lut_stride(int R) {
    return (2 * R + 1 + 2 * kLutPad + 8 + 3) / 4 * 4;
}

// Resident blocks per SM asked of ptxas, and stages of the row pipeline (the
// current row and the next).
template <int TPR, int CPT>
constexpr int relpos_fw_min_blocks() {
    return TPR > 256 ? 1 : (CPT <= 2 ? 4 : 3);
}
constexpr int kRelposFwStages = 2;
template <int TPR, int CPT>
constexpr size_t relpos_fw_smem(int R) {
    return (size_t)4 * relpos_lut_stride(R) * 4 +
           (size_t)kRelposFwStages * CPT * relpos_block<TPR>() * 16;
}

// Mask elements of a chunk, -inf outside [lo, hi).
template <typename T, bool VEC>
__device__ __forceinline__ void relpos_mask(const T *mrow, int j0, int lo, int hi,
                                            float (&mv)[Traits<T>::kVec]) {
    constexpr int V = Traits<T>::kVec;
    if (j0 >= lo && j0 + V <= hi) {
        if (VEC) {
            Traits<T>::unpack(ld_cached16(mrow + j0), mv);
        } else {
#pragma unroll
            for (int e = 0; e < V; ++e) mv[e] = Traits<T>::load1_cached(mrow + j0 + e);
        }
    } else {
#pragma unroll
        for (int e = 0; e < V; ++e)
            mv[e] = j0 + e >= lo && j0 + e < hi ? Traits<T>::load1_cached(mrow + j0 + e)
                                                : -INFINITY;
    }
}

// Measured on a GB300: [32,16,512,512] bf16 with padding 87.4 us, 5.4 TB/s of the
// bytes it cannot do without (the plain softmax of these inputs: 91.6 us), bound
// by issue (71 % of the slots; 80 registers, three blocks per SM);
// [4,8,333,777] fp32 with a mask added element by element 21.0 us (2.8 TB/s).
// Before rows were staged ahead and packed two to a warp: 146 us.
// MASKED: there is a mask (without one its registers and branches are gone: the
// backward of [8,12,777,777] fp16, causal, 85 -> 76 us).
// At the 80 registers of three blocks, 17 of the 92 instantiations of a 16-bit
// type spill 4 to 68 bytes (those with a mask and four chunks, rows of odd
// lengths most); none of fp32 do.
template <typename T, int TPR, int CPT, bool AL, bool MASKED>
__global__ void __launch_bounds__(relpos_block<TPR>(), (relpos_fw_min_blocks<TPR, CPT>()))
relpos_fw_vec(T *out, const T *inp, const T *mask_or_null, const T *table, const int32_t *bucket,
              const RelposShape p, int mask_vec) {
    pdl_begin();
    const T *const mask = MASKED ? mask_or_null : nullptr;
    using Tr = Traits<T>;
    constexpr int V = Tr::kVec;
    constexpr int H2 = V / 2;
    constexpr int BLOCK = relpos_block<TPR>();
    constexpr int G = BLOCK / TPR;
    constexpr int S = kRelposFwStages;
    static_assert(S == 2, "the row in flight is carried in registers");
    extern __shared__ __align__(128) uint4 dsmem[];
    uint4 *stage = dsmem + threadIdx.x;  // [S][CPT][BLOCK], a thread's own slots
    const float4 *lut4 = reinterpret_cast<const float4 *>(dsmem + S * CPT * BLOCK);
    float *lut = reinterpret_cast<float *>(dsmem + S * CPT * BLOCK);
    __shared__ float red_max[BLOCK / 32], red_sum[BLOCK / 32];
    __shared__ int2 wtab[MASKED ? kRelposWinMax : 1];
    const int lane = threadIdx.x % TPR;
    const int grp = threadIdx.x / TPR;
    const int sub = TPR < 32 ? grp % (32 / (TPR < 32 ? TPR : 32)) : 0;  // group of the warp
    const int Tk = (int)p.Tk, stride = relpos_lut_stride(p.R);
    const int top = (2 * p.R + kLutPad + 4) / 4;  // last 16-byte step a chunk may start at
    const int64_t total = p.rows * p.Tk;
    const int Tq = (int)p.Tq;
    const RelposStep step(p, G);
    const int phase = (int)((reinterpret_cast<uintptr_t>(inp) / sizeof(T)) % V);
    const float2 sc = f2(p.scale);

    const int64_t beg = (int64_t)blockIdx.x * p.per;
    const int64_t end = min(beg + p.per, p.rows);
    for (int64_t t0 = beg; t0 < end;) {
        const int64_t h = t0 / p.rows_per_head;
        const int r0 = (int)(t0 - h * p.rows_per_head);
        const int r1 = (int)min(end - h * p.rows_per_head, p.rows_per_head);
        __syncthreads();  // the last segment's bias and windows are no longer read
        const bool windows = relpos_find_windows<T, true, BLOCK>(wtab, mask, p, r0, r1);
        const int b0 = r0 / Tq;
        if (windows) __syncthreads();
        // Copies of a row's visible chunks into a stage: each thread its own
        // slots.  A chunk that reaches past the tensor is put there by hand.
        int r_issue = r0 + grp;
        RelposCursor ci(p, h, r_issue);
        RelposRow next;  // the row issued last
        auto issue = [&](int s) {
            next = relpos_row<AL, V>(p, ci, r_issue < r1, mask != nullptr,
                                     windows ? wtab : nullptr, b0, phase);
            if (r_issue < r1) {
#pragma unroll
                for (int k = 0; k < CPT; ++k) {
                    const int j0 = (k * TPR + lane) * V - next.s;
                    if (j0 < next.hi && j0 + V > next.lo) {
                        const int64_t at = next.off + j0;
                        if (AL || (at >= 0 && at + V <= total))
                            cp_async16(&stage[(s * CPT + k) * BLOCK], inp + at);
                        else
                            stage[(s * CPT + k) * BLOCK] = relpos_load<T, AL>(inp, at, total);
                    }
                }
                r_issue += G;
                ci.advance(Tq, step);
            }
            cp_async_commit();
        };
        issue(0);
        // the bias, while the first rows are on their way
        for (int x = threadIdx.x; x < stride; x += BLOCK) {
            const float v =
                relpos_bias<T>(table, bucket, p, h, min(max(x - kLutPad, 0), 2 * p.R));
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (x >= k) lut[k * stride + x - k] = v;
        }
        __syncthreads();
        int turn = 0;  // stage of the current row
        // groups that share a warp take the same number of turns (shuffles)
        for (int rw = r0 + grp - sub; rw < r1; rw += G, turn ^= 1) {
            const RelposRow w = next;
            const bool valid = rw + sub < r1;
            issue(turn ^ 1);
            cp_async_wait<1>();  // this thread's copies of the row have landed
            const int lo = w.lo, hi = w.hi, j_lane = lane * V - w.s;
            // keys of the warp's part of chunk k: [k * TPR * V + wj, ... + WK)
            const int wj = (TPR > 32 ? (lane & ~31) * V : 0) - w.s;
            constexpr int WK = (TPR < 32 ? TPR : 32) * V;
            // distance of the lane's first key, in elements from A[0]
            const int x_lane = j_lane - w.q + p.R + kLutPad;
            const float4 *lut_row = lut4 + (x_lane & 3) * (stride / 4);
            float2 v[CPT][H2];
            float m = -INFINITY;
#pragma unroll
            for (int k = 0; k < CPT; ++k) {
                const int j0 = k * TPR * V + j_lane;
                if (!(k * TPR * V + wj < hi && k * TPR * V + wj + WK > lo)) continue;
                unpack2<T>(stage[(turn * CPT + k) * BLOCK], v[k]);
                const float4 *bias =
                    lut_row + min(max((x_lane >> 2) + k * (TPR * V / 4), 0), top);
#pragma unroll
                for (int h2 = 0; h2 < H2; h2 += 2) {
                    const float4 b4 = bias[h2 / 2];
                    v[k][h2] = fma2(v[k][h2], sc, make_float2(b4.x, b4.y));
                    v[k][h2 + 1] = fma2(v[k][h2 + 1], sc, make_float2(b4.z, b4.w));
                }
                if (w.b >= 0) {
                    const T *mrow = mask + (int64_t)w.b * Tk;
                    float mv[V];
                    if (AL && mask_vec)
                        relpos_mask<T, true>(mrow, j0, lo, hi, mv);
                    else
                        relpos_mask<T, false>(mrow, j0, lo, hi, mv);
                    // -inf decides whatever the score (NaN too)
#pragma unroll
                    for (int h2 = 0; h2 < H2; ++h2) {
                        v[k][h2].x = mv[2 * h2] == -INFINITY ? -INFINITY : v[k][h2].x + mv[2 * h2];
                        v[k][h2].y = mv[2 * h2 + 1] == -INFINITY ? -INFINITY
                                                                 : v[k][h2].y + mv[2 * h2 + 1];
                    }
                } else if (j0 < lo || j0 + V > hi) {
                    const int a = lo - j0, b = hi - j0;
#pragma unroll
                    for (int h2 = 0; h2 < H2; ++h2) {
                        if (2 * h2 < a || 2 * h2 >= b) v[k][h2].x = -INFINITY;
                        if (2 * h2 + 1 < a || 2 * h2 + 1 >= b) v[k][h2].y = -INFINITY;
                    }
                }
#pragma unroll
                for (int h2 = 0; h2 < H2; ++h2) m = fmax3(m, v[k][h2].x, v[k][h2].y);
            }
            m = relpos_reduce<TPR, BLOCK, OpMax>(m, red_max, grp);
            // e^(z - m) as one fused multiply-add.  The rounding of m * log2 e
            // multiplies the whole row by one number, which the quotient loses:
            // at most 2^(1/16) for |m| < 2^20, but from 2^31 on it can leave
            // the range of ex2.  Rows of larger maxima (only keys hidden by a
            // finite mask are left) and infinite or missing ones take the
            // difference first.
            float2 nmL = f2(-m * kLog2e);
            if (!(fabsf(m) < 0x1p20f)) {
                const float2 nm = f2(m == -INFINITY ? 0.f : -m);
#pragma unroll
                for (int k = 0; k < CPT; ++k)
#pragma unroll
                    for (int h2 = 0; h2 < H2; ++h2) v[k][h2] = add2(v[k][h2], nm);
                nmL = f2(0.f);
            }
            float2 sum2 = f2(0.f);
#pragma unroll
            for (int k = 0; k < CPT; ++k) {
                if (!(k * TPR * V + wj < hi && k * TPR * V + wj + WK > lo)) continue;
#pragma unroll
                for (int h2 = 0; h2 < H2; ++h2) {
                    float2 e = fma2(v[k][h2], f2(kLog2e), nmL);
                    e.x = fast_exp2(e.x);
                    e.y = fast_exp2(e.y);
                    v[k][h2] = e;
                    sum2 = add2(sum2, e);
                }
            }
            const float sum = relpos_reduce<TPR, BLOCK, OpSum>(sum2.x + sum2.y, red_sum, grp);
            const float inv = sum == 0.f ? 0.f : fast_rcp(sum);
            T *orow = out + w.off;
#pragma unroll
            for (int k = 0; k < CPT; ++k) {
                const int j0 = k * TPR * V + j_lane;
                uint4 o = make_uint4(0u, 0u, 0u, 0u);
                if (k * TPR * V + wj < hi && k * TPR * V + wj + WK > lo) {
                    float2 yv[H2];
#pragma unroll
                    for (int h2 = 0; h2 < H2; ++h2) yv[h2] = mul2(v[k][h2], f2(inv));
                    if (inv != inv) {  // NaN or +inf among the scores: only visible keys
                        const uint32_t bits = relpos_bits<T>(
                            w.b >= 0 ? mask + (int64_t)w.b * Tk : nullptr, j0, lo, hi);
#pragma unroll
                        for (int h2 = 0; h2 < H2; ++h2) {
                            if (!((bits >> (2 * h2)) & 1u)) yv[h2].x = 0.f;
                            if (!((bits >> (2 * h2 + 1)) & 1u)) yv[h2].y = 0.f;
                        }
                    }
                    o = pack2<T>(yv);
                }
                if (valid && j0 < Tk) relpos_store<T, AL>(orow, j0, Tk, o);
            }
        }
        cp_async_wait<0>();  // (only empty groups are left)
        t0 = h * p.rows_per_head + r1;
    }
}

// ----------------------------------------------------------------------------
// Register-resident backward.  Rows are staged one ahead, y and dout.  dz is
// added by distance into arrays of the block.  As the bias in the forward, an
// array exists in four copies, one for each phase of a row's chunks, so that a
// chunk is added with two 16-byte loads and stores; it covers the distances
// [first, first + stride) that are not clipped and can occur and a chunk more
// on either side, so that a chunk is either wholly inside or wholly clipped.
//
// A row of several warps has one array (its keys have distinct distances, and
// the barrier of the row's sum keeps rows apart).  A warp of whole rows has an
// array for every four of its row groups.  Groups that share one work on
// consecutive queries, whose phases usually differ: they then add to different
// copies at the same time.  Where two phases agree (rows of odd lengths, the
// last query of a batch entry beside the next one's first) the groups take
// turns.
// ----------------------------------------------------------------------------
struct RelposBand {
    int first;   // distance of entry 0
    int stride;  // entries of a copy, a multiple of 4
};
template <int V>
__host__ __device__ inline RelposBand relpos_band(const RelposShape &p) {
    const int64_t last = p.causal ? 0 : p.Tq - 1;  // the largest j - q
    const int rmin = (int)(-p.R + 1 > 1 - p.Tk ? -p.R + 1 : 1 - p.Tk);
    const int rmax = (int)(p.R - 1 < last ? p.R - 1 : last);
    RelposBand b;
    b.first = rmin - V;
    // entries first ... rmax + V, and what the copies' shift leaves over
    b.stride = (((rmax > rmin ? rmax - rmin : 0) + 1 + 2 * V + 3) / 4 + 1) * 4;
    return b;
}

// Arrays of a warp (rows within it), arrays and shared memory of a block of n
// threads.
template <int TPR>
constexpr int relpos_warp_arrays() { return TPR >= 8 ? 1 : 8 / TPR; }
template <int TPR>
__host__ __device__ constexpr int relpos_bw_arrays(int n) {
    return TPR <= 32 ? n / 32 * relpos_warp_arrays<TPR>() : n / TPR;
}
constexpr int kRelposBwStages = 2;  // the current row and the next
template <int TPR, int CPT>
__host__ __device__ constexpr size_t relpos_bw_smem(int n, int band_stride) {
    return (size_t)relpos_bw_arrays<TPR>(n) * band_stride * 16 +
           (size_t)kRelposBwStages * 2 * CPT * n * 16;
}

// Measured on a GB300 with the fold below: [32,16,512,512] bf16 with padding
// 134.3 us (5.0 TB/s), [8,12,777,777] fp16 causal 73.6 us (3.2 TB/s).  Bound by
// issue at four warps per scheduler (128 registers: y and dout of a row are
// held as floats; reading them twice from shared memory instead measured 140
// against then 138.6 us, one stage and three blocks per SM at 80 registers 155).
// The cut into one run of rows per block is uneven under causal and padding: of
// the second case's 301 blocks the heaviest has 1.68 times the mean of visible
// keys and 1.34 times that of bytes, the heaviest pair of blocks of an SM 1.21
// and 1.11 times.  13 of the 76 instantiations of a 16-bit type spill 4 to 36
// bytes.
// blockDim.x: relpos_block<TPR>() threads, or fewer (whole warps and row
// groups) where the arrays would not fit.
template <typename T, int TPR, int CPT, bool AL, bool MASKED>
__global__ void __launch_bounds__(relpos_block<TPR>(), 512 / relpos_block<TPR>())
relpos_bw_vec(T *dinp, float *part, const T *dout, const T *y, const T *mask_or_null,
              const RelposShape p) {
    pdl_begin();
    const T *const mask = MASKED ? mask_or_null : nullptr;
    using Tr = Traits<T>;
    constexpr int V = Tr::kVec;
    constexpr int H2 = V / 2;
    constexpr int BLOCK = relpos_block<TPR>();
    constexpr int S = kRelposBwStages;
    static_assert(S == 2, "the row in flight is carried in registers");
    constexpr int TW = TPR < 32 ? TPR : 32;  // threads of a group in one warp
    extern __shared__ __align__(128) uint4 dsmem[];
    const int n = blockDim.x;
    uint4 *stage = dsmem + threadIdx.x;  // [S][CPT][2][n], a thread's own slots
    float4 *acc4 = reinterpret_cast<float4 *>(dsmem + S * CPT * 2 * n);
    float *acc = reinterpret_cast<float *>(acc4);  // [arrays][4][band.stride]
    __shared__ float red[2][BLOCK / 32];
    __shared__ float ends[2][BLOCK / 32];
    __shared__ int2 wtab[MASKED ? kRelposWinMax : 1];
    __shared__ uint4 keep[V + 1];
    relpos_keep_table<T>(keep);  // (seen after the first segment's barrier)
    const int G = n / TPR;
    const int lane = threadIdx.x % TPR;
    const int grp = threadIdx.x / TPR;
    const int sub = grp % (32 / TW);  // group of the warp
    const int Tk = (int)p.Tk;
    const RelposBand band = relpos_band<V>(p);
    const int arrays = relpos_bw_arrays<TPR>(n);
    float4 *mine =
        acc4 + (TPR <= 32 ? (threadIdx.x >> 5) * relpos_warp_arrays<TPR>() + sub / 4 : grp) *
                   band.stride;
    const int64_t total = p.rows * p.Tk;
    const int Tq = (int)p.Tq;
    const RelposStep step(p, G);
    const int phase = (int)((reinterpret_cast<uintptr_t>(y) / sizeof(T)) % V);

    const int64_t beg = (int64_t)blockIdx.x * p.per;
    const int64_t end = min(beg + p.per, p.rows);
    for (int64_t t0 = beg; t0 < end;) {
        const int64_t h = t0 / p.rows_per_head;
        const int r0 = (int)(t0 - h * p.rows_per_head);
        const int r1 = (int)min(end - h * p.rows_per_head, p.rows_per_head);
        const bool windows = relpos_find_windows<T, false, 0>(wtab, mask, p, r0, r1);
        const int b0 = r0 / Tq;
        if (windows) __syncthreads();
        int r_issue = r0 + grp;
        RelposCursor ci(p, h, r_issue);
        RelposRow next;  // the row issued last, and bit k: the thread's chunk k has a visible
        uint32_t next_see, next_edge;  // key (see), and an invisible one by the window (edge)
        auto issue = [&](int s) {
            next = relpos_row<AL, V>(p, ci, r_issue < r1, mask != nullptr,
                                     windows ? wtab : nullptr, b0, phase);
            next_see = next_edge = 0u;
#pragma unroll
            for (int k = 0; k < CPT; ++k) {
                const int j0 = (k * TPR + lane) * V - next.s;
                if (j0 < next.hi && j0 + V > next.lo) {
                    next_see |= 1u << k;
                    if (j0 < next.lo || j0 + V > next.hi) next_edge |= 1u << k;
                    const int64_t at = next.off + j0;
                    uint4 *slot = &stage[(s * CPT + k) * 2 * n];
                    if (AL || (at >= 0 && at + V <= total)) {
                        cp_async16(slot, y + at);
                        cp_async16(slot + n, dout + at);
                    } else {
                        slot[0] = relpos_load<T, AL>(y, at, total);
                        slot[n] = relpos_load<T, AL>(dout, at, total);
                    }
                }
            }
            r_issue += G;
            ci.advance(Tq, step);
            cp_async_commit();
        };
        issue(0);
        for (int x = threadIdx.x; x < arrays * band.stride; x += n)
            acc4[x] = make_float4(0.f, 0.f, 0.f, 0.f);
        __syncthreads();
        float2 lo2 = f2(0.f), hi2 = f2(0.f);  // the clipped ends
        int turn = 0;  // also the stage of the current row
        // groups that share a warp take the same number of turns (shuffles)
        for (int rw = r0 + grp - sub; rw < r1; rw += G) {
            const RelposRow w = next;
            const uint32_t see = next_see, edge = next_edge;
            const bool valid = rw + sub < r1;
            issue(turn ^ 1);
            cp_async_wait<1>();  // this thread's copies of the row have landed
            const int lo = w.lo, hi = w.hi, j_lane = lane * V - w.s;
            const T *mrow = w.b >= 0 ? mask + (int64_t)w.b * Tk : nullptr;

            // y and dout of chunk k, 0 at invisible keys
            auto load = [&](int k, float2(&yv)[H2], float2(&gv)[H2]) {
                const uint4 *slot = &stage[(turn * CPT + k) * 2 * n];
                uint4 yr = slot[0], gr4 = slot[n];
                const int j0 = k * TPR * V + j_lane;
                if (mrow) {
                    const uint32_t bits = relpos_bits<T>(mrow, j0, lo, hi);
                    keep_elements<T>(yr, bits);
                    keep_elements<T>(gr4, bits);
                } else if ((edge >> k) & 1u) {
                    const uint4 b = keep[min(hi - j0, V)], a = keep[max(lo - j0, 0)];
                    yr.x &= b.x & ~a.x;
                    yr.y &= b.y & ~a.y;
                    yr.z &= b.z & ~a.z;
                    yr.w &= b.w & ~a.w;
                    gr4.x &= b.x & ~a.x;
                    gr4.y &= b.y & ~a.y;
                    gr4.z &= b.z & ~a.z;
                    gr4.w &= b.w & ~a.w;
                }
                unpack2<T>(yr, yv);
                unpack2<T>(gr4, gv);
            };
            float2 yv[CPT][H2], gv[CPT][H2];
            float2 s2 = f2(0.f);
#pragma unroll
            for (int k = 0; k < CPT; ++k) {
                if (!((see >> k) & 1u)) continue;
                load(k, yv[k], gv[k]);
#pragma unroll
                for (int h2 = 0; h2 < H2; ++h2) s2 = fma2(yv[k][h2], gv[k][h2], s2);
            }
            // the group's barrier also orders this row's additions after the
            // last row's; `red` alternates so that one barrier is enough
            const float s = relpos_reduce<TPR, 0, OpSum>(s2.x + s2.y, red[turn], grp);
            const int x_lane = j_lane - w.q - band.first;  // entry of the lane's first key
            float4 *acc_row = mine + (x_lane & 3) * (band.stride / 4);
            // groups before this one with the same array and copy go first
            int rank = 0;
            if constexpr (TPR < 32 && !AL) {
                const int copy = x_lane & 3;
#pragma unroll
                for (int d = 1; d < 4 && d < 32 / TPR; ++d) {
                    const int other = __shfl_up_sync(0xffffffffu, copy, d * TPR);
                    rank += sub % 4 >= d && other == copy;
                }
            }
            auto dz_of = [&](int k, const float2(&yk)[H2], const float2(&gk)[H2],
                             float2(&dz)[H2]) {
#pragma unroll
                for (int h2 = 0; h2 < H2; ++h2) dz[h2] = mul2(yk[h2], add2(gk[h2], f2(-s)));
                if (!(fabsf(s) < INFINITY)) {  // 0 * NaN: invisible keys stay 0
                    const uint32_t bits =
                        relpos_bits<T>(mrow, k * TPR * V + j_lane, lo, hi);
#pragma unroll
                    for (int h2 = 0; h2 < H2; ++h2) {
                        if (!((bits >> (2 * h2)) & 1u)) dz[h2].x = 0.f;
                        if (!((bits >> (2 * h2 + 1)) & 1u)) dz[h2].y = 0.f;
                    }
                }
            };
            auto add = [&](int k, const float2(&dz)[H2]) {
                const int d0 = k * TPR * V + j_lane - w.q;
                if (d0 <= -p.R - V + 1) {
#pragma unroll
                    for (int h2 = 0; h2 < H2; ++h2) lo2 = add2(lo2, dz[h2]);
                } else if (d0 >= p.R) {
#pragma unroll
                    for (int h2 = 0; h2 < H2; ++h2) hi2 = add2(hi2, dz[h2]);
                } else {
                    float4 *at = acc_row + (x_lane >> 2) + k * (TPR * V / 4);
                    float4 a[H2 / 2];
#pragma unroll
                    for (int h2 = 0; h2 < H2 / 2; ++h2) a[h2] = at[h2];
#pragma unroll
                    for (int h2 = 0; h2 < H2 / 2; ++h2) {
                        const float2 u = add2(make_float2(a[h2].x, a[h2].y), dz[2 * h2]);
                        const float2 t = add2(make_float2(a[h2].z, a[h2].w), dz[2 * h2 + 1]);
                        at[h2] = make_float4(u.x, u.y, t.x, t.y);
                    }
                }
            };
#pragma unroll
            for (int k = 0; k < CPT; ++k) {
                const int j0 = k * TPR * V + j_lane;
                uint4 o = make_uint4(0u, 0u, 0u, 0u);
                if ((see >> k) & 1u) {
                    float2 dz[H2], dx[H2];
                    dz_of(k, yv[k], gv[k], dz);
#pragma unroll
                    for (int h2 = 0; h2 < H2; ++h2) dx[h2] = mul2(dz[h2], f2(p.scale));
                    o = pack2<T>(dx);
                    if (rank == 0) add(k, dz);
                }
                if (valid && j0 < Tk) relpos_store<T, AL>(dinp + w.off, j0, Tk, o);
            }
            if constexpr (TPR <= 32) __syncwarp();
            if constexpr (TPR < 32 && !AL) {
#pragma unroll 1
                for (int go = 1; __any_sync(0xffffffffu, rank >= go); ++go) {
#pragma unroll
                    for (int k = 0; k < CPT; ++k) {
                        if (rank == go && ((see >> k) & 1u)) {
                            float2 ya[H2], ga[H2], dz[H2];
                            load(k, ya, ga);
                            dz_of(k, ya, ga, dz);
                            add(k, dz);
                        }
                    }
                    __syncwarp();
                }
            }
            turn ^= 1;
        }
        cp_async_wait<0>();  // (only empty groups are left)
        // the block's sum of each distance: entries of all arrays and copies
        // in order, and at both ends the lanes' registers and the entries of
        // clipped distances
        __syncwarp();
        float lo_sum = lo2.x + lo2.y, hi_sum = hi2.x + hi2.y;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            lo_sum += __shfl_xor_sync(0xffffffffu, lo_sum, o);
            hi_sum += __shfl_xor_sync(0xffffffffu, hi_sum, o);
        }
        if ((threadIdx.x & 31) == 0) {
            ends[0][threadIdx.x >> 5] = lo_sum;
            ends[1][threadIdx.x >> 5] = hi_sum;
        }
        __syncthreads();
        const int W2 = 2 * p.R + 1;
        float *slot = part + ((int64_t)blockIdx.x + h) * W2;
        // entry `x` of the distances from band.first on
        auto entry = [&](int x) {
            float t = 0.f;
            for (int g = 0; g < arrays; ++g)
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    if (x >= c && x - c < band.stride)
                        t += acc[(g * 4 + c) * band.stride + x - c];
            return t;
        };
        for (int d = threadIdx.x; d < W2; d += n) {
            float v = 0.f;
            const int x = d - p.R - band.first;
            if (d == 0 || d == 2 * p.R) {
                for (int g = 0; g < n / 32; ++g) v += ends[d ? 1 : 0][g];
                for (int e = 0; e < V; ++e) {  // distances -R - e, R + e
                    const int xe = d ? x + e : x - e;
                    if (xe >= 0 && xe < band.stride + 3) v += entry(xe);
                }
            } else if (x >= 0 && x < band.stride + 3) {
                v = entry(x);
            }
            slot[d] = v;
        }
        __syncthreads();
        t0 = h * p.rows_per_head + r1;
    }
}

// dtable[k, h] for one head h = blockIdx.x and the buckets of blockIdx.y: the
// segment sums of each distance (four threads per distance, every fourth
// segment each, so that a long chain of loads does not set the time), then
// each bucket's distances, one warp per bucket.  All in a fixed order.  Four
// threads share a distance, because the loads of one wait for each other: the
// backward of [32,16,512,512] bf16 took 138.8 us with one, 134.3 with four.
constexpr int kRelposFoldBuckets = 32;
constexpr int kRelposFoldThreads = 1024;
constexpr size_t relpos_fold_smem(int R) { return (size_t)(2 * R + 1) * 8; }
static __global__ void __launch_bounds__(kRelposFoldThreads)
relpos_fold(float *dtable, const float *part, const int32_t *bucket, const RelposShape p) {
    pdl_begin();
    extern __shared__ float dist[];  // [2R + 1], then the bucket ids
    __shared__ float sums[4][256];
    const int W = 2 * p.R + 1;
    int32_t *ids = reinterpret_cast<int32_t *>(dist + W);
    const int64_t h = blockIdx.x;
    const bool any = p.rows_per_head > 0;
    const int64_t first = any ? h * p.rows_per_head / p.per : 0;
    const int64_t last = any ? ((h + 1) * p.rows_per_head - 1) / p.per : -1;
    const int tx = threadIdx.x & 255, ty = threadIdx.x >> 8;
    for (int d = threadIdx.x; d < W; d += kRelposFoldThreads) ids[d] = __ldg(bucket + d);
    for (int d0 = 0; d0 < W; d0 += 256) {
        const int d = d0 + tx;
        float v = 0.f;
        if (d < W) {
#pragma unroll 10
            for (int64_t k = first + ty; k <= last; k += 4)
                v += __ldcg(part + (k + h) * W + d);
        }
        sums[ty][tx] = v;
        __syncthreads();
        if (ty == 0 && d < W) dist[d] = (v + sums[1][tx]) + (sums[2][tx] + sums[3][tx]);
        __syncthreads();
    }
    const int lane = threadIdx.x & 31;
    const int64_t k = (int64_t)blockIdx.y * kRelposFoldBuckets + (threadIdx.x >> 5);
    if (k >= p.num_buckets) return;
    float v = 0.f;
    for (int d = lane; d < W; d += 32)
        if (ids[d] == k) v += dist[d];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if (lane == 0) dtable[k * p.H + h] = v;
}

}  // namespace lsr
