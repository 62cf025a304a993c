// diff_softmax.cuh -- the difference of two attention softmax maps with a
// learned weight, forward and backward (sm_103a).
//
// Query i (the Tq queries are the last Tq of the Tk key positions) of head h has
// two rows of scores, x1 and x2, over the same visible keys j:
//     z_aj  = scale * x_aj + mask[b, j],   p_a = softmax over the visible j of z_a
//     out_j = p_1j - lam_h p_2j
// Backward, with D_a = sum over visible j of p_aj g_j:
//     dx_1j = scale p_1j (g_j - D_1),   dx_2j = -scale lam_h p_2j (g_j - D_2)
//     dlam_h = -sum over b, i of D_2
// The forward saves each map's largest z and the inverse of its sum, 16 bytes
// per row, so that the backward makes the weights again from the scores
// instead of reading two stored maps: three tensors read and two written.
//
// Rows are in registers: a row is owned by TPR threads with CPT 16-byte chunks
// of either map each; a block's groups take the rows of a contiguous run in
// turn, and the next row is copied into shared memory (cp.async) while the
// current one is reduced.  The two maps, the output and the gradients may be
// slices with strides between batch entries and heads, so that at lengths that
// are no whole number of vectors their rows start at different offsets within
// 16 bytes.  Chunks then lie on 16-byte addresses of the written row, and a
// row that is read is staged by its own 16-byte addresses and shifted on the
// way out of shared memory (two neighbouring chunks make one).
#pragma once

#include "launch.h"
#include "ls_device.cuh"
#include "relpos.cuh"  // mask windows, group reductions, guarded chunks

namespace lsr {

// |m| up to which the largest z's rounding is left out of account: the forward's
// e^(z - m) is then one fused multiply-add before ex2, the backward's z - m one.
// The roundings of scale * log2 e and m * log2 e put up to 2 * 64 * 1.45 *
// 2^-24 = 1e-5 on a row's sum; the weights lose that in the quotient, and the
// saved inverse is corrected for it (DiffExp::inverse).  Beyond it z is rounded
// before m, the largest of the rounded ones, is taken off: a product that stays
// unrounded differs from m by up to 2^-24 |m|, which from |m| = 2^30 on leaves
// the exponent's range, and whichever kernel made the statistics, and whether it
// added the mask or knew its window, the backward meets the same differences.
constexpr float kDiffNear = 64.f;

template <int TPR>
constexpr int diff_block() { return TPR < 256 ? 256 : TPR; }

// Position of a row, for kernels that take rows in any order.
struct DiffCursor {
    int b, h, i;
    __device__ __forceinline__ DiffCursor(const DiffShape &p, int64_t row) {
        const int64_t bh = row / p.Tq;
        i = (int)(row - bh * p.Tq);
        b = (int)(bh / p.H);
        h = (int)(bh - (int64_t)b * p.H);
    }
};

// The rows of a block: from beg on, G at a time, `step` further each turn.  A run
// of its own (p.per rows), or, where rows differ in length (causal; the launcher's
// rule), turns that lie a whole grid apart, so that no block gets the long rows of
// a head alone ([8,6,777,777] fp16 backward: 96 us in runs, 83 dealt out; with
// turns of one run taken from a head's start and end alternately 89).
struct DiffBlock {
    int64_t beg, end;
    int step;
    __device__ __forceinline__ DiffBlock(const DiffShape &p, int G) {
        beg = blockIdx.x * (p.per ? p.per : (int64_t)G);
        end = p.per ? min(beg + p.per, p.rows) : p.rows;
        step = p.per ? G : G * (int)gridDim.x;
    }
};

// Position of a row group, advanced by a block's step without division.  (The
// launcher keeps a head's elements below 2^31.)
struct DiffWalk {
    int b, h, i;
    int gb, gh, gi;  // step = (gb * H + gh) * Tq + gi
    int64_t row;
    __device__ __forceinline__ DiffWalk(const DiffShape &p, int64_t first, int step) {
        const DiffCursor c(p, first);
        b = c.b;
        h = c.h;
        i = c.i;
        row = first;
        gh = step / (int)p.Tq;
        gi = step - gh * (int)p.Tq;
        gb = gh / (int)p.H;
        gh -= gb * (int)p.H;
    }
    __device__ __forceinline__ void advance(const DiffShape &p, int step) {
        row += step;
        i += gi;
        h += gh;
        b += gb;
        if (i >= (int)p.Tq) {
            i -= (int)p.Tq;
            ++h;
        }
        if (h >= (int)p.H) {
            h -= (int)p.H;
            ++b;
        }
    }
};

// Sum (or maximum) of two numbers over a row group, as relpos_reduce; `red`
// holds 2 * BLOCK / 32 floats.
template <int TPR, int BLOCK, typename Op>
__device__ __forceinline__ void diff_reduce2(float &a, float &b, float *red, int grp) {
    constexpr int W = TPR < 32 ? TPR : 32;
#pragma unroll
    for (int o = W / 2; o > 0; o >>= 1) {
        a = Op::apply(a, __shfl_xor_sync(0xffffffffu, a, o));
        b = Op::apply(b, __shfl_xor_sync(0xffffffffu, b, o));
    }
    if constexpr (TPR > 32) {
        constexpr int NW = TPR / 32, BW = BLOCK / 32;
        if ((threadIdx.x & 31) == 0) {
            red[threadIdx.x >> 5] = a;
            red[BW + (threadIdx.x >> 5)] = b;
        }
        if constexpr (BLOCK == TPR)
            __syncthreads();
        else
            asm volatile("bar.sync %0, %1;" ::"r"(1 + grp), "r"(TPR) : "memory");
        a = red[grp * NW];
        b = red[BW + grp * NW];
#pragma unroll
        for (int w = 1; w < NW; ++w) {
            a = Op::apply(a, red[grp * NW + w]);
            b = Op::apply(b, red[BW + grp * NW + w]);
        }
    }
}
template <int TPR, int BLOCK>
__device__ __forceinline__ void diff_group_sync(int grp) {
    if constexpr (TPR <= 32)
        __syncwarp();
    else if constexpr (BLOCK == TPR)
        __syncthreads();
    else
        asm volatile("bar.sync %0, %1;" ::"r"(1 + grp), "r"(TPR) : "memory");
}

// What a row group needs of one row.
struct DiffRow {
    int b, h, i;
    int s;        // elements from a 16-byte address to the written row's start
    int lo, hi;   // window of visible keys; empty for a row that is not there
    bool general; // the mask is added element by element
    // element offset of the row in a tensor
    template <typename P>
    __device__ __forceinline__ int64_t at(const DiffRows<P> &x, const DiffShape &p) const {
        return (int64_t)b * x.batch + (int64_t)h * x.head + i * (int)p.Tk;
    }
    __device__ __forceinline__ int64_t dense(const DiffShape &p) const {
        return ((int64_t)(b * p.H + h) * p.Tq + i) * p.Tk;
    }
    // its place among the rows of its head (the fold reads a head's in one piece)
    __device__ __forceinline__ int64_t by_head(const DiffShape &p) const {
        return ((int64_t)h * p.B + b) * p.Tq + i;
    }
};

// Stages the chunks of one read row that hold a visible key: chunk c is the
// c-th 16-byte vector from the one that holds the written row's chunk 0 on.
// Returns by how many elements a written chunk starts within it.
template <typename T, int TPR, int CPT, bool AL>
__device__ __forceinline__ int diff_stage(uint4 *slots, const T *base, int64_t extent, int64_t off,
                                          int s, int lo, int hi, int lane) {
    constexpr int V = Traits<T>::kVec;
    if constexpr (AL) {
        const T *at = base + off + lane * V;
        const uint32_t to = smem_addr(slots + lane);
#pragma unroll
        for (int k = 0; k < CPT; ++k) {
            const int j0 = (k * TPR + lane) * V;
            if (j0 < hi && j0 + V > lo)
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                                 to + k * TPR * 16),
                             "l"(at + k * TPR * V)
                             : "memory");
        }
        return 0;
    } else {
        const int phase = (int)(reinterpret_cast<uintptr_t>(base) / sizeof(T) % V);
        const int64_t e0 = phase + off - s;  // from a 16-byte address at or before the base
        const int d = (int)(e0 & (V - 1));
        const int64_t first = e0 - d - phase;  // element offset of staged chunk 0
        auto put = [&](int c) {
            const int j0 = c * V - s - d;
            if (!(j0 < hi && j0 + V > lo)) return;
            const int64_t at = first + (int64_t)c * V;
            if (at >= 0 && at + V <= extent)
                cp_async16(&slots[c], base + at);
            else
                slots[c] = relpos_load<T, false>(base, at, extent);
        };
#pragma unroll
        for (int k = 0; k < CPT; ++k) put(k * TPR + lane);
        if (lane == 0) put(CPT * TPR);
        return d;
    }
}

// Elements [d, d + V) of two neighbouring chunks.
template <typename T, bool AL>
__device__ __forceinline__ uint4 diff_chunk(const uint4 *slot, int d) {
    if constexpr (AL) {
        return slot[0];
    } else {
        const uint4 a = slot[0], b = slot[1];
        constexpr int kPer = 4 / sizeof(T);  // elements of a word
        const int w = d / kPer;
        uint32_t x0 = a.x, x1 = a.y, x2 = a.z, x3 = a.w, x4 = b.x, x5 = b.y, x6 = b.z, x7 = b.w;
        if (w & 2) {
            x0 = x2; x1 = x3; x2 = x4; x3 = x5; x4 = x6; x5 = x7;
        }
        if (w & 1) {
            x0 = x1; x1 = x2; x2 = x3; x3 = x4; x4 = x5;
        }
        if constexpr (kPer == 2) {
            const uint32_t half = (d & 1) * 16;
            x0 = __funnelshift_r(x0, x1, half);
            x1 = __funnelshift_r(x1, x2, half);
            x2 = __funnelshift_r(x2, x3, half);
            x3 = __funnelshift_r(x3, x4, half);
        }
        return make_uint4(x0, x1, x2, x3);
    }
}

// Windows of the batch entries of rows [beg, end), as relpos_find_windows.
template <typename T, bool ADDS, int BLOCK>
__device__ __forceinline__ bool diff_find_windows(int2 *wtab, const T *mask, const DiffShape &p,
                                                  int64_t beg, int64_t end) {
    const int64_t per_batch = p.H * p.Tq;
    const int64_t b0 = beg / per_batch;
    const int64_t nb = (end - 1) / per_batch - b0 + 1;
    if (!mask || p.Tq < kRelposWindowTq || nb > kRelposWinMax) return false;
    for (int k = threadIdx.x >> 5; k < nb; k += BLOCK / 32) {
        const int2 w = relpos_mask_window<T, ADDS>(mask + (b0 + k) * p.Tk, (int)p.Tk);
        if ((threadIdx.x & 31) == 0) wtab[k] = w;
    }
    return true;
}

template <int V, bool AL, bool MASKED>
__device__ __forceinline__ DiffRow diff_row(const DiffShape &p, const DiffWalk &cur,
                                            bool valid, const int2 *wtab, int b0, int phase) {
    DiffRow w;
    w.b = cur.b;
    w.h = cur.h;
    w.i = cur.i;
    w.s = AL ? 0 : (int)((w.dense(p) + phase) & (V - 1));
    w.lo = 0;
    w.hi = valid ? (int)p.Tk : 0;
    w.general = false;
    if (MASKED && valid) {
        const int2 win = wtab ? wtab[cur.b - b0] : make_int2(-1, 0);
        if (win.x < 0) {
            w.general = true;
        } else {
            w.lo = win.x;
            w.hi = win.y;
        }
    }
    if (p.causal) w.hi = min(w.hi, cur.i + (int)p.qoff + 1);
    if (w.hi <= w.lo) {  // no chunk, not even one that begins before the row, meets it
        w.lo = 0;
        w.hi = -2 * V;
    }
    return w;
}

constexpr int kDiffStages = 2;  // the current row and the next
template <int TPR, int CPT, bool AL>
__host__ __device__ constexpr int diff_slots() { return CPT * TPR + (AL ? 0 : 1); }
template <int TPR, int CPT, bool AL>
constexpr size_t diff_smem(int tensors) {
    return (size_t)kDiffStages * tensors * (diff_block<TPR>() / TPR) * diff_slots<TPR, CPT, AL>() *
           16;
}
// Resident blocks per SM asked of ptxas (of the backward's two chunks, 128
// registers: at 80 they spill 24 to 210 bytes, 135 against 120 us on
// [32,8,512,512] bf16).
template <int TPR, int CPT>
constexpr int diff_fw_min_blocks() {
    return TPR > 256 ? 1 : (CPT <= 2 ? 3 : 2);
}
template <int TPR, int CPT>
constexpr int diff_bw_min_blocks() {
    return TPR > 256 ? 1 : (CPT <= 1 ? 3 : 2);
}

// Values of one chunk of a map: z where a mask is added, else the scores; -inf
// at invisible keys.
template <typename T, bool AL>
__device__ __forceinline__ void diff_values(float2 (&v)[Traits<T>::kVec / 2], const uint4 &raw,
                                            const T *mrow, bool mask_vec, int j0, int lo, int hi,
                                            float scale) {
    constexpr int V = Traits<T>::kVec, H2 = V / 2;
    unpack2<T>(raw, v);
    if (mrow) {
        float mv[V];
        if (AL && mask_vec)
            relpos_mask<T, true>(mrow, j0, lo, hi, mv);
        else
            relpos_mask<T, false>(mrow, j0, lo, hi, mv);
        // -inf decides whatever the score (NaN too)
#pragma unroll
        for (int h2 = 0; h2 < H2; ++h2) {
            const float2 z =
                fma2(v[h2], f2(scale), make_float2(mv[2 * h2], mv[2 * h2 + 1]));
            v[h2].x = mv[2 * h2] == -INFINITY ? -INFINITY : z.x;
            v[h2].y = mv[2 * h2 + 1] == -INFINITY ? -INFINITY : z.y;
        }
    } else if (j0 < lo || j0 + V > hi) {
        const int a = lo - j0, b = hi - j0;
#pragma unroll
        for (int h2 = 0; h2 < H2; ++h2) {
            if (2 * h2 < a || 2 * h2 >= b) v[h2].x = -INFINITY;
            if (2 * h2 + 1 < a || 2 * h2 + 1 >= b) v[h2].y = -INFINITY;
        }
    }
}

// e^(mul * v - m) as a multiplier and an addend of v before ex2, given m = mul *
// the largest v; values far from 0 are rounded and shifted first.
struct DiffExp {
    float c, n;
    // 1 / sum without what the roundings of c and n put on the exponent at v = top,
    // where the row's weight lies (2^off is 1 + off ln 2)
    __device__ __forceinline__ float inverse(float inv, float top, float m, float mul) const {
        if (!(fabsf(m) < kDiffNear)) return inv;
        const float off = fmaf(top, fmaf(-mul, kLog2e, c), fmaf(m, kLog2e, n));
        return fmaf(inv, off * 0.6931471805599453f, inv);
    }
};
// scale * x rounded.  (Scalar products: the compiler does fuse a pair's product
// with the sum that follows it.)
__device__ __forceinline__ float2 diff_rounded(float2 v, float mul) {
    return make_float2(__fmul_rn(v.x, mul), __fmul_rn(v.y, mul));
}
template <int CPT, int H2>
__device__ __forceinline__ DiffExp diff_exponent(float2 (&v)[CPT][H2], float m, float mul) {
    if (fabsf(m) < kDiffNear) return DiffExp{mul * kLog2e, -m * kLog2e};
    const float2 nm = f2(m == -INFINITY ? 0.f : -m);
#pragma unroll
    for (int k = 0; k < CPT; ++k)
#pragma unroll
        for (int h2 = 0; h2 < H2; ++h2) v[k][h2] = add2(diff_rounded(v[k][h2], mul), nm);
    return DiffExp{kLog2e, 0.f};
}

template <typename T, int TPR, int CPT, bool AL, bool MASKED>
__global__ void __launch_bounds__(diff_block<TPR>(), (diff_fw_min_blocks<TPR, CPT>()))
diff_fw_vec(T *out, float4 *stats, const DiffRows<const T> x1, const DiffRows<const T> x2,
            const float *lam, const T *mask_or_null, const DiffShape p, int mask_vec) {
    pdl_begin();
    const T *const mask = MASKED ? mask_or_null : nullptr;
    using Tr = Traits<T>;
    constexpr int V = Tr::kVec, H2 = V / 2;
    constexpr int BLOCK = diff_block<TPR>(), G = BLOCK / TPR;
    constexpr int SLOTS = diff_slots<TPR, CPT, AL>();
    extern __shared__ __align__(128) uint4 dsmem[];  // [stage][map][group][SLOTS]
    __shared__ float red_max[2 * BLOCK / 32], red_sum[2 * BLOCK / 32];
    __shared__ int2 wtab[MASKED ? kRelposWinMax : 1];
    const int lane = threadIdx.x % TPR;
    const int grp = threadIdx.x / TPR;
    const int sub = TPR < 32 ? grp % (32 / (TPR < 32 ? TPR : 32)) : 0;  // group of the warp
    const int Tk = (int)p.Tk;
    const int phase = (int)(reinterpret_cast<uintptr_t>(out) / sizeof(T) % V);
    const DiffBlock blk(p, G);
    const int64_t beg = blk.beg, end = blk.end;
    const bool windows = diff_find_windows<T, true, BLOCK>(wtab, mask, p, beg, end);
    const int b0 = (int)(beg / (p.H * p.Tq));
    if (windows) __syncthreads();

    DiffWalk walk(p, beg + grp, blk.step);
    DiffRow next;  // the row issued last, its maps' shifts and its head's weight
    int next_d1 = 0, next_d2 = 0;
    float next_lam = 0.f;
    auto slots = [&](int s, int map) { return dsmem + ((s * 2 + map) * G + grp) * SLOTS; };
    auto issue = [&](int s) {
        if (!AL && TPR <= 32) __syncwarp();  // (wider groups: the last row's reductions)
        next = diff_row<V, AL, MASKED>(p, walk, walk.row < end, windows ? wtab : nullptr, b0,
                                       phase);
        if (walk.row < end) {
            next_d1 = diff_stage<T, TPR, CPT, AL>(slots(s, 0), x1.p, x1.extent, next.at(x1, p),
                                                  next.s, next.lo, next.hi, lane);
            next_d2 = diff_stage<T, TPR, CPT, AL>(slots(s, 1), x2.p, x2.extent, next.at(x2, p),
                                                  next.s, next.lo, next.hi, lane);
            next_lam = __ldg(lam + next.h * p.lam_step);
        }
        walk.advance(p, blk.step);
        cp_async_commit();
    };
    issue(0);
    int turn = 0;  // stage of the current row
    // groups that share a warp take the same number of turns (shuffles)
    for (int64_t rw = beg + grp - sub; rw < end; rw += blk.step, turn ^= 1) {
        const DiffRow w = next;
        const int d1 = next_d1, d2 = next_d2;
        const float lam_h = next_lam;
        const bool valid = rw + sub < end;
        issue(turn ^ 1);
        cp_async_wait<1>();  // this thread's copies of the row have landed
        if (!AL) diff_group_sync<TPR, BLOCK>(grp);
        const int lo = w.lo, hi = w.hi, j_lane = lane * V - w.s;
        // keys of the warp's part of chunk k: [k * TPR * V + wj, ... + WK)
        const int wj = (TPR > 32 ? (lane & ~31) * V : 0) - w.s;
        constexpr int WK = (TPR < 32 ? TPR : 32) * V;
        const T *mrow = MASKED && w.general ? mask + (int64_t)w.b * Tk : nullptr;
        const float mul = MASKED && w.general ? 1.f : p.scale;
        const uint4 *s1 = slots(turn, 0) + lane, *s2 = slots(turn, 1) + lane;
        float2 v1[CPT][H2], v2[CPT][H2];
        float m1 = -INFINITY, m2 = -INFINITY;
#pragma unroll
        for (int k = 0; k < CPT; ++k) {
            const int j0 = k * TPR * V + j_lane;
            if (!(k * TPR * V + wj < hi && k * TPR * V + wj + WK > lo)) continue;
            diff_values<T, AL>(v1[k], diff_chunk<T, AL>(s1 + k * TPR, d1), mrow, mask_vec != 0, j0,
                               lo, hi, p.scale);
            diff_values<T, AL>(v2[k], diff_chunk<T, AL>(s2 + k * TPR, d2), mrow, mask_vec != 0, j0,
                               lo, hi, p.scale);
#pragma unroll
            for (int h2 = 0; h2 < H2; ++h2) {
                m1 = fmax3(m1, v1[k][h2].x, v1[k][h2].y);
                m2 = fmax3(m2, v2[k][h2].x, v2[k][h2].y);
            }
        }
        diff_reduce2<TPR, BLOCK, OpMax>(m1, m2, red_max, grp);
        const float top1 = m1, top2 = m2;
        m1 *= mul;
        m2 *= mul;
        const DiffExp x1e = diff_exponent(v1, m1, mul), x2e = diff_exponent(v2, m2, mul);
        float2 t1 = f2(0.f), t2 = f2(0.f);
#pragma unroll
        for (int k = 0; k < CPT; ++k) {
            if (!(k * TPR * V + wj < hi && k * TPR * V + wj + WK > lo)) continue;
#pragma unroll
            for (int h2 = 0; h2 < H2; ++h2) {
                float2 a = fma2(v1[k][h2], f2(x1e.c), f2(x1e.n));
                float2 b = fma2(v2[k][h2], f2(x2e.c), f2(x2e.n));
                a.x = fast_exp2(a.x);
                a.y = fast_exp2(a.y);
                b.x = fast_exp2(b.x);
                b.y = fast_exp2(b.y);
                v1[k][h2] = a;
                v2[k][h2] = b;
                t1 = add2(t1, a);
                t2 = add2(t2, b);
            }
        }
        float sum1 = t1.x + t1.y, sum2 = t2.x + t2.y;
        diff_reduce2<TPR, BLOCK, OpSum>(sum1, sum2, red_sum, grp);
        const float i1 = sum1 == 0.f ? 0.f : fast_rcp(sum1);
        const float i2 = sum2 == 0.f ? 0.f : fast_rcp(sum2);
        const float li2 = -lam_h * i2;
        if (stats && valid && lane == 0)
            stats[rw + sub] = make_float4(m1 == -INFINITY ? 0.f : m1, x1e.inverse(i1, top1, m1, mul),
                                          m2 == -INFINITY ? 0.f : m2, x2e.inverse(i2, top2, m2, mul));
        T *orow = out + w.dense(p) + (AL ? lane * V : 0);
#pragma unroll
        for (int k = 0; k < CPT; ++k) {
            const int j0 = k * TPR * V + j_lane;
            uint4 o = make_uint4(0u, 0u, 0u, 0u);
            if (k * TPR * V + wj < hi && k * TPR * V + wj + WK > lo) {
                float2 y[H2];
#pragma unroll
                for (int h2 = 0; h2 < H2; ++h2)
                    y[h2] = fma2(v2[k][h2], f2(li2), mul2(v1[k][h2], f2(i1)));
                if (!(fabsf(i1 + li2) < INFINITY)) {  // NaN or infinite: only visible keys
                    const uint32_t bits = relpos_bits<T>(mrow, j0, lo, hi);
#pragma unroll
                    for (int h2 = 0; h2 < H2; ++h2) {
                        if (!((bits >> (2 * h2)) & 1u)) y[h2].x = 0.f;
                        if (!((bits >> (2 * h2 + 1)) & 1u)) y[h2].y = 0.f;
                    }
                }
                o = pack2<T>(y);
            }
            if (valid && j0 < Tk)
                relpos_store<T, AL>(orow, AL ? k * TPR * V : j0, Tk, o);
        }
    }
    cp_async_wait<0>();  // (only empty groups are left)
}

// ----------------------------------------------------------------------------
// Backward.  With the saved statistics the weights need no reduction, so a row
// is one pass for the two sums and one that writes.
// ----------------------------------------------------------------------------
template <typename T, int TPR, int CPT, bool AL, bool MASKED>
__global__ void __launch_bounds__(diff_block<TPR>(), (diff_bw_min_blocks<TPR, CPT>()))
diff_bw_vec(const DiffRows<T> dx1, const DiffRows<T> dx2, float *row_dot, const T *dout,
            const DiffRows<const T> x1, const DiffRows<const T> x2, const float *lam,
            const float4 *stats, const T *mask_or_null, const DiffShape p, int mask_vec) {
    pdl_begin();
    const T *const mask = MASKED ? mask_or_null : nullptr;
    using Tr = Traits<T>;
    constexpr int V = Tr::kVec, H2 = V / 2;
    constexpr int BLOCK = diff_block<TPR>(), G = BLOCK / TPR;
    constexpr int SLOTS = diff_slots<TPR, CPT, AL>();
    extern __shared__ __align__(128) uint4 dsmem[];  // [stage][x1, x2, dout][group][SLOTS]
    __shared__ float red[2][2 * BLOCK / 32];
    __shared__ int2 wtab[MASKED ? kRelposWinMax : 1];
    const int lane = threadIdx.x % TPR;
    const int grp = threadIdx.x / TPR;
    const int sub = TPR < 32 ? grp % (32 / (TPR < 32 ? TPR : 32)) : 0;  // group of the warp
    const int Tk = (int)p.Tk;
    const int phase = (int)(reinterpret_cast<uintptr_t>(dout) / sizeof(T) % V);
    const DiffBlock blk(p, G);
    const int64_t beg = blk.beg, end = blk.end;
    const bool windows = diff_find_windows<T, true, BLOCK>(wtab, mask, p, beg, end);
    const int b0 = (int)(beg / (p.H * p.Tq));
    if (windows) __syncthreads();

    DiffWalk walk(p, beg + grp, blk.step);
    DiffRow next;
    int next_d1 = 0, next_d2 = 0;
    float4 next_st = make_float4(0.f, 0.f, 0.f, 0.f);
    float next_lam = 0.f;
    auto slots = [&](int s, int t) { return dsmem + ((s * 3 + t) * G + grp) * SLOTS; };
    auto issue = [&](int s) {
        if (!AL && TPR <= 32) __syncwarp();  // (wider groups: the last row's reduction)
        next = diff_row<V, AL, MASKED>(p, walk, walk.row < end, windows ? wtab : nullptr, b0,
                                       phase);
        if (walk.row < end) {
            next_d1 = diff_stage<T, TPR, CPT, AL>(slots(s, 0), x1.p, x1.extent, next.at(x1, p),
                                                  next.s, next.lo, next.hi, lane);
            next_d2 = diff_stage<T, TPR, CPT, AL>(slots(s, 1), x2.p, x2.extent, next.at(x2, p),
                                                  next.s, next.lo, next.hi, lane);
            diff_stage<T, TPR, CPT, AL>(slots(s, 2), dout, p.rows * p.Tk, next.dense(p), next.s,
                                        next.lo, next.hi, lane);  // shift 0
            next_st = __ldg(stats + walk.row);
            next_lam = __ldg(lam + next.h * p.lam_step);
        }
        walk.advance(p, blk.step);
        cp_async_commit();
    };
    issue(0);
    int turn = 0;  // stage of the current row
    for (int64_t rw = beg + grp - sub; rw < end; rw += blk.step, turn ^= 1) {
        const DiffRow w = next;
        const int d1 = next_d1, d2 = next_d2;
        const float4 st = next_st;
        const float lam_h = next_lam;
        const bool valid = rw + sub < end;
        issue(turn ^ 1);
        cp_async_wait<1>();  // this thread's copies of the row have landed
        if (!AL) diff_group_sync<TPR, BLOCK>(grp);
        const int lo = w.lo, hi = w.hi, j_lane = lane * V - w.s;
        const T *mrow = MASKED && w.general ? mask + (int64_t)w.b * Tk : nullptr;
        const float mul = MASKED && w.general ? 1.f : p.scale;
        // z is rounded before m is taken off (of both maps: the weights of one that
        // is near move by less than its bound)
        const bool far = !(fmaxf(fabsf(st.x), fabsf(st.z)) < kDiffNear);
        const uint4 *s1 = slots(turn, 0) + lane, *s2 = slots(turn, 1) + lane;
        const uint4 *sg = slots(turn, 2) + lane;
        float2 v1[CPT][H2], v2[CPT][H2];
        uint4 g4[CPT];  // dout as it is stored, 0 at invisible keys
        float2 t1 = f2(0.f), t2 = f2(0.f);
#pragma unroll
        for (int k = 0; k < CPT; ++k) {
            const int j0 = k * TPR * V + j_lane;
            if (!(j0 < hi && j0 + V > lo)) continue;
            diff_values<T, AL>(v1[k], diff_chunk<T, AL>(s1 + k * TPR, d1), mrow, mask_vec != 0, j0,
                               lo, hi, p.scale);
            diff_values<T, AL>(v2[k], diff_chunk<T, AL>(s2 + k * TPR, d2), mrow, mask_vec != 0, j0,
                               lo, hi, p.scale);
            g4[k] = sg[k * TPR];
            if (mrow || j0 < lo || j0 + V > hi)  // what dout holds at invisible keys
                keep_elements<T>(g4[k], relpos_bits<T>(mrow, j0, lo, hi));
            float2 g[H2];
            unpack2<T>(g4[k], g);
            // z - m first, at one rounding: what is left of one in the exponent goes by the
            // difference and not by m, and dlam sums all rows' weights
            if (!far) {
#pragma unroll
                for (int h2 = 0; h2 < H2; ++h2) {
                    v1[k][h2] = fma2(v1[k][h2], f2(mul), f2(-st.x));
                    v2[k][h2] = fma2(v2[k][h2], f2(mul), f2(-st.z));
                }
            } else {
#pragma unroll
                for (int h2 = 0; h2 < H2; ++h2) {
                    v1[k][h2] = add2(diff_rounded(v1[k][h2], mul), f2(-st.x));
                    v2[k][h2] = add2(diff_rounded(v2[k][h2], mul), f2(-st.z));
                }
            }
#pragma unroll
            for (int h2 = 0; h2 < H2; ++h2) {
                float2 a = mul2(v1[k][h2], f2(kLog2e));
                float2 b = mul2(v2[k][h2], f2(kLog2e));
                a.x = fast_exp2(a.x);
                a.y = fast_exp2(a.y);
                b.x = fast_exp2(b.x);
                b.y = fast_exp2(b.y);
                v1[k][h2] = a;
                v2[k][h2] = b;
                t1 = fma2(a, g[h2], t1);
                t2 = fma2(b, g[h2], t2);
            }
        }
        float dot1 = t1.x + t1.y, dot2 = t2.x + t2.y;
        diff_reduce2<TPR, BLOCK, OpSum>(dot1, dot2, red[turn], grp);
        dot1 *= st.y;
        dot2 *= st.w;
        if (valid && lane == 0) row_dot[w.by_head(p)] = dot2;
        const float w1 = p.scale * st.y, w2 = -p.scale * lam_h * st.w;
        const bool odd = !(fabsf(dot1) + fabsf(dot2) + fabsf(w1) + fabsf(w2) < INFINITY);
        T *r1 = dx1.p + w.at(dx1, p) + (AL ? lane * V : 0);
        T *r2 = dx2.p + w.at(dx2, p) + (AL ? lane * V : 0);
#pragma unroll
        for (int k = 0; k < CPT; ++k) {
            const int j0 = k * TPR * V + j_lane;
            uint4 a4 = make_uint4(0u, 0u, 0u, 0u), b4 = a4;
            if (j0 < hi && j0 + V > lo) {
                float2 g[H2];
                unpack2<T>(g4[k], g);
#pragma unroll
                for (int h2 = 0; h2 < H2; ++h2) {  // g - D first: it cancels where one key has all weight
                    v1[k][h2] = mul2(mul2(v1[k][h2], f2(w1)), add2(g[h2], f2(-dot1)));
                    v2[k][h2] = mul2(mul2(v2[k][h2], f2(w2)), add2(g[h2], f2(-dot2)));
                }
                if (odd) {  // 0 * NaN: invisible keys stay 0
                    const uint32_t bits = relpos_bits<T>(mrow, j0, lo, hi);
#pragma unroll
                    for (int h2 = 0; h2 < H2; ++h2) {
                        if (!((bits >> (2 * h2)) & 1u)) v1[k][h2].x = v2[k][h2].x = 0.f;
                        if (!((bits >> (2 * h2 + 1)) & 1u)) v1[k][h2].y = v2[k][h2].y = 0.f;
                    }
                }
                a4 = pack2<T>(v1[k]);
                b4 = pack2<T>(v2[k]);
            }
            if (valid && j0 < Tk) {
                relpos_store<T, AL>(r1, AL ? k * TPR * V : j0, Tk, a4);
                relpos_store<T, AL>(r2, AL ? k * TPR * V : j0, Tk, b4);
            }
        }
    }
    cp_async_wait<0>();  // (only empty groups are left)
}

// ----------------------------------------------------------------------------
// Any length and alignment: TPR threads per row (a warp, or the whole block),
// scalar accesses; the row is read again for every pass.
// ----------------------------------------------------------------------------
template <typename T>
struct DiffPoint {  // z of both maps at one key
    const T *x1, *x2, *mrow;
    float scale;
    // false: the key is invisible
    __device__ __forceinline__ bool at(int64_t j, float &z1, float &z2) const {
        const float mv = mrow ? Traits<T>::load1_cached(mrow + j) : 0.f;
        if (mv == -INFINITY) return false;
        z1 = fmaf(Traits<T>::load1(x1 + j), scale, mv);
        z2 = fmaf(Traits<T>::load1(x2 + j), scale, mv);
        return true;
    }
};
__device__ __forceinline__ void diff_online(float &m, float &s, float z) {
    if (z > m) {
        s = (m == -INFINITY ? s : s * fast_exp2((m - z) * kLog2e)) + 1.f;
        m = z;
    } else if (z != -INFINITY) {
        s += fast_exp2((z - m) * kLog2e);
    }
}

template <typename T, int TPR>
__global__ void __launch_bounds__(256)
diff_fw_loop(T *out, float4 *stats, const DiffRows<const T> x1, const DiffRows<const T> x2,
             const float *lam, const T *mask, const DiffShape p) {
    pdl_begin();
    using Tr = Traits<T>;
    constexpr int G = 256 / TPR;
    __shared__ float red[64];
    const int lane = threadIdx.x % TPR;
    const int64_t turns = (p.rows + (int64_t)gridDim.x * G - 1) / ((int64_t)gridDim.x * G);
    for (int64_t n = 0; n < turns; ++n) {
        const int64_t row = (n * gridDim.x + blockIdx.x) * G + threadIdx.x / TPR;
        if (row >= p.rows) continue;  // (a whole group: with TPR 256 the whole block)
        const DiffCursor c(p, row);
        const int64_t q = c.i + p.qoff, jend = p.causal ? min(p.Tk, q + 1) : p.Tk;
        const DiffPoint<T> pt{x1.p + x1.at(c.b, c.h, c.i, p.Tk), x2.p + x2.at(c.b, c.h, c.i, p.Tk),
                              mask ? mask + c.b * p.Tk : nullptr, p.scale};
        float m1 = -INFINITY, s1 = 0.f, m2 = -INFINITY, s2 = 0.f, z1, z2;
        for (int64_t j = lane; j < jend; j += TPR) {
            if (!pt.at(j, z1, z2)) continue;
            diff_online(m1, s1, z1);
            diff_online(m2, s2, z2);
        }
        group_natural_merge<TPR>(m1, s1, red);
        group_natural_merge<TPR>(m2, s2, red);
        const float nan = __int_as_float(0x7fc00000);
        const float i1 = m1 == INFINITY ? nan : (s1 == 0.f ? 0.f : 1.f / s1);
        const float i2 = m2 == INFINITY ? nan : (s2 == 0.f ? 0.f : 1.f / s2);
        if (m1 == -INFINITY) m1 = 0.f;
        if (m2 == -INFINITY) m2 = 0.f;
        if (stats && lane == 0) stats[row] = make_float4(m1, i1, m2, i2);
        const float li2 = -__ldg(lam + c.h * p.lam_step) * i2;
        T *o = out + row * p.Tk;
        for (int64_t j = lane; j < p.Tk; j += TPR) {
            float y = 0.f;
            if (j < jend && pt.at(j, z1, z2))
                y = fmaf(fast_exp2((z2 - m2) * kLog2e), li2, fast_exp2((z1 - m1) * kLog2e) * i1);
            Tr::store1(o + j, y);
        }
    }
}

template <typename T, int TPR>
__global__ void __launch_bounds__(256)
diff_bw_loop(const DiffRows<T> dx1, const DiffRows<T> dx2, float *row_dot, const T *dout,
             const DiffRows<const T> x1, const DiffRows<const T> x2, const float *lam,
             const float4 *stats, const T *mask, const DiffShape p) {
    pdl_begin();
    using Tr = Traits<T>;
    constexpr int G = 256 / TPR;
    __shared__ float red[64];
    const int lane = threadIdx.x % TPR;
    const int64_t turns = (p.rows + (int64_t)gridDim.x * G - 1) / ((int64_t)gridDim.x * G);
    for (int64_t n = 0; n < turns; ++n) {
        const int64_t row = (n * gridDim.x + blockIdx.x) * G + threadIdx.x / TPR;
        if (row >= p.rows) continue;
        const DiffCursor c(p, row);
        const int64_t q = c.i + p.qoff, jend = p.causal ? min(p.Tk, q + 1) : p.Tk;
        const DiffPoint<T> pt{x1.p + x1.at(c.b, c.h, c.i, p.Tk), x2.p + x2.at(c.b, c.h, c.i, p.Tk),
                              mask ? mask + c.b * p.Tk : nullptr, p.scale};
        const T *g = dout + row * p.Tk;
        const float4 st = __ldg(stats + row);
        float a = 0.f, b = 0.f, z1, z2;
        for (int64_t j = lane; j < jend; j += TPR) {
            if (!pt.at(j, z1, z2)) continue;
            const float gj = Tr::load1(g + j);
            a = fmaf(fast_exp2((z1 - st.x) * kLog2e), gj, a);
            b = fmaf(fast_exp2((z2 - st.z) * kLog2e), gj, b);
        }
        group_sum2<TPR>(a, b, red);
        a *= st.y;
        b *= st.w;
        if (lane == 0) row_dot[((int64_t)c.h * p.B + c.b) * p.Tq + c.i] = b;
        const float f1 = p.scale * st.y;
        const float f2_ = -p.scale * __ldg(lam + c.h * p.lam_step) * st.w;
        T *o1 = dx1.p + dx1.at(c.b, c.h, c.i, p.Tk), *o2 = dx2.p + dx2.at(c.b, c.h, c.i, p.Tk);
        for (int64_t j = lane; j < p.Tk; j += TPR) {
            float y1 = 0.f, y2 = 0.f;
            if (j < jend && pt.at(j, z1, z2)) {
                const float gj = Tr::load1(g + j);
                y1 = fast_exp2((z1 - st.x) * kLog2e) * f1 * (gj - a);
                y2 = fast_exp2((z2 - st.z) * kLog2e) * f2_ * (gj - b);
            }
            Tr::store1(o1 + j, y1);
            Tr::store1(o2 + j, y2);
        }
    }
}

// dlam[h] = -sum over b, i of the row's D_2, which lie head by head; one block
// per head (or one for all): each thread its own rows in order, then the threads
// in order.
constexpr int kDiffFoldThreads = 1024;
static __global__ void __launch_bounds__(kDiffFoldThreads)
diff_fold(float *dlam, const float *row_dot, const DiffShape p) {
    pdl_begin();
    __shared__ double part[32];
    const int64_t n = p.lam_step == 0 ? p.rows : p.rows / p.H;  // rows of the sum
    const float *src = row_dot + blockIdx.x * n;
    const bool wide = n % 4 == 0;  // (the workspace is 16-byte aligned)
    const int64_t steps = wide ? n / 4 : n;
    double v = 0.0;
    for (int64_t k0 = threadIdx.x; k0 < steps; k0 += 8 * kDiffFoldThreads) {
        float f[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            const int64_t k = k0 + (int64_t)u * kDiffFoldThreads;
            f[u] = 0.f;
            if (k < steps) {
                if (wide) {
                    const float4 q = __ldcg(reinterpret_cast<const float4 *>(src) + k);
                    f[u] = (q.x + q.y) + (q.z + q.w);
                } else {
                    f[u] = __ldcg(src + k);
                }
            }
        }
        v += (double)((f[0] + f[1]) + (f[2] + f[3])) + (double)((f[4] + f[5]) + (f[6] + f[7]));
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int w = 1; w < kDiffFoldThreads / 32; ++w) v += part[w];
        dlam[blockIdx.x] = (float)-v;
    }
}

}  // namespace lsr
