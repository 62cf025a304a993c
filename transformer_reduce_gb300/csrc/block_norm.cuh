// block_norm.cuh -- the norms after and before a block of a Transformer layer in
// one pass with the block's gate and the scaled residual stream (sm_103a).
//
// x is a block's output, r the residual stream, N either norm:
//     n = N_post(x)  (or x),   h = a r + gate * n,   y = N_pre(h)  (or none)
// with N the LayerNorm (mean, variance, gamma, beta) or the RMSNorm of the row.
// Backward, with up = dh + N_pre's input gradient of dy:
//     dr = a up,   dx = N_post's input gradient of gate * up
//     dgamma_pre = sum dy hhat,            dbeta_pre = sum dy
//     dgamma_post = sum gate up xhat,      dbeta_post = sum gate up
//     dgate = sum over the gate's rows of up n
//
// Memory traffic bounds both: two rows read and two written forward, four and
// two backward.  A row is owned by TPR threads with CPT 16-byte chunks of each
// tensor, every thread the same columns of all of its rows, so a tensor is read
// once and the backward's column sums stay in registers.  Under one gate only
// A = sum up xhat and B = sum up are summed: the gate and the gammas are
// constant there, so dgamma_post = gate A, dbeta_post = gate B and
// dgate = gamma_post A + beta_post B.  Workers (row groups) own contiguous runs
// that lie inside one gate's rows or hold whole gates' rows; the sums of a
// block's workers, then of the blocks, are added in order.
#pragma once

#include "launch.h"
#include "ls_device.cuh"
#include "relpos.cuh"  // relpos_reduce

namespace lsr {

template <int TPR>
constexpr int bn_block() { return TPR < 256 ? 256 : TPR; }

// Sums of a row over its group; `red` alternates between two halves so that one
// barrier is enough.
template <int TPR, int BLOCK>
struct BnReduce {
    float *red;
    int grp, turn = 0;
    __device__ __forceinline__ void sum2(float &a, float &b) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            a += __shfl_xor_sync(0xffffffffu, a, o);
            b += __shfl_xor_sync(0xffffffffu, b, o);
        }
        if constexpr (TPR > 32) {
            constexpr int NW = TPR / 32, BW = BLOCK / 32;
            float *s = red + turn * 2 * BW;
            turn ^= 1;
            if ((threadIdx.x & 31) == 0) {
                s[threadIdx.x >> 5] = a;
                s[BW + (threadIdx.x >> 5)] = b;
            }
            if constexpr (BLOCK == TPR)
                __syncthreads();
            else
                asm volatile("bar.sync %0, %1;" ::"r"(1 + grp), "r"(TPR) : "memory");
            a = s[grp * NW];
            b = s[BW + grp * NW];
#pragma unroll
            for (int w = 1; w < NW; ++w) {
                a += s[grp * NW + w];
                b += s[BW + grp * NW + w];
            }
        }
    }
    __device__ __forceinline__ float sum(float a) {
        float b = 0.f;
        sum2(a, b);
        return a;
    }
};

// Chunk of V elements at column c of a row; columns from `hidden` on are 0.
// AL: rows of whole chunks on 16-byte addresses.  An output may be the same tensor:
// no loads that want memory to be read-only for the whole kernel.
template <typename T, bool AL>
__device__ __forceinline__ uint4 bn_row(const T *row, int c, int hidden) {
    constexpr int V = Traits<T>::kVec;
    if (AL) return ld_stream16(row + c);
    float f[V];
#pragma unroll
    for (int e = 0; e < V; ++e) f[e] = c + e < hidden ? Traits<T>::load1(row + c + e) : 0.f;
    return Traits<T>::pack(f);
}
// The same as pairs, of a gate, gamma or beta, which every row reads and no output is.
template <typename T, bool AL>
__device__ __forceinline__ void bn_pairs(const T *row, int c, int hidden,
                                         float2 (&f)[Traits<T>::kVec / 2]) {
    constexpr int V = Traits<T>::kVec;
    if (AL) {
        unpack2<T>(ld_cached16(row + c), f);
    } else {
        float v[V];
#pragma unroll
        for (int e = 0; e < V; ++e)
            v[e] = c + e < hidden ? Traits<T>::load1_cached(row + c + e) : 0.f;
        unpack2<T>(Traits<T>::pack(v), f);
    }
}
template <typename T, bool AL>
__device__ __forceinline__ void bn_store(T *row, int c, int hidden,
                                         const float2 (&f)[Traits<T>::kVec / 2]) {
    constexpr int H2 = Traits<T>::kVec / 2;
    if (AL) {
        st_stream16(row + c, pack2<T>(f));
    } else {
#pragma unroll
        for (int e = 0; e < H2; ++e) {
            if (c + 2 * e < hidden) Traits<T>::store1(row + c + 2 * e, f[e].x);
            if (c + 2 * e + 1 < hidden) Traits<T>::store1(row + c + 2 * e + 1, f[e].y);
        }
    }
}

// Mean and rstd of a row in registers: the mean first, then the squares of the
// differences, so that a large mean costs no digits.  RMSNorm has mean 0.
template <typename T, int TPR, int CPT, bool AL, bool LAYER, typename Red>
__device__ __forceinline__ void bn_stats(const float2 (&v)[CPT][Traits<T>::kVec / 2], int lane,
                                         int hidden, float eps, Red &red, float &mean,
                                         float &rstd) {
    constexpr int V = Traits<T>::kVec, H2 = V / 2;
    const float inv = 1.f / (float)hidden;
    mean = 0.f;
    if constexpr (LAYER) {
        float2 s = f2(0.f);
#pragma unroll
        for (int k = 0; k < CPT; ++k)
#pragma unroll
            for (int e = 0; e < H2; ++e) s = add2(s, v[k][e]);  // (columns past the row are 0)
        mean = red.sum(s.x + s.y) * inv;
    }
    float2 q = f2(0.f);
#pragma unroll
    for (int k = 0; k < CPT; ++k) {
        const int c = (k * TPR + lane) * V;
        if (LAYER && c >= hidden) continue;
#pragma unroll
        for (int e = 0; e < H2; ++e) {
            float2 d = LAYER ? add2(v[k][e], f2(-mean)) : v[k][e];
            if (LAYER && !AL) {
                if (c + 2 * e >= hidden) d.x = 0.f;
                if (c + 2 * e + 1 >= hidden) d.y = 0.f;
            }
            q = fma2(d, d, q);
        }
    }
    rstd = 1.f / sqrtf(red.sum(q.x + q.y) * inv + eps);
}

// Resident blocks per SM asked of ptxas.
template <int TPR, int CPT>
constexpr int bn_fw_min_blocks() { return TPR > 512 ? 1 : (CPT <= 2 ? 768 : 512) / bn_block<TPR>(); }

// The next row is on its way (in registers) while the current one is normed.
template <typename T, int TPR, int CPT, bool AL, bool LAYER>
__global__ void __launch_bounds__(bn_block<TPR>(), (bn_fw_min_blocks<TPR, CPT>()))
bn_fw(const BlockNorm<T> a, int64_t per) {
    pdl_begin();
    constexpr int V = Traits<T>::kVec, H2 = V / 2;
    constexpr int BLOCK = bn_block<TPR>(), G = BLOCK / TPR;
    __shared__ float red_s[4 * BLOCK / 32];
    const int lane = threadIdx.x % TPR, grp = threadIdx.x / TPR;
    const int hidden = (int)a.hidden;
    BnReduce<TPR, BLOCK> red{red_s, grp};
    const int64_t beg = ((int64_t)blockIdx.x * G + grp) * per;
    const int64_t end = min(beg + per, a.rows);
    int64_t gate_at = a.gate && beg < end ? beg / a.gate_rows : 0;
    int64_t gate_left = a.gate && beg < end ? (gate_at + 1) * a.gate_rows - beg : 0;
    uint4 xr[CPT], rr[CPT];
    auto fetch = [&](int64_t row) {
#pragma unroll
        for (int k = 0; k < CPT; ++k) {
            const int c = (k * TPR + lane) * V;
            xr[k] = rr[k] = make_uint4(0u, 0u, 0u, 0u);
            if (c < hidden && row < end) {
                xr[k] = bn_row<T, AL>(a.x + row * a.hidden, c, hidden);
                rr[k] = bn_row<T, AL>(a.r + row * a.hidden, c, hidden);
            }
        }
    };
    fetch(beg);
    for (int64_t row = beg; row < end; ++row) {
        const int64_t at = row * a.hidden;
        float2 v[CPT][H2];
        uint4 res[CPT];
#pragma unroll
        for (int k = 0; k < CPT; ++k) {
            unpack2<T>(xr[k], v[k]);
            res[k] = rr[k];
        }
        fetch(row + 1);
        float mean1 = 0.f, rstd1 = 1.f, mean2 = 0.f, rstd2 = 1.f;
        if (a.gamma_post)
            bn_stats<T, TPR, CPT, AL, LAYER>(v, lane, hidden, a.eps, red, mean1, rstd1);
        const T *gate = a.gate ? a.gate + gate_at * a.hidden : nullptr;
#pragma unroll
        for (int k = 0; k < CPT; ++k) {
            const int c = (k * TPR + lane) * V;
            if (c >= hidden) continue;
            float2 f[H2];
            if (a.gamma_post) {
                bn_pairs<T, AL>(a.gamma_post, c, hidden, f);
#pragma unroll
                for (int e = 0; e < H2; ++e) {
                    if (LAYER) v[k][e] = add2(v[k][e], f2(-mean1));
                    v[k][e] = mul2(mul2(v[k][e], f2(rstd1)), f[e]);
                }
                if (LAYER && a.beta_post) {
                    bn_pairs<T, AL>(a.beta_post, c, hidden, f);
#pragma unroll
                    for (int e = 0; e < H2; ++e) v[k][e] = add2(v[k][e], f[e]);
                }
            }
            if (gate) {
                bn_pairs<T, AL>(gate, c, hidden, f);
#pragma unroll
                for (int e = 0; e < H2; ++e) v[k][e] = mul2(v[k][e], f[e]);
            }
            unpack2<T>(res[k], f);
#pragma unroll
            for (int e = 0; e < H2; ++e) v[k][e] = fma2(f2(a.residual_scale), f[e], v[k][e]);
            bn_store<T, AL>(a.h + at, c, hidden, v[k]);
        }
        if (a.gamma_pre) {
            bn_stats<T, TPR, CPT, AL, LAYER>(v, lane, hidden, a.eps, red, mean2, rstd2);
#pragma unroll
            for (int k = 0; k < CPT; ++k) {
                const int c = (k * TPR + lane) * V;
                if (c >= hidden) continue;
                float2 f[H2];
                bn_pairs<T, AL>(a.gamma_pre, c, hidden, f);
#pragma unroll
                for (int e = 0; e < H2; ++e) {
                    if (LAYER) v[k][e] = add2(v[k][e], f2(-mean2));
                    v[k][e] = mul2(mul2(v[k][e], f2(rstd2)), f[e]);
                }
                if (LAYER && a.beta_pre) {
                    bn_pairs<T, AL>(a.beta_pre, c, hidden, f);
#pragma unroll
                    for (int e = 0; e < H2; ++e) v[k][e] = add2(v[k][e], f[e]);
                }
                bn_store<T, AL>(a.y + at, c, hidden, v[k]);
            }
        }
        if (lane == 0) {
            a.stats[row] = mean1;
            a.stats[a.rows + row] = rstd1;
            a.stats[2 * a.rows + row] = mean2;
            a.stats[3 * a.rows + row] = rstd2;
        }
        if (a.gate && --gate_left == 0) {
            ++gate_at;
            gate_left = a.gate_rows;
        }
    }
}

// Cut of the rows into the workers' runs.
struct BnCut {
    int64_t per;      // rows of a run
    int64_t parts;    // runs of one gate's rows, or 0: a run holds whole gates' rows
    int64_t workers;
    int64_t blocks;
    int single;       // no gate or one: its sums follow from the totals of A and B
};

// ----------------------------------------------------------------------------
// Backward.  MULTI: a run holds several gates' rows, whose sums are written as
// each gate ends.  FORM: what the call has, known where a row is worked on (one
// kernel that tested it took 26.5 instead of 20.7 million instructions and 65
// instead of 46 us on [16384,1024] bf16).
// ----------------------------------------------------------------------------
// The next row is copied ahead where two rows of four tensors fit a block.
template <int TPR, int CPT, bool AL>
constexpr bool bn_staged() { return AL && CPT * bn_block<TPR>() <= 1024; }
template <int TPR, int CPT, bool AL>
constexpr size_t bn_bw_smem(int vec) {
    // at the end a float per column and worker
    const size_t stage = bn_staged<TPR, CPT, AL>() ? (size_t)2 * 4 * CPT * bn_block<TPR>() * 16 : 0;
    const size_t sums = bn_block<TPR>() == TPR ? 0 : (size_t)bn_block<TPR>() * CPT * vec * 4;
    return stage < sums ? sums : stage;
}

// FP32 sums of a chunk's columns.
template <bool AL, int H2>
__device__ __forceinline__ void bn_sums(float *row, int c, int hidden, const float2 (&v)[H2]) {
    if (AL) {
#pragma unroll
        for (int e = 0; e < H2; e += 2)
            *reinterpret_cast<float4 *>(row + c + 2 * e) =
                make_float4(v[e].x, v[e].y, v[e + 1].x, v[e + 1].y);
    } else {
#pragma unroll
        for (int e = 0; e < H2; ++e) {
            if (c + 2 * e < hidden) row[c + 2 * e] = v[e].x;
            if (c + 2 * e + 1 < hidden) row[c + 2 * e + 1] = v[e].y;
        }
    }
}

enum {
    kBnAny = 0,    // tests its pointers
    kBnGate = 1,   // both norms, a gate and dh
    kBnPost = 2,   // both norms and dh
    kBnPlain = 3,  // the norm before the next block and dh
};

template <typename T, int TPR, int CPT, bool AL, bool LAYER, bool MULTI, int FORM>
__global__ void __launch_bounds__(bn_block<TPR>(), TPR > 512 ? 1 : 512 / bn_block<TPR>())
bn_bw(const BlockNorm<T> a, const BnCut cut, float *part, float *gate_part) {
    pdl_begin();
    constexpr int V = Traits<T>::kVec, H2 = V / 2;
    constexpr int BLOCK = bn_block<TPR>(), G = BLOCK / TPR;
    constexpr bool kStaged = bn_staged<TPR, CPT, AL>();
    extern __shared__ __align__(128) uint4 dsmem[];  // [2][4][CPT][BLOCK], a thread's own slots
    __shared__ float red_s[4 * BLOCK / 32];
    const int lane = threadIdx.x % TPR, grp = threadIdx.x / TPR;
    const int hidden = (int)a.hidden;
    BnReduce<TPR, BLOCK> red{red_s, grp};
    const float inv = 1.f / (float)hidden;
    const bool pre = FORM != kBnAny || a.gamma_pre, with_dh = FORM != kBnAny || a.dh;
    const bool post = FORM == kBnAny ? a.gamma_post != nullptr : FORM != kBnPlain;
    const bool gated = FORM == kBnAny ? a.gate != nullptr : FORM == kBnGate;
    const bool need_x = post || gated;
    const int64_t worker = (int64_t)blockIdx.x * G + grp;
    int64_t beg = worker * cut.per, end = min(beg + cut.per, a.rows), gate_at = 0;
    if (cut.parts > 0) {
        gate_at = worker / cut.parts;
        beg = gate_at * a.gate_rows + (worker - gate_at * cut.parts) * cut.per;
        end = min(min(beg + cut.per, (gate_at + 1) * a.gate_rows), a.rows);
    } else {
        gate_at = beg / a.gate_rows;
    }
    if (worker >= cut.workers) end = beg;
    int64_t gate_left = a.gate_rows;

    uint4 *stage = dsmem + threadIdx.x;
    auto issue = [&](int64_t row, int s) {
        if (kStaged && row < end) {
            const int64_t at = row * a.hidden;
#pragma unroll
            for (int k = 0; k < CPT; ++k) {
                const int c = (k * TPR + lane) * V;
                if (c >= hidden) continue;
                uint4 *slot = stage + (s * 4 * CPT + k) * BLOCK;
                if (pre) {
                    cp_async16(slot, a.dy + at + c);
                    cp_async16(slot + CPT * BLOCK, a.h_in + at + c);
                }
                if (with_dh) cp_async16(slot + 2 * CPT * BLOCK, a.dh + at + c);
                if (need_x) cp_async16(slot + 3 * CPT * BLOCK, a.x + at + c);
            }
        }
        if (kStaged) cp_async_commit();
    };
    auto fetch = [&](int which, const T *row, int s, int k, int c, float2 (&f)[H2]) {
        if (kStaged)
            unpack2<T>(stage[((s * 4 + which) * CPT + k) * BLOCK], f);
        else
            unpack2<T>(bn_row<T, AL>(row, c, hidden), f);
    };
    float2 g2[CPT][H2], b2[CPT][H2], sa[CPT][H2], sb[CPT][H2], gp[CPT][H2], bp[CPT][H2];
#pragma unroll
    for (int k = 0; k < CPT; ++k)
#pragma unroll
        for (int e = 0; e < H2; ++e)
            g2[k][e] = b2[k][e] = sa[k][e] = sb[k][e] = gp[k][e] = bp[k][e] = f2(0.f);

    // the next row's statistics, as its tensors on their way
    float next[4] = {0.f, 0.f, 0.f, 0.f};
    auto issue_stats = [&](int64_t row) {
        if (row >= end) return;
        if (post) {
            if (LAYER) next[0] = __ldg(a.stats_in + row);
            next[1] = __ldg(a.stats_in + a.rows + row);
        }
        if (pre) {
            if (LAYER) next[2] = __ldg(a.stats_in + 2 * a.rows + row);
            next[3] = __ldg(a.stats_in + 3 * a.rows + row);
        }
    };
    issue(beg, 0);
    issue_stats(beg);
    int turn = 0;
    for (int64_t row = beg; row < end; ++row, turn ^= 1) {
        const int64_t at = row * a.hidden;
        const float mean1 = next[0], rstd1 = next[1], mean2 = next[2], rstd2 = next[3];
        issue(row + 1, turn ^ 1);
        issue_stats(row + 1);
        if (kStaged) cp_async_wait<1>();  // this thread's copies of the row have landed
        // (v - mean) * rstd in one multiply-add
        auto hat_of = [&](float2 v, float mean, float rstd) {
            return LAYER ? mul2(add2(v, f2(-mean)), f2(rstd)) : mul2(v, f2(rstd));
        };
        float2 up[CPT][H2], hat[CPT][H2];
        // the norm before the next block: up holds dy * gamma
        float s1 = 0.f, s2 = 0.f;
        if (pre) {
            float2 p1 = f2(0.f), p2 = f2(0.f);
#pragma unroll
            for (int k = 0; k < CPT; ++k) {
                const int c = (k * TPR + lane) * V;
                if (c >= hidden) continue;
                float2 dy[H2], gm[H2];
                fetch(0, a.dy + at, turn, k, c, dy);
                fetch(1, a.h_in + at, turn, k, c, hat[k]);
                bn_pairs<T, AL>(a.gamma_pre, c, hidden, gm);
#pragma unroll
                for (int e = 0; e < H2; ++e) {
                    hat[k][e] = hat_of(hat[k][e], mean2, rstd2);
                    up[k][e] = mul2(dy[e], gm[e]);
                    if (LAYER) p1 = add2(p1, up[k][e]);
                    p2 = fma2(up[k][e], hat[k][e], p2);
                    g2[k][e] = fma2(dy[e], hat[k][e], g2[k][e]);
                    if (LAYER) b2[k][e] = add2(b2[k][e], dy[e]);
                }
            }
            s1 = p1.x + p1.y;
            s2 = p2.x + p2.y;
            red.sum2(s1, s2);
            s1 *= inv;
            s2 *= inv;
        }
        const T *gate = gated ? a.gate + gate_at * a.hidden : nullptr;
        float2 q1 = f2(0.f), q2 = f2(0.f);
#pragma unroll
        for (int k = 0; k < CPT; ++k) {
            const int c = (k * TPR + lane) * V;
            if (c >= hidden) continue;
            float2 f[H2];
            if (with_dh) {
                fetch(2, a.dh + at, turn, k, c, f);
            } else {
#pragma unroll
                for (int e = 0; e < H2; ++e) f[e] = f2(0.f);
            }
#pragma unroll
            for (int e = 0; e < H2; ++e) {
                if (pre) {
                    float2 g = LAYER ? add2(up[k][e], f2(-s1)) : up[k][e];
                    g = fma2(hat[k][e], f2(-s2), g);
                    up[k][e] = fma2(f2(rstd2), g, f[e]);
                } else {
                    up[k][e] = f[e];
                }
                f[e] = mul2(f2(a.residual_scale), up[k][e]);
            }
            if (need_x) {
                fetch(3, a.x + at, turn, k, c, hat[k]);
#pragma unroll
                for (int e = 0; e < H2; ++e) {
                    if (post) hat[k][e] = hat_of(hat[k][e], mean1, rstd1);
                    sa[k][e] = fma2(up[k][e], hat[k][e], sa[k][e]);
                    if (LAYER) sb[k][e] = add2(sb[k][e], up[k][e]);
                }
            }
            bn_store<T, AL>(a.dr + at, c, hidden, f);
            if (gated) {
                bn_pairs<T, AL>(gate, c, hidden, f);
#pragma unroll
                for (int e = 0; e < H2; ++e) up[k][e] = mul2(up[k][e], f[e]);
            }
            if (post) {
                bn_pairs<T, AL>(a.gamma_post, c, hidden, f);
#pragma unroll
                for (int e = 0; e < H2; ++e) {
                    up[k][e] = mul2(up[k][e], f[e]);
                    if (LAYER) q1 = add2(q1, up[k][e]);
                    q2 = fma2(up[k][e], hat[k][e], q2);
                }
            }
        }
        float t1 = 0.f, t2 = 0.f;
        if (post) {
            t1 = q1.x + q1.y;
            t2 = q2.x + q2.y;
            red.sum2(t1, t2);
            t1 *= inv;
            t2 *= inv;
        }
#pragma unroll
        for (int k = 0; k < CPT; ++k) {
            const int c = (k * TPR + lane) * V;
            if (c >= hidden) continue;
            if (post) {
#pragma unroll
                for (int e = 0; e < H2; ++e) {
                    const float2 g = LAYER ? add2(up[k][e], f2(-t1)) : up[k][e];
                    up[k][e] = mul2(f2(rstd1), fma2(hat[k][e], f2(-t2), g));
                }
            }
            bn_store<T, AL>(a.dx + at, c, hidden, up[k]);
        }
        if (MULTI && --gate_left == 0) {  // the gate's sums are complete
#pragma unroll
            for (int k = 0; k < CPT; ++k) {
                const int c = (k * TPR + lane) * V;
                if (c >= hidden) continue;
                float2 f[H2];
                bn_pairs<T, AL>(gate, c, hidden, f);
#pragma unroll
                for (int e = 0; e < H2; ++e) {
                    gp[k][e] = fma2(f[e], sa[k][e], gp[k][e]);
                    if (LAYER) bp[k][e] = fma2(f[e], sb[k][e], bp[k][e]);
                }
                if (post) {
                    bn_pairs<T, AL>(a.gamma_post, c, hidden, f);
#pragma unroll
                    for (int e = 0; e < H2; ++e) sa[k][e] = mul2(f[e], sa[k][e]);
                }
                if (LAYER && a.beta_post) {
                    bn_pairs<T, AL>(a.beta_post, c, hidden, f);
#pragma unroll
                    for (int e = 0; e < H2; ++e) sa[k][e] = fma2(f[e], sb[k][e], sa[k][e]);
                }
                bn_sums<AL>(a.dgate + gate_at * a.hidden, c, hidden, sa[k]);
#pragma unroll
                for (int e = 0; e < H2; ++e) sa[k][e] = sb[k][e] = f2(0.f);
            }
            ++gate_at;
            gate_left = a.gate_rows;
        }
    }
    if (kStaged) cp_async_wait<0>();  // (only empty groups are left)
    if (!MULTI) {
        // rows under one gate: its part of the gate's sums, and gate A, gate B
        const bool own = a.gate && !cut.single && worker < cut.workers;
#pragma unroll
        for (int k = 0; k < CPT; ++k) {
            const int c = (k * TPR + lane) * V;
            if (c >= hidden) continue;
#pragma unroll
            for (int e = 0; e < H2; ++e) {
                gp[k][e] = sa[k][e];
                bp[k][e] = sb[k][e];
            }
            if (!own) continue;
            float2 f[H2];
            bn_pairs<T, AL>(a.gate + gate_at * a.hidden, c, hidden, f);
#pragma unroll
            for (int e = 0; e < H2; ++e) {
                gp[k][e] = mul2(f[e], gp[k][e]);
                if (LAYER) bp[k][e] = mul2(f[e], bp[k][e]);
            }
            if (post) {
                bn_pairs<T, AL>(a.gamma_post, c, hidden, f);
#pragma unroll
                for (int e = 0; e < H2; ++e) sa[k][e] = mul2(f[e], sa[k][e]);
            }
            if (LAYER && a.beta_post) {
                bn_pairs<T, AL>(a.beta_post, c, hidden, f);
#pragma unroll
                for (int e = 0; e < H2; ++e) sa[k][e] = fma2(f[e], sb[k][e], sa[k][e]);
            }
            bn_sums<AL>(cut.parts == 1 ? a.dgate + gate_at * a.hidden
                                       : gate_part + worker * a.hidden,
                        c, hidden, sa[k]);
        }
    }
    // the block's sums: dgamma_pre, dgamma_post, dbeta_pre, dbeta_post
    float *sums = reinterpret_cast<float *>(dsmem);
    constexpr int kSums = LAYER ? 4 : 2;
#pragma unroll
    for (int s = 0; s < kSums; ++s) {
        float *out = part + ((int64_t)blockIdx.x * kSums + s) * a.hidden;
        if (G > 1) __syncthreads();  // the copies, or the last sums, are no longer read
#pragma unroll
        for (int k = 0; k < CPT; ++k) {
            const int c = (k * TPR + lane) * V;
            const float2(&v)[H2] = s == 0 ? g2[k] : s == 1 ? gp[k] : s == 2 ? b2[k] : bp[k];
            if (G > 1) {
#pragma unroll
                for (int e = 0; e < H2; ++e)
                    *reinterpret_cast<float2 *>(&sums[grp * TPR * CPT * V + c + 2 * e]) = v[e];
            } else if (c < hidden) {
                bn_sums<AL>(out, c, hidden, v);
            }
        }
        if (G > 1) {
            __syncthreads();
            for (int c = threadIdx.x; c < hidden; c += BLOCK) {
                float v = sums[c];
                for (int g = 1; g < G; ++g) v += sums[g * TPR * CPT * V + c];
                out[c] = v;
            }
        }
    }
}

// Column sums of the blocks' (or workers') parts: C neighbouring columns per
// lane of one vector, every 16th part per warp, then the warps in order.
// single: vector 1 (and 3) are A (and B), and the gate's gradient follows from
// both.
constexpr int kBnFoldWarps = 16;
template <typename T>
struct BnFold {
    const float *part, *gate_part;
    float *out[4];  // dgamma_pre, dgamma_post, dbeta_pre, dbeta_post (NULL: not wanted)
    float *dgate;
    const T *gate, *gamma_post, *beta_post;  // single
    int64_t hidden, blocks, parts;
    int sums, single;
};
template <int C>
struct BnColumns {
    float v[C];
    __device__ __forceinline__ void load(const float *p) {
        if constexpr (C == 4) {
            const float4 f = __ldcg(reinterpret_cast<const float4 *>(p));
            v[0] = f.x;
            v[1] = f.y;
            v[2] = f.z;
            v[3] = f.w;
        } else {
            v[0] = __ldcg(p);
        }
    }
};
// The first warp gets the sums over n parts.
template <int C>
__device__ __forceinline__ BnColumns<C> bn_fold_columns(const float *src, int64_t n, int64_t step,
                                                        bool there, float (*s)[32 * C]) {
    const int lane = threadIdx.x & 31, slice = threadIdx.x >> 5;
    BnColumns<C> t = {};
    if (there) {
        for (int64_t k0 = slice; k0 < n; k0 += 8 * kBnFoldWarps) {
            BnColumns<C> f[8];
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                const int64_t k = k0 + (int64_t)u * kBnFoldWarps;
                f[u] = BnColumns<C>{};
                if (k < n) f[u].load(src + k * step);
            }
#pragma unroll
            for (int i = 0; i < C; ++i)
                t.v[i] += ((f[0].v[i] + f[1].v[i]) + (f[2].v[i] + f[3].v[i])) +
                          ((f[4].v[i] + f[5].v[i]) + (f[6].v[i] + f[7].v[i]));
        }
    }
    __syncthreads();  // the last sums' slices have been read
#pragma unroll
    for (int i = 0; i < C; ++i) s[slice][lane * C + i] = t.v[i];
    __syncthreads();
    if (slice == 0)
        for (int k = 1; k < kBnFoldWarps; ++k)
#pragma unroll
            for (int i = 0; i < C; ++i) t.v[i] += s[k][lane * C + i];
    return t;
}
template <typename T, int C>
__global__ void __launch_bounds__(32 * kBnFoldWarps) bn_fold(const BnFold<T> f) {
    pdl_begin();
    __shared__ float s[kBnFoldWarps][32 * C];
    const int64_t c = ((int64_t)blockIdx.x * 32 + (threadIdx.x & 31)) * C;
    const int64_t v = blockIdx.y;
    const bool there = c < f.hidden, writes = there && threadIdx.x < 32;
    const int64_t step = f.sums * f.hidden;
    if (v >= f.sums) {  // a gate's parts
        const int64_t k = v - f.sums;
        const BnColumns<C> t = bn_fold_columns<C>(f.gate_part + k * f.parts * f.hidden + c, f.parts,
                                                  f.hidden, there, s);
        if (writes)
            for (int i = 0; i < C; ++i) f.dgate[k * f.hidden + c + i] = t.v[i];
        return;
    }
    const bool gate = f.single && f.gate && v == 1;
    const bool scaled = f.single && f.gate && (v & 1);
    float *out = f.out[v];
    if (!out && !gate) return;  // (the whole block)
    BnColumns<C> t = bn_fold_columns<C>(f.part + v * f.hidden + c, f.blocks, step, there, s);
    if (writes && out)
        for (int i = 0; i < C; ++i)
            out[c + i] = scaled ? t.v[i] * Traits<T>::load1_cached(f.gate + c + i) : t.v[i];
    if (!gate) return;
    if (writes && f.gamma_post)
        for (int i = 0; i < C; ++i) t.v[i] *= Traits<T>::load1_cached(f.gamma_post + c + i);
    if (f.beta_post) {
        const BnColumns<C> b =
            bn_fold_columns<C>(f.part + 3 * f.hidden + c, f.blocks, step, there, s);
        if (writes)
            for (int i = 0; i < C; ++i)
                t.v[i] = fmaf(b.v[i], Traits<T>::load1_cached(f.beta_post + c + i), t.v[i]);
    }
    if (writes)
        for (int i = 0; i < C; ++i) f.dgate[c + i] = t.v[i];
}

}  // namespace lsr
