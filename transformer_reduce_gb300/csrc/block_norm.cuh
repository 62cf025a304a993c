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
// AL: rows of whole chunks on 16-byte addresses.
template <typename T, bool AL>
__device__ __forceinline__ uint4 bn_load(const T *row, int c, int hidden, bool stream) {
    constexpr int V = Traits<T>::kVec;
    if (AL) return stream ? ld_stream16(row + c) : ld_cached16(row + c);
    float f[V];
#pragma unroll
    for (int e = 0; e < V; ++e)
        f[e] = c + e < hidden ? Traits<T>::load1_cached(row + c + e) : 0.f;
    return Traits<T>::pack(f);
}
template <typename T, bool AL>
__device__ __forceinline__ void bn_store(T *row, int c, int hidden, const float (&f)[Traits<T>::kVec]) {
    constexpr int V = Traits<T>::kVec;
    if (AL) {
        st_stream16(row + c, Traits<T>::pack(f));
    } else {
#pragma unroll
        for (int e = 0; e < V; ++e)
            if (c + e < hidden) Traits<T>::store1(row + c + e, f[e]);
    }
}
template <typename T, bool AL>
__device__ __forceinline__ void bn_floats(const T *row, int c, int hidden, float (&f)[Traits<T>::kVec]) {
    Traits<T>::unpack(bn_load<T, AL>(row, c, hidden, false), f);
}

// Mean and rstd of a row in registers: the mean first, then the squares of the
// differences, so that a large mean costs no digits.  RMSNorm has mean 0.
template <typename T, int TPR, int CPT, bool LAYER, typename Red>
__device__ __forceinline__ void bn_stats(const float (&v)[CPT][Traits<T>::kVec], int lane, int hidden,
                                         float eps, Red &red, float &mean, float &rstd) {
    constexpr int V = Traits<T>::kVec;
    const float inv = 1.f / (float)hidden;
    mean = 0.f;
    if constexpr (LAYER) {
        float s = 0.f;
#pragma unroll
        for (int k = 0; k < CPT; ++k)
#pragma unroll
            for (int e = 0; e < V; ++e) s += v[k][e];  // (columns past the row are 0)
        mean = red.sum(s) * inv;
    }
    float q = 0.f;
#pragma unroll
    for (int k = 0; k < CPT; ++k) {
        const int c = (k * TPR + lane) * V;
#pragma unroll
        for (int e = 0; e < V; ++e) {
            const float d = v[k][e] - mean;
            if (!LAYER || c + e < hidden) q = fmaf(d, d, q);
        }
    }
    rstd = 1.f / sqrtf(red.sum(q) * inv + eps);
}

template <typename T, int TPR, int CPT, bool AL, bool LAYER>
__global__ void __launch_bounds__(bn_block<TPR>())
bn_fw(const BlockNorm<T> a, int64_t per) {
    pdl_begin();
    constexpr int V = Traits<T>::kVec;
    constexpr int BLOCK = bn_block<TPR>(), G = BLOCK / TPR;
    __shared__ float red_s[4 * BLOCK / 32];
    const int lane = threadIdx.x % TPR, grp = threadIdx.x / TPR;
    const int hidden = (int)a.hidden;
    BnReduce<TPR, BLOCK> red{red_s, grp};
    const int64_t beg = ((int64_t)blockIdx.x * G + grp) * per;
    const int64_t end = min(beg + per, a.rows);
    int64_t gate_at = a.gate && beg < end ? beg / a.gate_rows : 0;
    int64_t gate_left = a.gate && beg < end ? (gate_at + 1) * a.gate_rows - beg : 0;
    for (int64_t row = beg; row < end; ++row) {
        const int64_t at = row * a.hidden;
        float v[CPT][V], res[CPT][V];
#pragma unroll
        for (int k = 0; k < CPT; ++k) {
            const int c = (k * TPR + lane) * V;
            uint4 xr = make_uint4(0u, 0u, 0u, 0u), rr = xr;
            if (c < hidden) {
                xr = bn_load<T, AL>(a.x + at, c, hidden, true);
                rr = bn_load<T, AL>(a.r + at, c, hidden, true);
            }
            Traits<T>::unpack(xr, v[k]);
            Traits<T>::unpack(rr, res[k]);
        }
        float mean1 = 0.f, rstd1 = 1.f, mean2 = 0.f, rstd2 = 1.f;
        if (a.gamma_post)
            bn_stats<T, TPR, CPT, LAYER>(v, lane, hidden, a.eps, red, mean1, rstd1);
        const T *gate = a.gate ? a.gate + gate_at * a.hidden : nullptr;
#pragma unroll
        for (int k = 0; k < CPT; ++k) {
            const int c = (k * TPR + lane) * V;
            if (c >= hidden) continue;
            float f[V];
            if (a.gamma_post) {
                bn_floats<T, AL>(a.gamma_post, c, hidden, f);
#pragma unroll
                for (int e = 0; e < V; ++e) v[k][e] = (v[k][e] - mean1) * rstd1 * f[e];
                if (LAYER && a.beta_post) {
                    bn_floats<T, AL>(a.beta_post, c, hidden, f);
#pragma unroll
                    for (int e = 0; e < V; ++e) v[k][e] += f[e];
                }
            }
            if (gate) {
                bn_floats<T, AL>(gate, c, hidden, f);
#pragma unroll
                for (int e = 0; e < V; ++e) v[k][e] *= f[e];
            }
#pragma unroll
            for (int e = 0; e < V; ++e)
                v[k][e] = AL || c + e < hidden ? fmaf(a.residual_scale, res[k][e], v[k][e]) : 0.f;
            bn_store<T, AL>(a.h + at, c, hidden, v[k]);
        }
        if (a.gamma_pre) {
            bn_stats<T, TPR, CPT, LAYER>(v, lane, hidden, a.eps, red, mean2, rstd2);
#pragma unroll
            for (int k = 0; k < CPT; ++k) {
                const int c = (k * TPR + lane) * V;
                if (c >= hidden) continue;
                float f[V];
                bn_floats<T, AL>(a.gamma_pre, c, hidden, f);
#pragma unroll
                for (int e = 0; e < V; ++e) v[k][e] = (v[k][e] - mean2) * rstd2 * f[e];
                if (LAYER && a.beta_pre) {
                    bn_floats<T, AL>(a.beta_pre, c, hidden, f);
#pragma unroll
                    for (int e = 0; e < V; ++e) v[k][e] += f[e];
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
};

// ----------------------------------------------------------------------------
// Backward.  MULTI: a run holds several gates' rows, whose sums are written as
// each gate ends.
// ----------------------------------------------------------------------------
// The next row is copied ahead where two rows of four tensors fit a block.
template <int TPR, int CPT, bool AL>
constexpr bool bn_staged() { return AL && CPT * bn_block<TPR>() <= 1024; }
template <int TPR, int CPT, bool AL>
constexpr size_t bn_bw_smem(int vec) {
    // at the end a float per column and worker
    const size_t stage = bn_staged<TPR, CPT, AL>() ? (size_t)2 * 4 * CPT * bn_block<TPR>() * 16 : 0;
    const size_t sums = bn_block<TPR>() == TPR ? 0 : (size_t)bn_block<TPR>() * CPT * vec * 4;
    return stage > sums ? stage : sums;
}

template <typename T, int TPR, int CPT, bool AL, bool LAYER, bool MULTI>
__global__ void __launch_bounds__(bn_block<TPR>(), bn_block<TPR>() <= 512 ? 512 / bn_block<TPR>() : 1)
bn_bw(const BlockNorm<T> a, const BnCut cut, float *part, float *gate_part) {
    pdl_begin();
    constexpr int V = Traits<T>::kVec;
    constexpr int BLOCK = bn_block<TPR>(), G = BLOCK / TPR;
    constexpr bool kStaged = bn_staged<TPR, CPT, AL>();
    extern __shared__ __align__(128) uint4 dsmem[];  // [2][4][CPT][BLOCK], a thread's own slots
    __shared__ float red_s[4 * BLOCK / 32];
    const int lane = threadIdx.x % TPR, grp = threadIdx.x / TPR;
    const int hidden = (int)a.hidden;
    BnReduce<TPR, BLOCK> red{red_s, grp};
    const float inv = 1.f / (float)hidden;
    const bool post = a.gamma_post != nullptr, pre = a.gamma_pre != nullptr;
    const bool need_x = post || a.gate;
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
                if (a.dh) cp_async16(slot + 2 * CPT * BLOCK, a.dh + at + c);
                if (need_x) cp_async16(slot + 3 * CPT * BLOCK, a.x + at + c);
            }
        }
        if (kStaged) cp_async_commit();
    };
    auto fetch = [&](int which, const T *row, int s, int k, int c, float (&f)[V]) {
        if (kStaged)
            Traits<T>::unpack(stage[((s * 4 + which) * CPT + k) * BLOCK], f);
        else
            bn_floats<T, AL>(row, c, hidden, f);
    };
    float g2[CPT][V], b2[CPT][V], sa[CPT][V], sb[CPT][V], gp[CPT][V], bp[CPT][V];
#pragma unroll
    for (int k = 0; k < CPT; ++k)
#pragma unroll
        for (int e = 0; e < V; ++e)
            g2[k][e] = b2[k][e] = sa[k][e] = sb[k][e] = gp[k][e] = bp[k][e] = 0.f;

    issue(beg, 0);
    int turn = 0;
    for (int64_t row = beg; row < end; ++row, turn ^= 1) {
        issue(row + 1, turn ^ 1);
        if (kStaged) cp_async_wait<1>();  // this thread's copies of the row have landed
        const int64_t at = row * a.hidden;
        const float mean1 = LAYER ? __ldg(a.stats_in + row) : 0.f;
        const float rstd1 = __ldg(a.stats_in + a.rows + row);
        const float mean2 = LAYER ? __ldg(a.stats_in + 2 * a.rows + row) : 0.f;
        const float rstd2 = __ldg(a.stats_in + 3 * a.rows + row);
        float up[CPT][V];
        // the norm before the next block
        float s1 = 0.f, s2 = 0.f;
        if (pre) {
#pragma unroll
            for (int k = 0; k < CPT; ++k) {
                const int c = (k * TPR + lane) * V;
                if (c >= hidden) continue;
                float dy[V], hv[V], gm[V];
                fetch(0, a.dy + at, turn, k, c, dy);
                fetch(1, a.h_in + at, turn, k, c, hv);
                bn_floats<T, AL>(a.gamma_pre, c, hidden, gm);
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    const float hat = (hv[e] - mean2) * rstd2, g = dy[e] * gm[e];
                    if (LAYER) s1 += g;
                    s2 = fmaf(g, hat, s2);
                    g2[k][e] = fmaf(dy[e], hat, g2[k][e]);
                    if (LAYER) b2[k][e] += dy[e];
                }
            }
            red.sum2(s1, s2);
            s1 *= inv;
            s2 *= inv;
        }
        const T *gate = a.gate ? a.gate + gate_at * a.hidden : nullptr;
        float t1 = 0.f, t2 = 0.f;
#pragma unroll
        for (int k = 0; k < CPT; ++k) {
            const int c = (k * TPR + lane) * V;
            if (c >= hidden) continue;
            float f[V];
            if (a.dh) {
                fetch(2, a.dh + at, turn, k, c, up[k]);
            } else {
#pragma unroll
                for (int e = 0; e < V; ++e) up[k][e] = 0.f;
            }
            if (pre) {
                float dy[V], hv[V];
                fetch(0, a.dy + at, turn, k, c, dy);
                fetch(1, a.h_in + at, turn, k, c, hv);
                bn_floats<T, AL>(a.gamma_pre, c, hidden, f);
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    const float hat = (hv[e] - mean2) * rstd2;
                    up[k][e] = fmaf(rstd2, fmaf(-hat, s2, fmaf(dy[e], f[e], -s1)), up[k][e]);
                }
            }
            if (!AL) {  // (columns past the row)
#pragma unroll
                for (int e = 0; e < V; ++e)
                    if (c + e >= hidden) up[k][e] = 0.f;
            }
#pragma unroll
            for (int e = 0; e < V; ++e) f[e] = a.residual_scale * up[k][e];
            float xv[V], gm[V];
            if (need_x) {
                fetch(3, a.x + at, turn, k, c, xv);
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    xv[e] = post ? (xv[e] - mean1) * rstd1 : xv[e];
                    sa[k][e] = fmaf(up[k][e], xv[e], sa[k][e]);
                    if (LAYER) sb[k][e] += up[k][e];
                }
            }
            bn_store<T, AL>(a.dr + at, c, hidden, f);
            if (gate) {
                bn_floats<T, AL>(gate, c, hidden, gm);
#pragma unroll
                for (int e = 0; e < V; ++e) up[k][e] *= gm[e];
            }
            if (post) {
                bn_floats<T, AL>(a.gamma_post, c, hidden, gm);
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    up[k][e] *= gm[e];
                    if (LAYER) t1 += up[k][e];
                    t2 = fmaf(up[k][e], xv[e], t2);
                }
            }
        }
        if (post) {
            red.sum2(t1, t2);
            t1 *= inv;
            t2 *= inv;
        }
#pragma unroll
        for (int k = 0; k < CPT; ++k) {
            const int c = (k * TPR + lane) * V;
            if (c >= hidden) continue;
            if (post) {
                float xv[V];
                fetch(3, a.x + at, turn, k, c, xv);
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    const float hat = (xv[e] - mean1) * rstd1;
                    up[k][e] = rstd1 * fmaf(-hat, t2, up[k][e] - t1);
                }
            }
            bn_store<T, AL>(a.dx + at, c, hidden, up[k]);
        }
        if (MULTI && --gate_left == 0) {  // the gate's sums are complete
#pragma unroll
            for (int k = 0; k < CPT; ++k) {
                const int c = (k * TPR + lane) * V;
                if (c >= hidden) continue;
                float gm[V], gam[V], bet[V];
                bn_floats<T, AL>(gate, c, hidden, gm);
                if (post) bn_floats<T, AL>(a.gamma_post, c, hidden, gam);
                if (LAYER && a.beta_post) bn_floats<T, AL>(a.beta_post, c, hidden, bet);
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    gp[k][e] = fmaf(gm[e], sa[k][e], gp[k][e]);
                    if (LAYER) bp[k][e] = fmaf(gm[e], sb[k][e], bp[k][e]);
                    float d = post ? gam[e] * sa[k][e] : sa[k][e];
                    if (LAYER && a.beta_post) d = fmaf(bet[e], sb[k][e], d);
                    if (AL || c + e < hidden) a.dgate[gate_at * a.hidden + c + e] = d;
                    sa[k][e] = sb[k][e] = 0.f;
                }
            }
            ++gate_at;
            gate_left = a.gate_rows;
        }
    }
    if (kStaged) cp_async_wait<0>();  // (only empty groups are left)
    if (!MULTI) {
        // one gate (or none): its part of the gate's sums, and gate A, gate B
        const T *gate = a.gate && worker < cut.workers ? a.gate + gate_at * a.hidden : nullptr;
#pragma unroll
        for (int k = 0; k < CPT; ++k) {
            const int c = (k * TPR + lane) * V;
            if (c >= hidden) continue;
            float gm[V], gam[V], bet[V];
            if (gate) bn_floats<T, AL>(gate, c, hidden, gm);
            if (gate && post) bn_floats<T, AL>(a.gamma_post, c, hidden, gam);
            if (LAYER && a.beta_post) bn_floats<T, AL>(a.beta_post, c, hidden, bet);
#pragma unroll
            for (int e = 0; e < V; ++e) {
                gp[k][e] = gate ? gm[e] * sa[k][e] : sa[k][e];
                bp[k][e] = gate ? gm[e] * sb[k][e] : sb[k][e];
                if (gate && (AL || c + e < hidden)) {
                    float d = post ? gam[e] * sa[k][e] : sa[k][e];
                    if (LAYER && post && a.beta_post) d = fmaf(bet[e], sb[k][e], d);
                    if (cut.parts == 1)
                        a.dgate[gate_at * a.hidden + c + e] = d;
                    else
                        gate_part[worker * a.hidden + c + e] = d;
                }
            }
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
#pragma unroll
            for (int e = 0; e < V; ++e) {
                const float v = s == 0 ? g2[k][e] : s == 1 ? gp[k][e] : s == 2 ? b2[k][e] : bp[k][e];
                if (G > 1)
                    sums[grp * TPR * CPT * V + c + e] = v;
                else if (c + e < hidden)
                    out[c + e] = v;
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

// Column sums of the blocks' (or workers') parts: 32 columns of one vector per
// block, every eighth part per slice, then the slices in order.
struct BnFold {
    const float *part, *gate_part;
    float *out[4];  // dgamma_pre, dgamma_post, dbeta_pre, dbeta_post (NULL: not wanted)
    float *dgate;
    int64_t hidden, blocks, parts;
    int sums;
};
static __global__ void __launch_bounds__(256) bn_fold(const BnFold f) {
    pdl_begin();
    __shared__ float s[8][32];
    const int col = threadIdx.x & 31, slice = threadIdx.x >> 5;
    const int64_t c = (int64_t)blockIdx.x * 32 + col;
    const int64_t v = blockIdx.y;
    const float *src;
    float *dst;
    int64_t n, step;
    if (v < f.sums) {
        dst = f.out[v];
        src = f.part + v * f.hidden;
        n = f.blocks;
        step = f.sums * f.hidden;
    } else {
        dst = f.dgate + (v - f.sums) * f.hidden;
        src = f.gate_part + (v - f.sums) * f.parts * f.hidden;
        n = f.parts;
        step = f.hidden;
    }
    if (!dst) return;  // (the whole block)
    float t = 0.f;
    if (c < f.hidden) {
#pragma unroll 8
        for (int64_t k = slice; k < n; k += 8) t += __ldcg(src + k * step + c);
    }
    s[slice][col] = t;
    __syncthreads();
    if (slice == 0 && c < f.hidden) {
        for (int k = 1; k < 8; ++k) t += s[k][col];
        dst[c] = t;
    }
}

}  // namespace lsr
