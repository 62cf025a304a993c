// qk_norm_rope.cuh -- RMSNorm of every query and key head with the position
// rotation in the same pass, forward and backward (sm_103a).
//
// A head is a row x of D features.  With c, s the cosine and sine of the
// row's position and pair index p < rot / 2:
//     rstd = 1 / sqrt(mean(x^2) + eps),   n_j = x_j * rstd * gamma_j
//     (y_a, y_b) = (n_a c_p - n_b s_p,  n_b c_p + n_a s_p)
// over the pairs (a, b) = (p, p + rot/2), or (2p, 2p + 1) when interleaved;
// features from rot on are not rotated.  Backward, with the rotation undone:
//     dn = R^T dy,  g = gamma * dn,  xhat = x * rstd
//     dx_j = rstd * (g_j - xhat_j * sum_k(g_k xhat_k) / D)
//     dgamma_j = sum over all rows of dn_j * xhat_j
// Everything is FP32 between one load and one rounding: the normed value is
// not rounded before the rotation.
#pragma once

#include "launch.h"
#include "ls_device.cuh"

namespace lsr {

// Cosine and sine of pair p at one token's position; NaN for a position
// outside the table (there is no device-side trap).
__device__ __forceinline__ float2 qk_angle(const QkRope &r, int64_t pos, int p) {
    if (pos < 0 || pos >= r.max_pos) return f2(__int_as_float(0x7fc00000));
    const int64_t at = pos * (r.rot / 2) + p;
    return make_float2(__ldg(r.cos + at), __ldg(r.sin + at));
}

// The two features of slot u of a row: the rotation's pairs first, then the
// unrotated features two by two (b == D: the last of an odd count, alone).
__device__ __forceinline__ void qk_slot(const QkRope &r, int u, int &a, int &b) {
    const int half = r.rot / 2;
    if (u < half) {
        a = r.interleaved ? 2 * u : u;
        b = r.interleaved ? 2 * u + 1 : u + half;
    } else {
        a = 2 * u;  // rot + 2 (u - half)
        b = a + 1;
    }
}

// ----------------------------------------------------------------------------
// Any head size and alignment: one warp per head, a lane owns the slots lane,
// lane + 32, ... and both features of each, so calls may be in place.
// ----------------------------------------------------------------------------
template <typename T>
__global__ void __launch_bounds__(256)
qk_fw_loop(const QkSide<T> qs, const QkSide<T> ks, const QkRope r) {
    pdl_begin();
    using Tr = Traits<T>;
    const int lane = threadIdx.x & 31;
    const int64_t heads = qs.heads + ks.heads;
    const int64_t rows = r.tokens * heads;
    const int slots = (r.D + 1) / 2;
    for (int64_t row = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5); row < rows;
         row += (int64_t)gridDim.x * 8) {
        const int64_t tok = row / heads;
        int64_t h = row - tok * heads;
        const bool isq = h < qs.heads;
        const QkSide<T> &sd = isq ? qs : ks;
        if (!isq) h -= qs.heads;
        const T *x = sd.x + tok * sd.x_stride + h * r.D;
        T *o = sd.out + tok * sd.out_stride + h * r.D;
        float ss = 0.f;
        for (int j = lane; j < r.D; j += 32) {
            const float v = Tr::load1(x + j);
            ss = fmaf(v, v, ss);
        }
        ss = group_reduce<32, OpSum>(ss, nullptr);
        const float rstd = 1.f / sqrtf(ss / (float)r.D + r.eps);
        if (lane == 0 && sd.rstd_out) sd.rstd_out[tok * sd.heads + h] = rstd;
        const int64_t pos = r.rot ? __ldg(r.positions + tok) : 0;
        for (int u = lane; u < slots; u += 32) {
            int a, b;
            qk_slot(r, u, a, b);
            const bool two = b < r.D;
            float na = Tr::load1(x + a) * rstd * Tr::load1_cached(sd.gamma + a);
            float nb = two ? Tr::load1(x + b) * rstd * Tr::load1_cached(sd.gamma + b) : 0.f;
            if (u < r.rot / 2) {
                const float2 cs = qk_angle(r, pos, u);
                const float ya = na * cs.x - nb * cs.y;
                nb = nb * cs.x + na * cs.y;
                na = ya;
            }
            Tr::store1(o + a, na);
            if (two) Tr::store1(o + b, nb);
        }
    }
}

// Backward: block b < q_blocks works on query heads, the others on key heads,
// each on a contiguous run of its side's rows, with the run's gamma gradient
// in shared memory (one array per warp: a lane's features are its own).
template <typename T>
__global__ void __launch_bounds__(256)
qk_bw_loop(const QkSide<T> qs, const QkSide<T> ks, const QkRope r, float *part, int q_blocks) {
    pdl_begin();
    using Tr = Traits<T>;
    extern __shared__ float acc[];  // [8][D]
    const int lane = threadIdx.x & 31;
    const int warp = threadIdx.x >> 5;
    const bool isq = (int)blockIdx.x < q_blocks;
    const QkSide<T> &sd = isq ? qs : ks;
    const int64_t nblk = isq ? q_blocks : (int)gridDim.x - q_blocks;
    const int64_t blk = isq ? blockIdx.x : (int)blockIdx.x - q_blocks;
    const int64_t rows = r.tokens * sd.heads;
    const int64_t per = (rows + nblk - 1) / nblk;
    const int64_t beg = blk * per, end = min(beg + per, rows);
    const int slots = (r.D + 1) / 2;
    float *mine = acc + warp * r.D;
    for (int j = lane; j < r.D; j += 32) mine[j] = 0.f;
    __syncwarp();
    for (int64_t row = beg + warp; row < end; row += 8) {
        const int64_t tok = row / sd.heads, h = row - tok * sd.heads;
        const T *x = sd.x + tok * sd.x_stride + h * r.D;
        const T *dy = sd.dout + tok * sd.dout_stride + h * r.D;
        T *dx = sd.out + tok * sd.out_stride + h * r.D;
        const float rstd = __ldg(sd.rstd + row);
        const int64_t pos = r.rot ? __ldg(r.positions + tok) : 0;
        // dn and xhat of one slot
        auto slot = [&](int u, int a, int b, float &da, float &db, float &xa, float &xb) {
            const bool two = b < r.D;
            da = Tr::load1(dy + a);
            db = two ? Tr::load1(dy + b) : 0.f;
            xa = Tr::load1(x + a) * rstd;
            xb = two ? Tr::load1(x + b) * rstd : 0.f;
            if (u < r.rot / 2) {
                const float2 cs = qk_angle(r, pos, u);
                const float na = da * cs.x + db * cs.y;
                db = db * cs.x - da * cs.y;
                da = na;
            }
        };
        float s = 0.f;
        for (int u = lane; u < slots; u += 32) {
            int a, b;
            float da, db, xa, xb;
            qk_slot(r, u, a, b);
            slot(u, a, b, da, db, xa, xb);
            s = fmaf(da * Tr::load1_cached(sd.gamma + a), xa, s);
            if (b < r.D) s = fmaf(db * Tr::load1_cached(sd.gamma + b), xb, s);
        }
        s = group_reduce<32, OpSum>(s, nullptr) / (float)r.D;
        for (int u = lane; u < slots; u += 32) {
            int a, b;
            float da, db, xa, xb;
            qk_slot(r, u, a, b);
            slot(u, a, b, da, db, xa, xb);
            mine[a] = fmaf(da, xa, mine[a]);
            Tr::store1(dx + a, rstd * (da * Tr::load1_cached(sd.gamma + a) - xa * s));
            if (b < r.D) {
                mine[b] = fmaf(db, xb, mine[b]);
                Tr::store1(dx + b, rstd * (db * Tr::load1_cached(sd.gamma + b) - xb * s));
            }
        }
    }
    __syncthreads();
    for (int j = threadIdx.x; j < r.D; j += 256) {
        float v = acc[j];
        for (int w = 1; w < 8; ++w) v += acc[w * r.D + j];
        part[(int64_t)blockIdx.x * r.D + j] = v;
    }
}

// dgamma of both sides: the blocks' sums added in order.  blockIdx.y: side.
__global__ void __launch_bounds__(256)
qk_fold(float *dgq, float *dgk, const float *part, int D, int q_blocks, int blocks) {
    pdl_begin();
    __shared__ float sum[8][33];
    const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
    const int j = blockIdx.x * 32 + tx;
    const int beg = blockIdx.y ? q_blocks : 0, end = blockIdx.y ? blocks : q_blocks;
    float v = 0.f;
    if (j < D) {
#pragma unroll 8
        for (int b = beg + ty; b < end; b += 8) v += __ldg(part + (int64_t)b * D + j);
    }
    sum[ty][tx] = v;
    __syncthreads();
    float *out = blockIdx.y ? dgk : dgq;
    if (ty == 0 && j < D && out) {
#pragma unroll
        for (int t = 1; t < 8; ++t) v += sum[t][tx];
        out[j] = v;
    }
}

}  // namespace lsr
