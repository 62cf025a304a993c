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

#include <type_traits>

#include "launch.h"
#include "ls_device.cuh"

namespace lsr {

// ----------------------------------------------------------------------------
// Any head size and alignment.  One warp per head; its features go in slots of
// two: the rotation's pairs first, then the unrotated features two by two (the
// last of an odd count alone).  A lane owns the slots lane + 32 i, i < NS, and
// both features of each, so calls may be in place.  A warp takes a token, loads
// its angles once and goes through the heads, the next one's features loading
// while it works on the current one.  Bound by the latency
// of its loads (one head ahead; issue 56 and 34 % of the slots, the load pipe
// 20 %): [8192,(16,16),101] bf16 forward 72 us, backward 94 us (1.5 and 1.7 TB/s).
// The backward of more than 512 features spills about 460 bytes at 255 registers.
// ----------------------------------------------------------------------------
template <int NS>
struct QkSlots {
    int a[NS], b[NS];      // the features; -1: there is none
    float2 cs[NS];         // cosine and sine, (1, 0) where nothing is rotated
    __device__ __forceinline__ QkSlots(const QkRope &r, int lane) {
        const int half = r.rot / 2;
#pragma unroll
        for (int i = 0; i < NS; ++i) {
            const int u = lane + 32 * i;
            const bool far = !r.interleaved && u < half;
            a[i] = far ? u : 2 * u;
            b[i] = far ? u + half : 2 * u + 1;
            if (a[i] >= r.D) a[i] = -1;
            if (b[i] >= r.D) b[i] = -1;
            cs[i] = make_float2(1.f, 0.f);
        }
    }
    // The angles of a position; NaN outside the table (there is no device-side
    // trap).
    __device__ __forceinline__ void angles(const QkRope &r, int lane, int64_t tok) {
        const int half = r.rot / 2;
        if (half == 0) return;
        const int64_t pos = __ldg(r.positions + tok);
        const bool in = pos >= 0 && pos < r.max_pos;
#pragma unroll
        for (int i = 0; i < NS; ++i) {
            const int u = lane + 32 * i;
            if (u < half)
                cs[i] = in ? make_float2(__ldg(r.cos + pos * half + u),
                                         __ldg(r.sin + pos * half + u))
                           : f2(__int_as_float(0x7fc00000));
        }
    }
    template <typename T>
    __device__ __forceinline__ void load(const T *p, float2 (&v)[NS]) const {
#pragma unroll
        for (int i = 0; i < NS; ++i) {
            v[i].x = a[i] >= 0 ? Traits<T>::load1(p + a[i]) : 0.f;
            v[i].y = b[i] >= 0 ? Traits<T>::load1(p + b[i]) : 0.f;
        }
    }
    template <typename T>
    __device__ __forceinline__ void gamma(const T *p, float2 (&v)[NS]) const {
#pragma unroll
        for (int i = 0; i < NS; ++i) {
            v[i].x = a[i] >= 0 ? Traits<T>::load1_cached(p + a[i]) : 0.f;
            v[i].y = b[i] >= 0 ? Traits<T>::load1_cached(p + b[i]) : 0.f;
        }
    }
    template <typename T>
    __device__ __forceinline__ void store(T *p, const float2 (&v)[NS]) const {
#pragma unroll
        for (int i = 0; i < NS; ++i) {
            if (a[i] >= 0) Traits<T>::store1(p + a[i], v[i].x);
            if (b[i] >= 0) Traits<T>::store1(p + b[i], v[i].y);
        }
    }
    // Whether slot i is rotated.
    __device__ __forceinline__ bool turns(const QkRope &r, int lane, int i) const {
        return lane + 32 * i < r.rot / 2;
    }
};

template <typename T, int NS>
__global__ void __launch_bounds__(256)
qk_fw_slots(const QkSide<T> qs, const QkSide<T> ks, const QkRope r, int per_item) {
    pdl_begin();
    const int lane = threadIdx.x & 31;
    const int Hq = (int)qs.heads, heads = Hq + (int)ks.heads;
    const int per_token = (heads + per_item - 1) / per_item;
    const int64_t items = r.tokens * per_token;
    const float invD = 1.f / (float)r.D;
    QkSlots<NS> sl(r, lane);
    for (int64_t item = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5); item < items;
         item += (int64_t)gridDim.x * 8) {
        const int64_t tok = item / per_token;
        const int f0 = (int)(item - tok * per_token) * per_item, f1 = min(f0 + per_item, heads);
        auto row = [&](int f) {
            return f < Hq ? qs.x + tok * qs.x_stride + (int64_t)f * r.D
                          : ks.x + tok * ks.x_stride + (int64_t)(f - Hq) * r.D;
        };
        float2 next[NS], g[NS];
        sl.load(row(f0), next);
        sl.angles(r, lane, tok);
        for (int f = f0; f < f1; ++f) {
            const bool isq = f < Hq;
            const int h = isq ? f : f - Hq;
            if (f == f0 || f == Hq) sl.gamma(isq ? qs.gamma : ks.gamma, g);
            float2 v[NS];
            float2 ss = f2(0.f);
#pragma unroll
            for (int i = 0; i < NS; ++i) {
                v[i] = next[i];
                ss = fma2(v[i], v[i], ss);
            }
            if (f + 1 < f1) sl.load(row(f + 1), next);
            const float sum = group_reduce<32, OpSum>(ss.x + ss.y, nullptr);
            const float rstd = rsqrtf(fmaf(sum, invD, r.eps));
#pragma unroll
            for (int i = 0; i < NS; ++i) {
                v[i] = mul2(mul2(v[i], f2(rstd)), g[i]);
                if (sl.turns(r, lane, i)) {
                    const float2 n = v[i], cs = sl.cs[i];
                    v[i] = make_float2(fmaf(n.x, cs.x, -(n.y * cs.y)), fmaf(n.y, cs.x, n.x * cs.y));
                }
            }
            sl.store(isq ? qs.out + tok * qs.out_stride + (int64_t)h * r.D
                         : ks.out + tok * ks.out_stride + (int64_t)h * r.D,
                     v);
            float *rstd_out = isq ? qs.rstd_out : ks.rstd_out;
            if (lane == 0 && rstd_out) rstd_out[tok * (isq ? qs.heads : ks.heads) + h] = rstd;
        }
    }
}

// Backward: block b < q_blocks works on query heads, the others on key heads,
// with the gamma gradients of the lane's features in registers; the block's
// warps are added in shared memory at the end.
template <typename T, int NS>
__global__ void __launch_bounds__(256)
qk_bw_slots(const QkSide<T> qs, const QkSide<T> ks, const QkRope r, float *part, int q_blocks) {
    pdl_begin();
    extern __shared__ float acc[];  // [8][D]
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const bool isq = (int)blockIdx.x < q_blocks;
    const QkSide<T> &sd = isq ? qs : ks;
    const int64_t nblk = isq ? q_blocks : (int)gridDim.x - q_blocks;
    const int64_t blk = isq ? blockIdx.x : (int)blockIdx.x - q_blocks;
    const float invD = 1.f / (float)r.D;
    QkSlots<NS> sl(r, lane);
    float2 g[NS], dg[NS];
    sl.gamma(sd.gamma, g);
#pragma unroll
    for (int i = 0; i < NS; ++i) dg[i] = f2(0.f);
    for (int64_t tok = blk * 8 + warp; tok < r.tokens; tok += nblk * 8) {
        const T *xt = sd.x + tok * sd.x_stride, *yt = sd.dout + tok * sd.dout_stride;
        float2 nx[NS], ny[NS];
        sl.load(xt, nx);
        sl.load(yt, ny);
        float nr = __ldg(sd.rstd + tok * sd.heads);
        sl.angles(r, lane, tok);
        for (int64_t h = 0; h < sd.heads; ++h) {
            float2 x[NS], d[NS];
            const float rstd = nr;
            float2 t = f2(0.f);
#pragma unroll
            for (int i = 0; i < NS; ++i) {
                x[i] = mul2(nx[i], f2(rstd));  // xhat
                d[i] = ny[i];
                if (sl.turns(r, lane, i)) {  // dn
                    const float2 y = ny[i], cs = sl.cs[i];
                    d[i] = make_float2(fmaf(y.x, cs.x, y.y * cs.y), fmaf(y.y, cs.x, -(y.x * cs.y)));
                }
                const float2 p = mul2(d[i], x[i]);
                dg[i] = add2(dg[i], p);
                t = fma2(p, g[i], t);
            }
            if (h + 1 < sd.heads) {
                sl.load(xt + (h + 1) * r.D, nx);
                sl.load(yt + (h + 1) * r.D, ny);
                nr = __ldg(sd.rstd + tok * sd.heads + h + 1);
            }
            const float mean = group_reduce<32, OpSum>(t.x + t.y, nullptr) * invD;
#pragma unroll
            for (int i = 0; i < NS; ++i)
                d[i] = mul2(f2(rstd), fma2(x[i], f2(-mean), mul2(d[i], g[i])));
            sl.store(sd.out + tok * sd.out_stride + h * r.D, d);
        }
    }
#pragma unroll
    for (int i = 0; i < NS; ++i) {
        if (sl.a[i] >= 0) acc[warp * r.D + sl.a[i]] = dg[i].x;
        if (sl.b[i] >= 0) acc[warp * r.D + sl.b[i]] = dg[i].y;
    }
    __syncthreads();
    for (int j = threadIdx.x; j < r.D; j += 256) {
        float v = acc[j];
        for (int w = 1; w < 8; ++w) v += acc[w * r.D + j];
        part[(int64_t)blockIdx.x * r.D + j] = v;
    }
}

// ----------------------------------------------------------------------------
// Heads of whole vectors of V elements: 16 bytes where the head size, the
// rotated part, the pointers and the strides are multiples of them, else 8 or 4
// bytes.  LPR lanes hold a head, two vectors each:
//   halves       lane l < rot / 2V holds vectors l and l + rot / 2V, whose
//                elements are each other's partners; the other lanes hold the
//                unrotated vectors in the same manner;
//   interleaved  lane l holds vectors l and l + (half of the vectors), with
//                their pairs inside.
// (Neighbouring lanes hold neighbouring vectors: a 16-byte copy of every other
// vector would fetch each 32-byte sector twice.)
// Either way a lane needs V angles of its token's position, the same for every
// head of the token: a warp takes one token, loads them once, and goes through
// the heads of both sides, 32 / LPR at a time, the next heads' vectors loading
// while it works on the current ones.
// ----------------------------------------------------------------------------
// A vector of V elements as it lies in memory.
template <typename T, int V>
struct alignas(V * sizeof(T)) QkRaw {
    static constexpr int N = V * (int)sizeof(T) / 4;  // words
    uint32_t w[N];
};
template <typename T, int V>
__device__ __forceinline__ QkRaw<T, V> qk_zero() {
    QkRaw<T, V> r;
#pragma unroll
    for (int i = 0; i < QkRaw<T, V>::N; ++i) r.w[i] = 0u;
    return r;
}
// Gamma's vector at p, or zeros.
template <typename T, int V>
__device__ __forceinline__ QkRaw<T, V> qk_gamma(const T *p, bool there) {
    constexpr int N = QkRaw<T, V>::N;
    QkRaw<T, V> r = qk_zero<T, V>();
    if (there) {
        if constexpr (N == 4) {
            const uint4 u = ld_cached16(p);
            r.w[0] = u.x;
            r.w[1] = u.y;
            r.w[2] = u.z;
            r.w[3] = u.w;
        } else if constexpr (N == 2) {
            const uint2 u = __ldg(reinterpret_cast<const uint2 *>(p));
            r.w[0] = u.x;
            r.w[1] = u.y;
        } else {
            r.w[0] = __ldg(reinterpret_cast<const uint32_t *>(p));
        }
    }
    return r;
}
template <typename T, int V>
__device__ __forceinline__ void qk_unpack(const QkRaw<T, V> &r, float2 (&f)[V / 2]) {
#pragma unroll
    for (int h = 0; h < V / 2; ++h) {
        if constexpr (sizeof(T) == 4)
            f[h] = make_float2(__uint_as_float(r.w[2 * h]), __uint_as_float(r.w[2 * h + 1]));
        else if constexpr (std::is_same<T, __half>::value)
            f[h] = Traits<__half>::two(r.w[h]);
        else
            f[h] = bf16x2_to_float2(r.w[h]);
    }
}
template <typename T, int V>
__device__ __forceinline__ void qk_store(T *p, const float2 (&f)[V / 2]) {
    constexpr int N = QkRaw<T, V>::N;
    uint32_t w[N];
#pragma unroll
    for (int h = 0; h < V / 2; ++h) {
        if constexpr (sizeof(T) == 4) {
            w[2 * h] = __float_as_uint(f[h].x);
            w[2 * h + 1] = __float_as_uint(f[h].y);
        } else {
            w[h] = Traits<T>::word(f[h].x, f[h].y);
        }
    }
    if constexpr (N == 4)
        __stcs(reinterpret_cast<uint4 *>(p), make_uint4(w[0], w[1], w[2], w[3]));
    else if constexpr (N == 2)
        __stcs(reinterpret_cast<uint2 *>(p), make_uint2(w[0], w[1]));
    else
        __stcs(reinterpret_cast<uint32_t *>(p), w[0]);
}
// Asynchronous copy of one vector into the thread's slot.
template <typename T, int V>
__device__ __forceinline__ void qk_copy(QkRaw<T, V> *slot, const T *p) {
    if constexpr (QkRaw<T, V>::N == 4)
        cp_async16(slot, p);
    else if constexpr (QkRaw<T, V>::N == 2)
        asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(smem_addr(slot)), "l"(p)
                     : "memory");
    else
        cp_async4(slot, p);
}

struct QkLane {
    int va, vb;   // vectors
    bool ha, hb;  // there are such vectors
    bool ra, rb;  // they are rotated
};
template <int V, bool INTER>
__device__ __forceinline__ QkLane qk_lane(const QkRope &r, int l) {
    const int nv = r.D / V, hv = INTER ? 0 : r.rot / 2 / V;
    const int rest = (nv - 2 * hv + 1) / 2;  // lanes of the vectors that have no partner
    QkLane q;
    q.va = l < hv ? l : hv + l;
    q.vb = l < hv ? l + hv : hv + l + rest;
    q.ha = l < hv + rest;
    q.hb = q.ha && q.vb < nv;
    q.ra = INTER ? q.ha && q.va * V < r.rot : l < hv;
    q.rb = INTER ? q.hb && q.vb * V < r.rot : l < hv;
    return q;
}
// Lanes that hold a head (INTER as above).
inline int qk_lanes(int D, int rot, int V, bool inter) {
    const int nv = D / V, hv = inter ? 0 : rot / 2 / V;
    return hv + (nv - 2 * hv + 1) / 2;
}

// Cosines and sines of the lane's V angles, two by two (halves: those of
// vector va's features; interleaved: V / 2 for the pairs of vector va, then V / 2
// for vb's); 1 and 0 where nothing is rotated.
template <int V, bool INTER>
__device__ __forceinline__ void qk_angles(const QkRope &r, const QkLane &q, int64_t pos,
                                          float2 (&c)[V / 2], float2 (&s)[V / 2]) {
#pragma unroll
    for (int h = 0; h < V / 2; ++h) {
        c[h] = f2(1.f);
        s[h] = f2(0.f);
    }
    if (!q.ra) return;  // (vector vb is rotated only if va is)
    const int half = r.rot / 2;
    if (pos < 0 || pos >= r.max_pos) {
#pragma unroll
        for (int h = 0; h < V / 2; ++h) c[h] = s[h] = f2(__int_as_float(0x7fc00000));
        return;
    }
    const float *cp = r.cos + pos * half, *sp = r.sin + pos * half;
    if constexpr (INTER && V == 2) {
        c[0].x = __ldg(cp + q.va);
        s[0].x = __ldg(sp + q.va);
        if (q.rb) {
            c[0].y = __ldg(cp + q.vb);
            s[0].y = __ldg(sp + q.vb);
        }
    } else {
#pragma unroll
        for (int h = 0; h < V / 2; ++h) {
            const bool second = INTER && h >= V / 4;
            const int p = INTER ? (second ? q.vb * (V / 2) - V / 2 : q.va * (V / 2)) : q.va * V;
            if (!second || q.rb) {
                c[h] = __ldg(reinterpret_cast<const float2 *>(cp + p + 2 * h));
                s[h] = __ldg(reinterpret_cast<const float2 *>(sp + p + 2 * h));
            }
        }
    }
}

// One pair of features turned by (c, s).
__device__ __forceinline__ float2 qk_turn1(float2 v, float c, float s) {
    return make_float2(fmaf(v.x, c, -(v.y * s)), fmaf(v.y, c, v.x * s));
}

// Turns the lane's two vectors (BACK: by the opposite angles).
template <int V, bool INTER, bool BACK>
__device__ __forceinline__ void qk_turn(const QkLane &q, const float2 (&c)[V / 2],
                                        const float2 (&s)[V / 2], float2 (&a)[V / 2],
                                        float2 (&b)[V / 2]) {
    if (!q.ra) return;
    if constexpr (INTER) {
        auto at = [](const float2(&v)[V / 2], int i) { return i & 1 ? v[i / 2].y : v[i / 2].x; };
#pragma unroll
        for (int h = 0; h < V / 2; ++h)
            a[h] = qk_turn1(a[h], at(c, h), BACK ? -at(s, h) : at(s, h));
        if (q.rb) {
#pragma unroll
            for (int h = 0; h < V / 2; ++h) {
                const int i = V / 2 + h;
                b[h] = qk_turn1(b[h], at(c, i), BACK ? -at(s, i) : at(s, i));
            }
        }
    } else {
#pragma unroll
        for (int h = 0; h < V / 2; ++h) {
            const float2 up = BACK ? make_float2(-s[h].x, -s[h].y) : s[h];
            const float2 down = BACK ? s[h] : make_float2(-s[h].x, -s[h].y);
            const float2 x = a[h], y = b[h];
            a[h] = fma2(x, c[h], mul2(y, down));
            b[h] = fma2(y, c[h], mul2(x, up));
        }
    }
}

// Sum over the LPR lanes of a head.
template <int LPR>
__device__ __forceinline__ float qk_sum(float v) {
#pragma unroll
    for (int o = LPR / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

constexpr int kQkStages = 3;  // the current group and two on their way
template <typename T, int V>
constexpr size_t qk_bw_smem() { return (size_t)kQkStages * 256 * (4 * sizeof(QkRaw<T, V>) + 4); }

// Measured on a GB300, [16384,(16,16),64] bf16, packed: forward 26.6 us (5.1
// TB/s), backward with its fold 35.3 us (5.8 TB/s); memory latency with two
// blocks per SM (three, at 80 registers, measured 31.3 us forward).
//
// A group is the 32 / LPR heads of one side that a warp takes at once; an item
// is up to `per_item` groups of one token (all of them, unless that would
// leave too few items for the GPU).  ngq, ngk: groups of the two sides.
template <typename T, int V, int LPR, bool INTER>
__global__ void __launch_bounds__(256, 2)
qk_fw_vec(const QkSide<T> qs, const QkSide<T> ks, const QkRope r, int ngq, int ngk, int per_item) {
    pdl_begin();
    using Raw = QkRaw<T, V>;
    constexpr int H2 = V / 2;
    constexpr int RPW = 32 / LPR;
    const int lane = threadIdx.x & 31, l = lane % LPR, sub = lane / LPR;
    const QkLane q = qk_lane<V, INTER>(r, l);
    const int ng = ngq + ngk, per_token = (ng + per_item - 1) / per_item;
    const int64_t items = r.tokens * per_token;
    const float invD = 1.f / (float)r.D;
    const Raw zero = qk_zero<T, V>();
    const int64_t hop = (int64_t)gridDim.x * 8;
    // The warp's groups in order, copied kQkStages - 1 ahead: each thread its
    // own two vectors into its own slots.
    __shared__ __align__(128) Raw stage[kQkStages][2][256];
    int64_t i_item = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
    int64_t i_tok = per_token == 1 ? i_item : i_item / per_token;
    int i_f = (int)(i_item - i_tok * per_token) * per_item, i_end = min(i_f + per_item, ng);
    auto issue = [&](int st) {
        if (i_item < items) {
            const bool isq = i_f < ngq;
            const int h = (isq ? i_f : i_f - ngq) * RPW + sub;
            Raw *slot = &stage[st][0][threadIdx.x];
            const bool there = h < (int)(isq ? qs.heads : ks.heads);
            const T *x = (isq ? qs.x + i_tok * qs.x_stride : ks.x + i_tok * ks.x_stride) + h * r.D;
            if (there && q.ha)
                qk_copy<T, V>(slot, x + q.va * V);
            else
                slot[0] = zero;
            if (there && q.hb)
                qk_copy<T, V>(slot + 256, x + q.vb * V);
            else
                slot[256] = zero;
            if (++i_f == i_end) {
                i_item += hop;
                i_tok = per_token == 1 ? i_item : i_item / per_token;
                i_f = (int)(i_item - i_tok * per_token) * per_item;
                i_end = min(i_f + per_item, ng);
            }
        }
        cp_async_commit();
    };
#pragma unroll
    for (int st = 0; st < kQkStages - 1; ++st) issue(st);
    int st_cur = 0;
    int64_t item = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
    int64_t tok = per_token == 1 ? item : item / per_token;
    int pos = r.rot && item < items ? __ldg(r.positions + tok) : 0;
    for (int64_t next; item < items; item = next) {
        next = item + hop;
        const int64_t tok_next = per_token == 1 ? next : next / per_token;
        const int f0 = (int)(item - tok * per_token) * per_item, f1 = min(f0 + per_item, ng);
        float2 c[H2], s[H2];
        qk_angles<V, INTER>(r, q, pos, c, s);
        if (r.rot && next < items) pos = __ldg(r.positions + tok_next);
        for (int f = f0; f < f1;) {  // one side at a time
            const bool isq = f < ngq;
            const T *gamma = isq ? qs.gamma : ks.gamma;
            T *out = (isq ? qs.out + tok * qs.out_stride : ks.out + tok * ks.out_stride);
            float *rstd_out = isq ? qs.rstd_out : ks.rstd_out;
            const int heads = (int)(isq ? qs.heads : ks.heads);
            const int g0 = isq ? 0 : ngq, g1 = isq ? min(f1, ngq) : f1;
            if (rstd_out) rstd_out += tok * heads;
            float2 ga[H2], gb[H2];
            qk_unpack<T, V>(qk_gamma<T, V>(gamma + q.va * V, q.ha), ga);
            qk_unpack<T, V>(qk_gamma<T, V>(gamma + q.vb * V, q.hb), gb);
            for (; f < g1; ++f) {
                const int h = (f - g0) * RPW + sub;
                float2 a[H2], b[H2];
                issue(st_cur == 0 ? kQkStages - 1 : st_cur - 1);
                cp_async_wait<kQkStages - 1>();  // this thread's copies of the group have landed
                qk_unpack<T, V>(stage[st_cur][0][threadIdx.x], a);
                qk_unpack<T, V>(stage[st_cur][1][threadIdx.x], b);
                st_cur = st_cur + 1 == kQkStages ? 0 : st_cur + 1;
                float2 ss = f2(0.f);
#pragma unroll
                for (int e = 0; e < H2; ++e) ss = fma2(a[e], a[e], fma2(b[e], b[e], ss));
                // rsqrt.approx: at most 2 units in the last place off
                const float rstd = rsqrtf(fmaf(qk_sum<LPR>(ss.x + ss.y), invD, r.eps));
#pragma unroll
                for (int e = 0; e < H2; ++e) {
                    a[e] = mul2(mul2(a[e], f2(rstd)), ga[e]);
                    b[e] = mul2(mul2(b[e], f2(rstd)), gb[e]);
                }
                qk_turn<V, INTER, false>(q, c, s, a, b);
                if (h < heads) {
                    T *o = out + h * r.D;
                    if (q.ha) qk_store<T, V>(o + q.va * V, a);
                    if (q.hb) qk_store<T, V>(o + q.vb * V, b);
                    if (l == 0 && rstd_out) rstd_out[h] = rstd;
                }
            }
        }
        tok = tok_next;
    }
}

// Backward.  Blocks b < q_blocks work on query heads, the others on key heads,
// so that a lane has the gamma gradients of its 2V features of one side in
// registers; they are added over a warp's heads by shuffles and over the
// block's warps in shared memory at the end.  With p = dn * x and
// S = sum gamma p (x not normed): dgamma += rstd p and
// dx = rstd gamma dn - x rstd^3 S / D.
template <typename T, int V, int LPR, bool INTER>
__global__ void __launch_bounds__(256, 2)
qk_bw_vec(const QkSide<T> qs, const QkSide<T> ks, const QkRope r, float *part, int q_blocks) {
    pdl_begin();
    using Raw = QkRaw<T, V>;
    constexpr int H2 = V / 2;
    constexpr int RPW = 32 / LPR;
    __shared__ float sum[8][LPR * 2 * V + 1];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, l = lane % LPR, sub = lane / LPR;
    const QkLane q = qk_lane<V, INTER>(r, l);
    const bool isq = (int)blockIdx.x < q_blocks;
    const QkSide<T> &sd = isq ? qs : ks;
    const int64_t nblk = isq ? q_blocks : (int)gridDim.x - q_blocks;
    const int64_t blk = isq ? blockIdx.x : (int)blockIdx.x - q_blocks;
    const int heads = (int)sd.heads, ng = (heads + RPW - 1) / RPW;
    const float invD = 1.f / (float)r.D;
    const Raw zero = qk_zero<T, V>();
    float2 ga[H2], gb[H2], da[H2], db[H2];  // gamma and its gradients
    qk_unpack<T, V>(qk_gamma<T, V>(sd.gamma + q.va * V, q.ha), ga);
    qk_unpack<T, V>(qk_gamma<T, V>(sd.gamma + q.vb * V, q.hb), gb);
#pragma unroll
    for (int e = 0; e < H2; ++e) da[e] = db[e] = f2(0.f);
    extern __shared__ __align__(128) uint4 dsmem[];
    Raw *stage = reinterpret_cast<Raw *>(dsmem);  // [kQkStages][4][256], then the rows' rstd
    float *rs = reinterpret_cast<float *>(stage + kQkStages * 4 * 256) + threadIdx.x;
    const int64_t hop = nblk * 8;
    int64_t i_tok = blk * 8 + warp;
    int i_f = 0;
    auto issue = [&](int st) {
        if (i_tok < r.tokens) {
            const int h = i_f * RPW + sub;
            Raw *slot = stage + st * 4 * 256 + threadIdx.x;
            const bool there = h < heads;
            const T *x = sd.x + i_tok * sd.x_stride + h * r.D;
            const T *dy = sd.dout + i_tok * sd.dout_stride + h * r.D;
            if (there && q.ha) {
                qk_copy<T, V>(slot, x + q.va * V);
                qk_copy<T, V>(slot + 256, dy + q.va * V);
            } else {
                slot[0] = slot[256] = zero;
            }
            if (there && q.hb) {
                qk_copy<T, V>(slot + 512, x + q.vb * V);
                qk_copy<T, V>(slot + 768, dy + q.vb * V);
            } else {
                slot[512] = slot[768] = zero;
            }
            if (there) cp_async4(rs + st * 256, sd.rstd + i_tok * heads + h);
            else rs[st * 256] = 0.f;
            if (++i_f == ng) {
                i_f = 0;
                i_tok += hop;
            }
        }
        cp_async_commit();
    };
#pragma unroll
    for (int st = 0; st < kQkStages - 1; ++st) issue(st);
    int st_cur = 0;
    int pos = r.rot && blk * 8 + warp < r.tokens ? __ldg(r.positions + blk * 8 + warp) : 0;
    for (int64_t tok = blk * 8 + warp; tok < r.tokens; tok += hop) {
        T *dt = sd.out + tok * sd.out_stride;
        float2 c[H2], s[H2];
        qk_angles<V, INTER>(r, q, pos, c, s);
        if (r.rot && tok + hop < r.tokens) pos = __ldg(r.positions + tok + hop);
        for (int f = 0; f < ng; ++f) {
            const int h = f * RPW + sub;
            float2 a[H2], b[H2], x[H2], u[H2];
            issue(st_cur == 0 ? kQkStages - 1 : st_cur - 1);
            cp_async_wait<kQkStages - 1>();  // this thread's copies of the group have landed
            const Raw *slot = stage + st_cur * 4 * 256 + threadIdx.x;
            const float rstd = rs[st_cur * 256];
            qk_unpack<T, V>(slot[0], x);
            qk_unpack<T, V>(slot[256], a);
            qk_unpack<T, V>(slot[512], u);
            qk_unpack<T, V>(slot[768], b);
            st_cur = st_cur + 1 == kQkStages ? 0 : st_cur + 1;
            qk_turn<V, INTER, true>(q, c, s, a, b);  // dn
            float2 t = f2(0.f);
#pragma unroll
            for (int e = 0; e < H2; ++e) {
                const float2 p = mul2(a[e], x[e]), w = mul2(b[e], u[e]);
                da[e] = fma2(p, f2(rstd), da[e]);
                db[e] = fma2(w, f2(rstd), db[e]);
                t = fma2(p, ga[e], fma2(w, gb[e], t));
            }
            const float S = qk_sum<LPR>(t.x + t.y);
            if (h < heads) {
                // x rstd first: rstd^3 alone could leave fp32's range
                const float k = -(S * invD) * rstd;
                T *dx = dt + h * r.D;
#pragma unroll
                for (int e = 0; e < H2; ++e) {
                    a[e] = mul2(f2(rstd), fma2(mul2(x[e], f2(rstd)), f2(k), mul2(a[e], ga[e])));
                    b[e] = mul2(f2(rstd), fma2(mul2(u[e], f2(rstd)), f2(k), mul2(b[e], gb[e])));
                }
                if (q.ha) qk_store<T, V>(dx + q.va * V, a);
                if (q.hb) qk_store<T, V>(dx + q.vb * V, b);
            }
        }
    }
    // the warp's heads: lanes l of all subs; then the block's warps
#pragma unroll
    for (int e = 0; e < H2; ++e) {
#pragma unroll
        for (int o = 16; o >= LPR; o >>= 1) {
            da[e].x += __shfl_xor_sync(0xffffffffu, da[e].x, o);
            da[e].y += __shfl_xor_sync(0xffffffffu, da[e].y, o);
            db[e].x += __shfl_xor_sync(0xffffffffu, db[e].x, o);
            db[e].y += __shfl_xor_sync(0xffffffffu, db[e].y, o);
        }
        if (sub == 0) {
            float *to = &sum[warp][l * 2 * V + 2 * e];
            to[0] = da[e].x;
            to[1] = da[e].y;
            to[V] = db[e].x;
            to[V + 1] = db[e].y;
        }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < LPR * 2 * V; i += 256) {
        const QkLane w = qk_lane<V, INTER>(r, i / (2 * V));
        const bool second = i % (2 * V) >= V;
        if (second ? w.hb : w.ha) {
            float v = sum[0][i];
#pragma unroll
            for (int k = 1; k < 8; ++k) v += sum[k][i];
            part[(int64_t)blockIdx.x * r.D + (second ? w.vb : w.va) * V + i % V] = v;
        }
    }
}

// dgamma of both sides: the blocks' sums, 32 threads per feature, in a fixed
// order.  blockIdx.y: side.
static __global__ void __launch_bounds__(1024)
qk_fold(float *dgq, float *dgk, const float *part, int D, int q_blocks, int blocks) {
    pdl_begin();
    __shared__ float sum[32][33];
    const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
    const int j = blockIdx.x * 32 + tx;
    const int beg = blockIdx.y ? q_blocks : 0, end = blockIdx.y ? blocks : q_blocks;
    float v = 0.f;
    if (j < D) {
#pragma unroll 8
        for (int b = beg + ty; b < end; b += 32) v += __ldcg(part + (int64_t)b * D + j);
    }
    sum[ty][tx] = v;
    __syncthreads();
    float *out = blockIdx.y ? dgk : dgq;
    v = sum[tx][ty];  // one warp per feature
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    const int jo = blockIdx.x * 32 + ty;
    if (tx == 0 && jo < D && out) out[jo] = v;
}

}  // namespace lsr
