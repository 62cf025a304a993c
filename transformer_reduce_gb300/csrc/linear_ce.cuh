// linear_ce.cuh -- softmax cross entropy taken from hidden states x [rows, D]
// and a vocabulary matrix W [V, D] without keeping the logits z = x W^T, and its
// gradients (sm_103a, fifth-generation tensor cores).
//
//     lse_r  = log sum_v exp(z_rv),   loss_r = lse_r - z_r,t(r)
//     q_rv   = dloss_r (exp(z_rv - lse_r) - [v == t(r)])
//     dx     = q W,   dW = q^T x
//
// Three matrix products of 2 rows D V operations bound all of it (the backward
// needs the logits again, so it makes three, the forward one).
//
//  * The rows that count (target >= 0) are first gathered into a dense copy of x
//    in their order, so that ignored rows cost nothing and what they hold, NaN
//    or not, touches nothing.
//  * One persistent kernel makes every product, in pairs of blocks on tiles of
//    256 by 256: in either block one warp loads 128 rows of A and of B, 64
//    elements wide, with TMA, one thread of the pair issues tcgen05.mma on both
//    blocks' operands, and eight warps read the block's 128 rows of FP32
//    accumulators from tensor memory, which holds two tiles so that the next
//    product runs meanwhile.  (A block alone on 128 by 256 reads all of B itself:
//    shared memory then takes as long as the tensor cores, and [8192,1024] bf16
//    by 50257 took 595 us forward.)
//  * Forward: the eight warps reduce a tile of logits to each row's largest
//    logit and sum of exponentials, per 128 columns; a second kernel joins a
//    row's parts in order.
//  * Backward, by pieces of the vocabulary: the logits of a piece become q,
//    rounded to the operands' 16-bit type, in the workspace; q W is added to dx
//    in FP32 over the pieces, q^T x is the piece's rows of dW.
//  * fp32 operands are three bf16 planes each (8 + 8 + 8 bits of the 24); six
//    products of planes, smallest first, leave out terms below 2^-24.
//  * The tensor cores cut the accumulator off where a step of 16 is added, so that
//    a long sum drifts: sums of so many elements (lce_cut) are therefore added up
//    in registers, rounding to nearest.
//
// Every sum has one order, given by the sizes: the results are reproducible.
#pragma once

#include <type_traits>

#include "launch.h"
#include "tensor_core.cuh"

namespace lsr {

constexpr int kLceM = 256, kLceN = 256, kLceK = 64;  // tile, and elements of a step along K
constexpr int kLceHalf = 128;  // rows of A, rows of B and rows of the accumulator in a block
constexpr int kLceStages = 6;
constexpr int kLceBox = 64 * kLceK * 2;  // bytes of one 64 x 64 TMA box
constexpr int kLceStage = 2 * kLceHalf / 64 * kLceBox;
constexpr int kLceThreads = 320;  // loader, issuer, eight warps on the accumulators
// Columns that a warp turns at a time where the rows of an output do not start on
// 16-byte addresses, and the floats it takes.
constexpr int kLceTurn = 16;
constexpr int kLceTurnFloats = 32 * (kLceTurn + 1);
constexpr size_t kLceSmem = (size_t)kLceStages * kLceStage + 8 * kLceTurnFloats * 4 + 1024;
constexpr int kLceSms = 152;  // what the cuts are made for
constexpr int kLceChunk = 1024;  // rows counted together
constexpr int kLcePackRows = 8;  // one per warp
// Rows up to which every block of the packing counts all targets itself,
// without a launch before it (at 8192 rows that took 35 us in the backward
// instead of 5 and 10).
constexpr int64_t kLceCountRows = 2048;

enum { kLceStats = 0, kLceQ = 1, kLceGrads = 2 };

// Steps of kLceK whose products the tensor cores sum before registers add them to
// the tile's sum.  The accumulator is cut off, not rounded, where a step of 16 is
// added, so that a sum of terms of one sign loses up to 2^-23 of itself with each
// (measured: two thirds of that): uncut, dW of [2097152,8] was 1.2 % off and the
// lse of 65536 hidden elements 8e-3.  With these cuts 64 * 16 elements lose at most
// 8e-6 and 64 * 64 3e-5.  (Cuts of 4 and 16 steps took 8 % of the forward and of
// the backward of [8192,1024] bf16 by 50257.)  fp32 sums are cut every 256 elements
// (dx of [1001,333] by 10007 was 1.9e-5 of its largest off uncut), the logits at
// every step: exp(z - lse) - 1 of a row whose weight is on its target magnifies
// their errors.  Of [14,1024] by 65 with such targets dx and dW were four times as
// far from 64 bits as a plain FP32 form's at cuts of 4 steps, twice at 2, and are as
// near as those at 1 (the backward of [1001,333] by 10007: 129, 133 and 137 us).
template <int EPI, typename T>
constexpr int lce_cut() {
    return sizeof(T) == 4 ? (EPI == kLceGrads ? 4 : 1) : EPI == kLceGrads ? 64 : 16;
}

// What the kernels of one call share.
struct LceArgs {
    int64_t rows, D, V;     // as given
    int64_t row_cap;        // rows of the dense copy, a multiple of kLceM
    int64_t v0, vc;         // the piece: vocabulary entries [v0, v0 + vc)
    int64_t q_pitch;        // elements of a row of q
    int bf16;               // operand type of the products
    int first, last;        // of the pieces
    int with_dw;
    int64_t splits, split_k;  // cuts of the sum over a piece in dx, and steps of K of each
    // in the workspace
    const int *count;       // rows that count
    const int *row_of;      // [row_cap] their index
    const int *target;      // [row_cap]
    const float *row_lse;   // [row_cap]
    const float *row_up;    // [row_cap] dloss / unscale
    const float *unscale;   // what q is to be multiplied with
    float *row_hit;         // [row_cap] the target's logit
    float2 *part;           // [half tiles of V][row_cap] (largest logit * log2 e, sum)
    void *q;                // [1, fp32: 3][row_cap][q_pitch]
    float *dx_sum;          // [splits][row_cap][sum_pitch] over the pieces so far
    int64_t sum_pitch;
    int aligned;            // the rows of dx and dw start on 16-byte addresses
    void *dx, *dw;          // outputs
};

// The planes of the s-th product of two fp32 operands, smallest terms first: of
// A 2, 0, 1, 1, 0, 0 and of B 0, 2, 1, 0, 1, 0.
__device__ __forceinline__ int2 lce_planes(int s) {
    return make_int2((0x001102 >> (4 * s)) & 3, (0x010120 >> (4 * s)) & 3);
}

// x in planes of the operand type: the value itself, or its three bf16 parts.
template <typename T>
struct LceSplit {
    using O = T;
    static constexpr int kPlanes = 1;
    __device__ __forceinline__ static void put(O *p, int64_t, T v) { *p = v; }
};
template <>
struct LceSplit<float> {
    using O = __nv_bfloat16;
    static constexpr int kPlanes = 3;
    __device__ __forceinline__ static void parts(float v, O (&o)[3]) {
        o[0] = __float2bfloat16_rn(v);
        const float a = __bfloat162float(o[0]);
        // what is left of a finite value; an infinite one would leave NaN
        const float r = fabsf(a) < INFINITY ? v - a : 0.f;
        o[1] = __float2bfloat16_rn(r);
        o[2] = __float2bfloat16_rn(r - __bfloat162float(o[1]));
    }
    __device__ __forceinline__ static void put(O *p, int64_t plane, float v) {
        O o[3];
        parts(v, o);
        p[0] = o[0];
        p[plane] = o[1];
        p[2 * plane] = o[2];
    }
};

// ----------------------------------------------------------------------------
// Rows that count.
// ----------------------------------------------------------------------------
struct LcePack {
    int64_t rows, D, V, row_cap, pitch;  // pitch: elements of a row of the copy
    int backward;
    const int32_t *target;
    const float *lse, *dloss;
    int *chunk_count;     // [chunks], NULL: up to kLceCountRows rows
    float *chunk_up;      // [chunks] largest |dloss|
    int *count, *row_of, *row_target;
    float *row_lse, *row_up, *unscale;
    float *loss, *lse_out;  // forward: of the rows that do not count
};

// A row counts when it has a class.  (The backward keeps those beyond the
// vocabulary too: their gradients are NaN.)
__device__ __forceinline__ bool lce_counts(const LcePack &p, int32_t t) {
    return t >= 0 && (p.backward || t < p.V);
}

static __global__ void __launch_bounds__(256) lce_count(const LcePack p) {
    pdl_begin();
    __shared__ int n_s[8];
    __shared__ float up_s[8];
    int n = 0;
    float up = 0.f;
    bool odd = false;  // a gradient that is not finite
    for (int i = threadIdx.x; i < kLceChunk; i += 256) {
        const int64_t r = (int64_t)blockIdx.x * kLceChunk + i;
        if (r < p.rows && lce_counts(p, __ldg(p.target + r))) {
            ++n;
            if (p.backward) {
                const float g = fabsf(__ldg(p.dloss + r));
                odd |= !(g < INFINITY);
                up = fmaxf(up, g);
            }
        }
    }
    if (odd) up = INFINITY;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        n += __shfl_xor_sync(0xffffffffu, n, o);
        up = fmaxf(up, __shfl_xor_sync(0xffffffffu, up, o));
    }
    if ((threadIdx.x & 31) == 0) {
        n_s[threadIdx.x >> 5] = n;
        up_s[threadIdx.x >> 5] = up;
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int w = 1; w < 8; ++w) {
            n += n_s[w];
            up = fmaxf(up, up_s[w]);
        }
        p.chunk_count[blockIdx.x] = n;
        p.chunk_up[blockIdx.x] = up;
    }
}

// Copies kLcePackRows rows of x to their places.  T: type of x.  dx: of a backward, where the
// rows that do not count become 0.
template <typename T>
__global__ void __launch_bounds__(256)
lce_pack_rows(typename LceSplit<T>::O *out, const T *x, T *dx, const LcePack p) {
    pdl_begin();
    using O = typename LceSplit<T>::O;
    __shared__ int before_s[8], all_s[8];
    __shared__ float up_s[8];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int64_t row0 = (int64_t)blockIdx.x * kLcePackRows;
    const int64_t chunk = row0 / kLceChunk;
    const int64_t chunks = (p.rows + kLceChunk - 1) / kLceChunk;
    int before = 0, all = 0;
    float up = 0.f;
    if (p.chunk_count) {
        for (int64_t c = tid; c < chunks; c += 256) {
            const int n = p.chunk_count[c];
            all += n;
            if (c < chunk) before += n;
            up = fmaxf(up, p.chunk_up[c]);
        }
        for (int64_t r = chunk * kLceChunk + tid; r < row0; r += 256)
            before += lce_counts(p, __ldg(p.target + r));
    } else {
#pragma unroll 4
        for (int r = tid; r < (int)p.rows; r += 256) {
            const bool counts = lce_counts(p, __ldg(p.target + r));
            all += counts;
            before += counts && r < row0;
            if (p.backward) {
                const float g = counts ? fabsf(__ldg(p.dloss + r)) : 0.f;
                up = g < INFINITY ? fmaxf(up, g) : INFINITY;  // (of NaN too)
            }
        }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        before += __shfl_xor_sync(0xffffffffu, before, o);
        all += __shfl_xor_sync(0xffffffffu, all, o);
        up = fmaxf(up, __shfl_xor_sync(0xffffffffu, up, o));
    }
    if (lane == 0) {
        before_s[warp] = before;
        all_s[warp] = all;
        up_s[warp] = up;
    }
    __syncthreads();
    before = all = 0;
    up = 0.f;
    for (int w = 0; w < 8; ++w) {
        before += before_s[w];
        all += all_s[w];
        up = fmaxf(up, up_s[w]);
    }
    // q is made of dloss over the largest |dloss|: equal gradients, as of a mean
    // loss, then put no rounding of their own on all of q.  For fp16 that is
    // scaled by 2^14: a weight of 2^-28 is still a normal number.
    const bool scaled = p.backward && up > 0.f && up < INFINITY;
    const float top = scaled ? up : 1.f;
    const float scale = scaled && std::is_same<T, __half>::value ? 0x1p14f : 1.f;
    if (blockIdx.x == 0 && tid == 0) {
        *p.count = all;
        if (p.backward) *p.unscale = top / scale;
    }
    const int64_t plane = p.row_cap * p.pitch;
    // the block's rows: a ballot of the targets gives every row its place
    const int64_t mine = row0 + lane;
    const bool there = lane < kLcePackRows && mine < p.rows;
    const int32_t t_lane = there ? __ldg(p.target + mine) : -1;
    const uint32_t live = __ballot_sync(0xffffffffu, there && lce_counts(p, t_lane));
    const int i = warp;
    const int64_t r = row0 + i;
    if (r < p.rows) {
        const int32_t t = __shfl_sync(0xffffffffu, t_lane, i);
        const T *xr = x + r * p.D;
        if (!((live >> i) & 1u)) {
            if (p.backward) {
                for (int64_t d = lane; d < p.D; d += 32) dx[r * p.D + d] = T(0.f);
            } else if (lane == 0) {
                const float v = t < 0 ? 0.f : __int_as_float(0x7fc00000);
                p.loss[r] = v;
                p.lse_out[r] = v;
            }
        } else {
            const int64_t at = before + __popc(live & ((1u << i) - 1u));
            O *o = out + at * p.pitch;
            if (lane == 0) {
                p.row_of[at] = (int)r;
                p.row_target[at] = t;
                if (p.backward) {
                    const bool in = t < p.V;
                    p.row_lse[at] = in ? __ldg(p.lse + r) : __int_as_float(0x7fc00000);
                    p.row_up[at] = __ldg(p.dloss + r) / top * scale;
                }
            }
            constexpr int V = Traits<T>::kVec;
            if (sizeof(T) == 2 && p.D % V == 0 && reinterpret_cast<uintptr_t>(x) % 16 == 0) {
#pragma unroll 4
                for (int64_t c = lane; c < p.D / V; c += 32)
                    reinterpret_cast<uint4 *>(o)[c] = ld_cached16(xr + c * V);
            } else {
#pragma unroll 8
                for (int64_t d = lane; d < p.D; d += 32)
                    LceSplit<T>::put(o + d, plane, __ldg(xr + d));
            }
            for (int64_t d = p.D + lane; d < p.pitch; d += 32)
                LceSplit<T>::put(o + d, plane, T(0.f));
        }
    }
    // The product q^T x goes over whole steps of K: the rows up to the next are 0.
    // (Others past the last only meet outputs that are not written.)
    if (p.backward && blockIdx.x == gridDim.x - 1) {
        const int64_t end = ((int64_t)all + kLceK - 1) / kLceK * kLceK;
        const int64_t vectors = (end - all) * p.pitch / 8;
#pragma unroll
        for (int k = 0; k < LceSplit<T>::kPlanes; ++k)
            for (int64_t c = tid; c < vectors; c += 256)
                reinterpret_cast<uint4 *>(out + k * plane + all * p.pitch)[c] =
                    make_uint4(0u, 0u, 0u, 0u);
    }
}

// W in planes with rows of `pitch` elements (fp32, and rows that TMA cannot
// address).
template <typename T>
__global__ void __launch_bounds__(256)
lce_pack_weight(typename LceSplit<T>::O *out, const T *w, int64_t V, int64_t D, int64_t pitch) {
    pdl_begin();
    const int64_t n = V * pitch;
    const int lane = threadIdx.x & 31;
    for (int64_t v = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5); v < V; v += (int64_t)gridDim.x * 8) {
#pragma unroll 8
        for (int64_t d = lane; d < D; d += 32)
            LceSplit<T>::put(out + v * pitch + d, n, __ldg(w + v * D + d));
        for (int64_t d = D + lane; d < pitch; d += 32)
            LceSplit<T>::put(out + v * pitch + d, n, T(0.f));
    }
}

// ----------------------------------------------------------------------------
// The products.
// ----------------------------------------------------------------------------
// A tile of a launch.
struct LceTile {
    int job;        // kLceGrads: 0 dx, 1 dW
    int64_t m, n;   // tile indexes
    int64_t k0, nk; // first step along K and steps (of each product of planes)
    int64_t split;  // dx: which cut of K
};

// The tiles of one pair of blocks, in order.  Products of logits: pair c takes
// tiles c, c + pairs, ..., M fastest, so that the tiles in flight share the rows
// of W (x stays in L2).  Gradients: first the dx tiles the same way, N fastest
// (they share the rows of q); a dx tile is several dW tiles long, and pairs with
// one more of them take the fewer dW tiles, so that all end together.
template <int EPI>
struct LceWalk {
    int64_t mt, nt, pair, pairs, dx_tiles, dw_tiles, dx_mine, dw_mine, dw_first, dw_step, nk_m, nk_v;
    int64_t i, fast, slow, fast_n, step_f, step_s;  // the next tile, and from it to the one after
    __device__ __forceinline__ LceWalk(const LceArgs &g, int64_t count) {
        pair = blockIdx.x >> 1;
        pairs = gridDim.x >> 1;
        mt = (count + kLceM - 1) / kLceM;
        if (EPI != kLceGrads) {
            nt = (g.vc + kLceN - 1) / kLceN;
            nk_v = (g.D + kLceK - 1) / kLceK;
            dx_tiles = mt * nt;
            dw_mine = 0;
        } else {
            nt = (g.D + kLceN - 1) / kLceN;
            nk_v = (g.vc + kLceK - 1) / kLceK;
            nk_m = (count + kLceK - 1) / kLceK;
            dx_tiles = mt * nt * g.splits;
            dw_tiles = g.with_dw ? (g.vc + kLceM - 1) / kLceM * nt : 0;
        }
        const int64_t most = dx_tiles / pairs, longer = dx_tiles - most * pairs;
        dx_mine = most + (pair < longer ? 1 : 0);
        if (EPI == kLceGrads) {
            const int64_t lx = g.split_k, lw = nk_m < 1 ? 1 : nk_m;
            // dW tiles of a pair with one more dx tile
            int64_t fewer =
                ((dx_tiles * lx + dw_tiles * lw) / pairs - (most + 1) * lx + lw / 2) / lw;
            fewer = min(max(fewer, (int64_t)0), dw_tiles / pairs);
            if (pair < longer) {
                dw_first = pair;
                dw_step = longer;
                dw_mine = fewer;
            } else {
                dw_first = longer * fewer + pair - longer;
                dw_step = pairs - longer;
                dw_mine = dw_first < dw_tiles ? (dw_tiles - dw_first + dw_step - 1) / dw_step : 0;
            }
        }
    }
    __device__ __forceinline__ int64_t tiles() const { return dx_mine + dw_mine; }
    // Divides once per run of tiles, not per tile: the loader's tiles are as short
    // as 16 steps, and four divisions in each cost it a third of its time.
    __device__ __forceinline__ void start(int64_t first, int64_t step, int64_t n) {
        fast_n = n < 1 ? 1 : n;
        slow = first / fast_n;
        fast = first - slow * fast_n;
        step_s = step / fast_n;
        step_f = step - step_s * fast_n;
    }
    __device__ __forceinline__ void begin() {
        i = 0;
        if (EPI != kLceGrads)
            start(pair, pairs, mt);
        else if (dx_mine > 0)
            start(pair, pairs, nt);
        else
            start(dw_first, dw_step, nt);
    }
    __device__ __forceinline__ LceTile next(const LceArgs &g) {
        LceTile t;
        t.job = 0;
        t.k0 = t.split = 0;
        if (EPI != kLceGrads) {
            t.n = slow;
            t.m = fast;
            t.nk = nk_v;
        } else if (i < dx_mine) {
            t.n = fast;
            t.split = 0;
            t.m = slow;
            while (t.m >= mt) {  // (at most kLceMaxCuts times)
                t.m -= mt;
                ++t.split;
            }
            t.k0 = t.split * g.split_k;
            t.nk = max(min(g.split_k, nk_v - t.k0), (int64_t)0);
        } else {
            t.job = 1;
            t.m = slow;
            t.n = fast;
            t.nk = nk_m;
        }
        ++i;
        if (EPI == kLceGrads && i == dx_mine) {
            start(dw_first, dw_step, nt);
        } else {
            fast += step_f;
            slow += step_s;
            if (fast >= fast_n) {
                fast -= fast_n;
                ++slow;
            }
        }
        return t;
    }
};

template <typename T>
__device__ __forceinline__ T lce_round(float v);
template <>
__device__ __forceinline__ float lce_round<float>(float v) { return v; }
template <>
__device__ __forceinline__ __half lce_round<__half>(float v) { return __float2half_rn(v); }
template <>
__device__ __forceinline__ __nv_bfloat16 lce_round<__nv_bfloat16>(float v) {
    return __float2bfloat16_rn(v);
}

// 32 values to consecutive elements, the first n of them: whole 32-byte sectors
// where they are aligned (a lane's row lies far from the next lane's, and halves
// of a sector cost as much as all of it).
template <typename T>
__device__ __forceinline__ void lce_store32(T *p, const float (&f)[32], int n) {
    constexpr int V = Traits<T>::kVec;
    if (n >= 32 && reinterpret_cast<uintptr_t>(p) % 32 == 0) {
#pragma unroll
        for (int c = 0; c < 32; c += 2 * V) {
            float e0[V], e1[V];
#pragma unroll
            for (int i = 0; i < V; ++i) {
                e0[i] = f[c + i];
                e1[i] = f[c + V + i];
            }
            const uint4 a = Traits<T>::pack(e0), b = Traits<T>::pack(e1);
            asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p + c),
                         "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b.x), "r"(b.y), "r"(b.z),
                         "r"(b.w)
                         : "memory");
        }
    } else if (n >= 32 && reinterpret_cast<uintptr_t>(p) % 16 == 0) {
#pragma unroll
        for (int c = 0; c < 32; c += V) {
            float e[V];
#pragma unroll
            for (int i = 0; i < V; ++i) e[i] = f[c + i];
            *reinterpret_cast<uint4 *>(p + c) = Traits<T>::pack(e);
        }
    } else {
#pragma unroll
        for (int c = 0; c < 32; ++c)
            if (c < n) p[c] = lce_round<T>(f[c]);
    }
}

// A warp's 32 rows of N values to rows that start anywhere: turned in shared
// memory so that 16 lanes write neighbouring columns (a lane that writes its own
// row touches a sector per element: the gradients' product of [1001,333] fp32 by
// 10007 took 98 us, 74 turned).  out: the lane's row, or NULL.
template <typename T, int N>
__device__ __forceinline__ void lce_store_turned(float *turn, T *out, const float (&f)[N], float un,
                                                 int width) {
    const int lane = threadIdx.x & 31, col = lane & (kLceTurn - 1);
#pragma unroll
    for (int c = 0; c < N; c += kLceTurn) {
        if (c >= width) break;
        __syncwarp();
#pragma unroll
        for (int e = 0; e < kLceTurn; ++e) turn[lane * (kLceTurn + 1) + e] = f[c + e] * un;
        __syncwarp();
#pragma unroll 4
        for (int r = lane / kLceTurn; r < 32; r += 32 / kLceTurn) {
            T *row = reinterpret_cast<T *>(
                __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(out), r));
            if (row && c + col < width)
                row[c + col] = lce_round<T>(turn[r * (kLceTurn + 1) + col]);
        }
    }
}

// T: storage type of the call.  Maps: a0, b0 of the only product or of dx; a1,
// b1 of dW; in boxes of 64 by 128 rows where the operand lies along K, else of
// 64 by 64.
// PARTS: sums along K of more than lce_cut steps are taken in parts.
template <int EPI, typename T, bool PARTS>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kLceThreads, 1)
lce_product(const __grid_constant__ CUtensorMap a0, const __grid_constant__ CUtensorMap b0,
            const __grid_constant__ CUtensorMap a1, const __grid_constant__ CUtensorMap b1,
            const LceArgs g) {
    // what needs nothing of the kernels before runs while they end
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    extern __shared__ __align__(1024) uint8_t lce_smem[];
    __shared__ __align__(8) uint64_t bars[2 * kLceStages + 5];
    __shared__ uint32_t tmem_at;
    __shared__ int abort_s;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = (int)cluster_rank();
    const uint32_t base = (smem_addr(lce_smem) + 1023u) & ~1023u;
    const uint32_t bar0 = smem_addr(bars);
    // operands of both blocks have arrived (the first block's counts)
    auto full = [&](int s) { return bar0 + 8u * s; };
    auto empty = [&](int s) { return bar0 + 8u * (kLceStages + s); };
    auto acc_full = [&](int b) { return bar0 + 8u * (2 * kLceStages + b); };
    // both blocks' accumulators have been read (the first block's counts)
    auto acc_empty = [&](int b) { return bar0 + 8u * (2 * kLceStages + 2 + b); };
    const uint32_t drained = bar0 + 8u * (2 * kLceStages + 4);
    if (threadIdx.x == 0) {
        for (int s = 0; s < kLceStages; ++s) {
            mbar_init(full(s), 1);
            mbar_init(empty(s), 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(acc_full(b), 1);
            mbar_init(acc_empty(b), 16);
        }
        mbar_init(drained, 1);
        mbar_init_fence();
        abort_s = 0;
    }
    if (warp == 1) tmem_alloc(smem_addr(&tmem_at), 512);
    tc_fence_before();
    __syncthreads();
    cluster_sync();
    tc_fence_after();
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const uint32_t tmem = tmem_at;
    volatile int *abort = &abort_s;
    const int64_t count = *g.count;
    LceWalk<EPI> walk(g, count);
    walk.begin();
    const int64_t tiles = walk.tiles();
    constexpr int kBufs = 2;  // accumulators in turn
    constexpr int kSegs = sizeof(T) == 4 ? 6 : 1;  // products of planes
    constexpr int kCut = lce_cut<EPI, T>();
    auto part_of = [](int64_t left) { return PARTS && left > kCut ? (int64_t)kCut : left; };

    if (warp == 0) {
        // ---- loader ----
        if (lane == 0) {
            tma_prefetch_map(&a0);
            tma_prefetch_map(&b0);
            const uint32_t first = cluster_addr(bar0, 0) - bar0;  // to the first block's barriers
            int s = 0;
            uint32_t phase = 0;
            int64_t issued = 0;
            bool ok = true;
            for (int64_t i = 0; i < tiles && ok; ++i) {
                const LceTile t = walk.next(g);
                const CUtensorMap *ma = t.job ? &a1 : &a0, *mb = t.job ? &b1 : &b0;
                const bool a_mn = t.job == 1, b_mn = EPI == kLceGrads;
                const int m0 = (int)(t.m * kLceM) + rank * kLceHalf;
                const int n0 = (int)(t.n * kLceN) + rank * kLceHalf;
                for (int64_t kp = 0; kp < t.nk && ok; kp += kCut) {
                    const int len = (int)part_of(t.nk - kp);
                    for (int j = 0, seg = 0, k0 = (int)(t.k0 + kp) * kLceK; seg < kSegs;) {
                        const int2 pl = kSegs > 1 ? lce_planes(seg) : make_int2(0, 0);
                        ok = mbar_wait(empty(s), phase ^ 1u, abort);
                        if (!ok) break;
                        if (rank == 0) mbar_expect(full(s), 2 * kLceStage);
                        const uint32_t at = base + s * kLceStage;
                        const uint32_t here = full(s) + first;
                        // along K: 128 rows at once; along M or N: 64 and 64 columns
                        if (a_mn) {
                            tma_load_3d(at, ma, here, m0, k0, pl.x);
                            tma_load_3d(at + kLceBox, ma, here, m0 + 64, k0, pl.x);
                        } else {
                            tma_load_3d(at, ma, here, k0, m0, pl.x);
                        }
                        if (b_mn) {
                            tma_load_3d(at + 2 * kLceBox, mb, here, n0, k0, pl.y);
                            tma_load_3d(at + 3 * kLceBox, mb, here, n0 + 64, k0, pl.y);
                        } else {
                            tma_load_3d(at + 2 * kLceBox, mb, here, k0, n0, pl.y);
                        }
                        ++issued;
                        k0 += kLceK;
                        if (++j == len) {  // the next product of planes
                            j = 0;
                            ++seg;
                            k0 = (int)(t.k0 + kp) * kLceK;
                        }
                        if (++s == kLceStages) {
                            s = 0;
                            phase ^= 1u;
                        }
                    }
                    if (!PARTS) break;
                }
            }
            // no copy may be in flight when the block ends: the last ones have been
            // multiplied, or, after a wait that ran out, have arrived
            for (int64_t j = issued > kLceStages ? issued - kLceStages : 0; j < issued; ++j) {
                const uint32_t p = (uint32_t)((j / kLceStages) & 1);
                if (ok || rank != 0)
                    mbar_wait(empty((int)(j % kLceStages)), p, nullptr);
                else
                    mbar_wait(full((int)(j % kLceStages)), p, nullptr);
            }
        }
    } else if (warp == 1) {
        // ---- issuer, in the first block ----
        if (lane == 0 && rank == 0) {
            int s = 0, buf = 0;
            uint32_t phase = 0, acc_phase = 0;
            bool ok = true;
            for (int64_t i = 0; i < tiles && ok; ++i) {
                const LceTile t = walk.next(g);
                if (t.nk == 0) continue;
                const bool a_mn = t.job == 1, b_mn = EPI == kLceGrads;
                const uint32_t idesc = tc_idesc(g.bf16 != 0, a_mn, b_mn, kLceM, kLceN);
                for (int64_t kp = 0; kp < t.nk && ok; kp += kCut) {
                    const int len = (int)part_of(t.nk - kp) * kSegs;
                    ok = mbar_wait(acc_empty(buf), acc_phase ^ 1u, abort);
                    if (!ok) break;
                    tc_fence_after();
                    const uint32_t d = tmem + buf * kLceN;
                    for (int k = 0; k < len; ++k) {
                        ok = mbar_wait(full(s), phase, abort);
                        if (!ok) break;
                        tc_fence_after();
                        const uint32_t at = base + s * kLceStage;
                        const uint64_t da = tc_desc(at, kLceBox);
                        const uint64_t db = tc_desc(at + 2 * kLceBox, kLceBox);
                        // 16 elements further along K: 32 bytes of a row, or 16 rows
                        const uint64_t sa = a_mn ? 16 * 128 / 16 : 32 / 16;
                        const uint64_t sb = b_mn ? 16 * 128 / 16 : 32 / 16;
#pragma unroll
                        for (int kk = 0; kk < kLceK / 16; ++kk)
                            tc_mma(d, da + kk * sa, db + kk * sb, idesc, k > 0 || kk > 0);
                        tc_commit(empty(s));
                        if (++s == kLceStages) {
                            s = 0;
                            phase ^= 1u;
                        }
                    }
                    if (!ok) break;
                    tc_commit(acc_full(buf));
                    if (++buf == kBufs) {
                        buf = 0;
                        acc_phase ^= 1u;
                    }
                    if (!PARTS) break;
                }
            }
            tc_commit_own(drained);
            mbar_wait(drained, 0, nullptr);
        }
    } else {
        // ---- accumulators ----
        // a warp reads the 32 rows that its number allows, and half of the columns
        const int quarter = warp & 3;
        float *turn = reinterpret_cast<float *>(lce_smem + (base - smem_addr(lce_smem)) +
                                                kLceStages * kLceStage) +
                      (warp - 2) * kLceTurnFloats;
        const int half = (warp - 2) >> 2;
        const int row_in = rank * kLceHalf + 32 * quarter + lane;
        int buf = 0;
        uint32_t acc_phase = 0;
        bool ok = true;
        for (int64_t i = 0; i < tiles; ++i) {
            const LceTile t = walk.next(g);
            const uint32_t mine =
                tmem + ((uint32_t)(32 * quarter) << 16) + half * (kLceN / 2);
            auto arrived = [&]() {  // the whole warp agrees on whether the product came
                if (ok) ok = __all_sync(0xffffffffu, mbar_wait(acc_full(buf), acc_phase, abort));
                tc_fence_after();
            };
            auto release = [&]() {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_cluster(cluster_addr(acc_empty(buf), 0));
                if (++buf == kBufs) {
                    buf = 0;
                    acc_phase ^= 1u;
                }
            };
            const int64_t row = t.m * kLceM + row_in;
            // The row's half of the tile, summed over its parts along K (rounding to
            // nearest).  An accumulator is free once it is read.
            constexpr int kCols = kLceN / 2;
            float f[kCols];
            if (t.nk > 0) {
                arrived();
                const uint32_t src = mine + buf * kLceN;
#pragma unroll
                for (int c = 0; c < kCols; c += 32) tmem_load32(f, c, src + c);
                tmem_wait(f);
                release();
            } else {
#pragma unroll
                for (int e = 0; e < kCols; ++e) f[e] = 0.f;
            }
            for (int64_t left = PARTS ? t.nk - kCut : 0; left > 0; left -= kCut) {
                arrived();
                const uint32_t src = mine + buf * kLceN;
#pragma unroll
                for (int c = 0; c < kCols; c += 16) {
                    float part[16];
                    tmem_load16(part, src + c);
                    tmem_wait16(part);
                    if (c + 16 == kCols) release();
#pragma unroll
                    for (int e = 0; e < 16; e += 2) {
                        const float2 v = add2(make_float2(f[c + e], f[c + e + 1]),
                                              make_float2(part[e], part[e + 1]));
                        f[c + e] = v.x;
                        f[c + e + 1] = v.y;
                    }
                }
            }
            // what a tile whose product did not come is multiplied with
            const float gone = ok ? 1.f : __int_as_float(0x7fc00000);
            if constexpr (EPI == kLceStats) {
                const int64_t n0 = t.n * kLceN + half * kCols;
                const int width = (int)min((int64_t)kCols, g.V - n0);
                const int hit = row < count ? g.target[row] - (int)n0 : -1;
                if (width < kCols) {
#pragma unroll
                    for (int e = 0; e < kCols; ++e)
                        if (e >= width) f[e] = -INFINITY;
                }
                if ((unsigned)hit < (unsigned)kCols) {
                    float v = 0.f;
#pragma unroll
                    for (int e = 0; e < kCols; ++e)
                        if (hit == e) v = f[e];
                    g.row_hit[row] = v * gone;
                }
                // four chains each
                float top[4];
                float2 s2[4];
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    top[c] = fmaxf(f[2 * c], f[2 * c + 1]);
                    s2[c] = f2(0.f);
                }
#pragma unroll
                for (int e = 8; e < kCols; e += 8)
#pragma unroll
                    for (int c = 0; c < 4; ++c)
                        top[c] = fmax3(top[c], f[e + 2 * c], f[e + 2 * c + 1]);
                const float m = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])) * kLog2e;
                const float use = m == -INFINITY ? 0.f : m;
#pragma unroll
                for (int e = 0; e < kCols; e += 2) {
                    float2 z = fma2(make_float2(f[e], f[e + 1]), f2(kLog2e), f2(-use));
                    z.x = fast_exp2(z.x);
                    z.y = fast_exp2(z.y);
                    s2[e / 2 % 4] = add2(s2[e / 2 % 4], z);
                }
                const float2 t2 = add2(add2(s2[0], s2[1]), add2(s2[2], s2[3]));
                const float sum = (t2.x + t2.y) * gone;
                if (row < count) g.part[(2 * t.n + half) * g.row_cap + row] = make_float2(m, sum);
            } else if constexpr (EPI == kLceQ) {
                using O = typename LceSplit<T>::O;
                const int64_t n0 = t.n * kLceN + half * kCols;  // within the piece
                const int width = (int)min((int64_t)kCols, g.V - g.v0 - n0);
                const bool live = row < count;
                const float l = live ? g.row_lse[row] : 0.f;
                const float up = live ? g.row_up[row] * gone : 0.f;
                const int hit = live ? g.target[row] - (int)(g.v0 + n0) : -1;
                O *q = static_cast<O *>(g.q) + row * g.q_pitch + n0;
                const int64_t plane = g.row_cap * g.q_pitch;
#pragma unroll
                for (int e = 0; e < kCols; e += 2) {
                    // the difference first: where a row's weight is on its target, p - 1
                    // would carry the rounding of lse log2 e
                    const float2 z =
                        mul2(add2(make_float2(f[e], f[e + 1]), f2(-l)), f2(kLog2e));
                    f[e] = fast_exp2(z.x);
                    f[e + 1] = fast_exp2(z.y);
                }
                if ((unsigned)hit < (unsigned)kCols) {
#pragma unroll
                    for (int e = 0; e < kCols; ++e)
                        if (hit == e) f[e] -= 1.f;
                }
#pragma unroll
                for (int e = 0; e < kCols; ++e) f[e] *= up;
                if (!live || width < kCols) {
#pragma unroll
                    for (int e = 0; e < kCols; ++e)
                        if (!live || e >= width) f[e] = 0.f;
                }
#pragma unroll
                for (int c = 0; c < kCols; c += 32) {
                    float p0[32];
#pragma unroll
                    for (int e = 0; e < 32; ++e) p0[e] = f[c + e];
                    if constexpr (LceSplit<T>::kPlanes == 1) {
                        lce_store32<O>(q + c, p0, 32);
                    } else {
                        float p1[32], p2[32];
#pragma unroll
                        for (int e = 0; e < 32; ++e) {
                            O o[3];
                            LceSplit<float>::parts(p0[e], o);
                            p0[e] = __bfloat162float(o[0]);
                            p1[e] = __bfloat162float(o[1]);
                            p2[e] = __bfloat162float(o[2]);
                        }
                        lce_store32<O>(q + c, p0, 32);
                        lce_store32<O>(q + plane + c, p1, 32);
                        lce_store32<O>(q + 2 * plane + c, p2, 32);
                    }
                }
            } else {
                const float un = *g.unscale * gone;
                const int64_t n0 = t.n * kLceN + half * kCols;
                const int width = (int)min((int64_t)kCols, g.D - n0);
                const bool live = t.job ? row < g.vc : row < count;
                T *out = nullptr;
                if (live)
                    out = t.job ? static_cast<T *>(g.dw) + (g.v0 + row) * g.D + n0
                                : static_cast<T *>(g.dx) + (int64_t)g.row_of[row] * g.D + n0;
                if (!g.aligned && (t.job || (g.first && g.last && g.splits == 1))) {
                    lce_store_turned<T>(turn, out, f, un, width);
                    continue;
                }
                const bool add = !t.job && !g.first, keep = !t.job && !(g.last && g.splits == 1);
                float *sums = g.dx_sum + (t.split * g.row_cap + row) * g.sum_pitch + n0;
                if (live) {
#pragma unroll
                    for (int c = 0; c < kCols; c += 32) {
                        const int n = width - c;
                        if (n <= 0) continue;
                        float v[32];
#pragma unroll
                        for (int e = 0; e < 32; ++e) v[e] = f[c + e] * un;
                        if (add) {  // (the rows of the sums reach to a multiple of 8)
#pragma unroll
                            for (int e = 0; e < 32; e += 4) {
                                if (e >= n) continue;
                                const float4 q =
                                    *reinterpret_cast<const float4 *>(sums + c + e);
                                v[e] += q.x;
                                v[e + 1] += q.y;
                                v[e + 2] += q.z;
                                v[e + 3] += q.w;
                            }
                        }
                        if (keep)
                            lce_store32<float>(sums + c, v, (n + 7) & ~7);
                        else
                            lce_store32<T>(out + c, v, n);
                    }
                }
            }
        }
    }
    // (neither block ends while the other may still reach into it)
    tc_fence_before();
    __syncthreads();
    cluster_sync();
    if (warp == 1) {
        tc_fence_after();
        tmem_free(tmem, 512);
    }
}

// dx of the rows that count, where the sum over the vocabulary was cut.
template <typename T>
__global__ void __launch_bounds__(256) lce_join_dx(const LceArgs g) {
    pdl_begin();
    const int64_t step = g.row_cap * g.sum_pitch;
    for (int64_t r = blockIdx.x; r < *g.count; r += gridDim.x) {
        const float *src = g.dx_sum + r * g.sum_pitch;
        T *dst = static_cast<T *>(g.dx) + (int64_t)g.row_of[r] * g.D;
        for (int64_t d = threadIdx.x; d < g.D; d += 256) {
            float v = __ldcg(src + d);
#pragma unroll 8
            for (int64_t s = 1; s < g.splits; ++s) v += __ldcg(src + s * step + d);
            dst[d] = lce_round<T>(v);
        }
    }
}

// lse and loss of the rows that count, from the parts' (largest, sum): 32 rows
// per block, each by 32 threads that take every 32nd part, eight at a time; the
// threads' pairs are joined in order.
constexpr int kLceJoin = 32;
static __global__ void __launch_bounds__(32 * kLceJoin)
lce_join(float *loss, float *lse, const LceArgs g, int64_t parts) {
    pdl_begin();
    __shared__ float m_s[kLceJoin][33], s_s[kLceJoin][33];
    const int r_in = threadIdx.x & 31, part = threadIdx.x >> 5;
    const int64_t count = *g.count;
    for (int64_t r0 = (int64_t)blockIdx.x * 32; r0 < count; r0 += (int64_t)gridDim.x * 32) {
        const int64_t row = r0 + r_in;
        float m = -INFINITY, s = 0.f;
        if (row < count) {
            for (int64_t t = part; t < parts; t += 8 * kLceJoin) {
                float2 v[8];
#pragma unroll
                for (int u = 0; u < 8; ++u) {
                    const int64_t k = t + (int64_t)u * kLceJoin;
                    v[u] = k < parts ? __ldcg(g.part + k * g.row_cap + row)
                                     : make_float2(-INFINITY, 0.f);
                }
                float top = m;
#pragma unroll
                for (int u = 0; u < 8; ++u) top = fmaxf(top, v[u].x);
                const float use = top == -INFINITY ? 0.f : top;
                s = m == -INFINITY ? s : s * exp2f(m - use);
#pragma unroll
                for (int u = 0; u < 8; ++u)
                    s += v[u].x == -INFINITY ? v[u].y : v[u].y * exp2f(v[u].x - use);
                m = top;
            }
        }
        m_s[part][r_in] = m;
        s_s[part][r_in] = s;
        __syncthreads();
        // warp w joins row w
        const int64_t mine = r0 + part;
        if (mine < count) {
            float mm = m_s[r_in][part], ss = s_s[r_in][part];
            float top = mm;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1)
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
            const float use = top == -INFINITY ? 0.f : top;
            ss = mm == -INFINITY ? ss : ss * exp2f(mm - use);
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
            if (r_in == 0) {
                const float l = (top + log2f(ss)) * 0.6931471805599453f;
                const int64_t at = g.row_of[mine];
                lse[at] = l;
                loss[at] = l - g.row_hit[mine];
            }
        }
        __syncthreads();
    }
}

}  // namespace lsr
