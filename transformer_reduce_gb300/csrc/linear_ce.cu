// linear_ce.cu -- launchers and instantiations of the cross entropy taken from
// hidden states and the vocabulary matrix.
#include <cstring>
#include <type_traits>

#include "dispatch.cuh"
#include "linear_ce.cuh"

namespace lsr {

// Bytes of q in the workspace that the pieces of the vocabulary are cut to, and
// the narrowest piece (dx is read and written once per piece: of a piece of
// 4096 entries that is a tenth of its products' time).
constexpr int64_t kLceQBytes = (int64_t)512 << 20;
constexpr int64_t kLceMinPiece = 4096;
// Fewest steps of K of a cut of dx, and most cuts.
constexpr int64_t kLceMinCut = 16;
constexpr int64_t kLceMaxCuts = 32;

// Where everything lies in the workspace.
struct LceLayout {
    int64_t row_cap, chunks, pitch, w_pitch, vc, pieces, q_pitch, splits, split_k;
    int planes;
    bool pack_w;
    size_t chunk_count, chunk_up, single, row_of, row_target, row_lse, row_up, row_hit, x, w, part,
        q, dx_sum, total;
};

static int64_t round_up(int64_t v, int64_t to) { return (v + to - 1) / to * to; }

static LceLayout lce_layout(bool backward, int64_t rows, int64_t D, int64_t V, size_t es) {
    LceLayout l = {};
    l.planes = es == 4 ? 3 : 1;
    l.row_cap = round_up(rows < 1 ? 1 : rows, kLceM);
    l.chunks = rows > kLceCountRows ? ceil_div(rows, kLceChunk) : 0;
    l.pitch = round_up(D, 8);  // TMA wants rows of whole 16 bytes
    l.pack_w = es == 4 || D % 8 != 0;
    l.w_pitch = l.pitch;
    l.vc = V;
    l.pieces = 1;
    if (backward) {
        int64_t most = kLceQBytes / (2 * l.planes * l.row_cap) / kLceN * kLceN;
        if (most < kLceMinPiece) most = kLceMinPiece;
        if (most < V) {
            l.pieces = ceil_div(V, most);
            l.vc = round_up(ceil_div(V, l.pieces), kLceN);
            l.pieces = ceil_div(V, l.vc);
        }
        l.q_pitch = round_up(l.vc, kLceN);
        // dx is cut along the vocabulary where its few tiles would be longer than
        // half of a pair's share of the gradients' work
        const int64_t nt = ceil_div(D, kLceN), mt = l.row_cap / kLceM;
        const int64_t nk = ceil_div(l.vc, kLceK), dw = ceil_div(l.vc, kLceM) * nt;
        const int64_t work = mt * nt * nk + dw * (l.row_cap / kLceK);
        int64_t k = work / kLceSms;
        if (k < kLceMinCut) k = kLceMinCut;
        if (k < ceil_div(nk, kLceMaxCuts)) k = ceil_div(nk, kLceMaxCuts);
        l.splits = k < nk ? ceil_div(nk, k) : 1;
        l.split_k = ceil_div(nk, l.splits);
        l.splits = ceil_div(nk, l.split_k);
    }
    size_t at = 0;
    auto take = [&](int64_t bytes) {
        const size_t here = at;
        at += (size_t)round_up(bytes, 256);
        return here;
    };
    l.chunk_count = take(l.chunks * 4);
    l.chunk_up = take(l.chunks * 4);
    l.single = take(8);
    l.row_of = take(l.row_cap * 4);
    l.row_target = take(l.row_cap * 4);
    l.x = take(l.planes * l.row_cap * l.pitch * 2);
    if (l.pack_w) l.w = take(l.planes * V * l.w_pitch * 2);
    if (backward) {
        l.row_lse = take(l.row_cap * 4);
        l.row_up = take(l.row_cap * 4);
        l.q = take(l.planes * l.row_cap * l.q_pitch * 2);
        if (l.pieces > 1 || l.splits > 1) l.dx_sum = take(l.splits * l.row_cap * round_up(D, 8) * 4);
    } else {
        l.row_hit = take(l.row_cap * 4);
        l.part = take(2 * ceil_div(V, kLceN) * l.row_cap * 8);
    }
    l.total = at;
    return l;
}

size_t linear_ce_workspace(bool backward, int64_t rows, int64_t D, int64_t V, size_t es) {
    return lce_layout(backward, rows, D, V, es).total;
}

// Map of [planes][rows][cols] 16-bit elements, rows `pitch` apart, in boxes of
// 64 columns by 128 rows for an operand that lies along K in memory, by 64 for
// others; elements beyond the rows or columns read as 0.
static cudaError_t lce_map(CUtensorMap *map, bool along_k, const void *base, bool bf16, int64_t cols,
                           int64_t rows, int64_t planes, int64_t pitch, int64_t plane) {
    using Encode = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *,
                                const cuuint64_t *, const cuuint64_t *, const cuuint32_t *,
                                const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                                CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
    static std::atomic<void *> known;
    void *fn = known.load(std::memory_order_acquire);
    if (!fn) {
        cudaDriverEntryPointQueryResult found;
        const cudaError_t e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000,
                                                               cudaEnableDefault, &found);
        if (e != cudaSuccess) return e;
        if (found != cudaDriverEntryPointSuccess || !fn) return cudaErrorNotSupported;
        known.store(fn, std::memory_order_release);
    }
    const cuuint64_t dims[3] = {(cuuint64_t)cols, (cuuint64_t)rows, (cuuint64_t)planes};
    const cuuint64_t strides[2] = {(cuuint64_t)pitch * 2, (cuuint64_t)plane * 2};
    const cuuint32_t box[3] = {64, along_k ? 128u : 64u, 1}, step[3] = {1, 1, 1};
    const CUresult r = reinterpret_cast<Encode>(fn)(
        map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3,
        const_cast<void *>(base), dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
        CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

template <int EPI, typename T, bool PARTS>
cudaError_t lce_launch_parts(const CUtensorMap &a0, const CUtensorMap &b0, const CUtensorMap &a1,
                       const CUtensorMap &b1, const LceArgs &g, cudaStream_t st) {
    constexpr auto K = lce_product<EPI, T, PARTS>;
    ensure_dynamic_smem<K>(kLceSmem);
    const int64_t mt = ceil_div(g.rows, kLceM), nt = ceil_div(g.D, kLceN);
    const int64_t tiles = EPI == kLceGrads
                              ? (mt * g.splits + (g.with_dw ? ceil_div(g.vc, kLceM) : 0)) * nt
                              : mt * ceil_div(g.vc, kLceN);
    if (tiles == 0) return cudaSuccess;
    const int64_t pairs = device_sm_count() / 2;
    return launch_pdl(K, dim3((unsigned)(2 * (tiles < pairs ? tiles : pairs))), dim3(kLceThreads),
                      kLceSmem, st, a0, b0, a1, b1, g);
}

// Hidden sizes of one part have kernels without the code that adds parts (with it
// the forward of [8192,1024] bf16 by 50257 took 401 us instead of 391).
template <int EPI, typename T>
cudaError_t lce_launch(const CUtensorMap &a0, const CUtensorMap &b0, const CUtensorMap &a1,
                       const CUtensorMap &b1, const LceArgs &g, cudaStream_t st) {
    if constexpr (EPI != kLceGrads && sizeof(T) == 2)
        if (ceil_div(g.D, kLceK) <= lce_cut<EPI, T>())
            return lce_launch_parts<EPI, T, false>(a0, b0, a1, b1, g, st);
    return lce_launch_parts<EPI, T, true>(a0, b0, a1, b1, g, st);
}

// Packs the rows that count and, where needed, W; fills what both directions
// share of the arguments.
template <typename T>
cudaError_t lce_prepare(LceArgs *g, const void **w_at, const LceLayout &l, bool backward,
                        uint8_t *ws, const T *x, const T *w, const int32_t *target,
                        const float *lse, const float *dloss, float *loss, float *lse_out, T *dx,
                        int64_t rows, int64_t D, int64_t V, cudaStream_t st) {
    using O = typename LceSplit<T>::O;
    LcePack p = {};
    p.rows = rows;
    p.D = D;
    p.V = V;
    p.row_cap = l.row_cap;
    p.pitch = l.pitch;
    p.backward = backward;
    p.target = target;
    p.lse = lse;
    p.dloss = dloss;
    p.chunk_count = l.chunks > 0 ? reinterpret_cast<int *>(ws + l.chunk_count) : nullptr;
    p.chunk_up = reinterpret_cast<float *>(ws + l.chunk_up);
    p.count = reinterpret_cast<int *>(ws + l.single);
    p.unscale = reinterpret_cast<float *>(ws + l.single + 4);
    p.row_of = reinterpret_cast<int *>(ws + l.row_of);
    p.row_target = reinterpret_cast<int *>(ws + l.row_target);
    p.row_lse = reinterpret_cast<float *>(ws + l.row_lse);
    p.row_up = reinterpret_cast<float *>(ws + l.row_up);
    p.loss = loss;
    p.lse_out = lse_out;
    cudaError_t e = cudaSuccess;
    if (l.chunks > 0)
        e = launch_pdl(lce_count, dim3((unsigned)l.chunks), dim3(256), 0, st, p);
    if (e != cudaSuccess) return e;
    const int64_t groups = ceil_div(rows, kLcePackRows);
    e = launch_pdl(lce_pack_rows<T>, dim3((unsigned)(groups < 1 ? 1 : groups)), dim3(256), 0, st,
                   reinterpret_cast<O *>(ws + l.x), x, dx, p);
    if (e != cudaSuccess) return e;
    *w_at = w;
    if (l.pack_w) {
        *w_at = ws + l.w;
        const int64_t blocks = ceil_div(V, 8);
        const int64_t most = (int64_t)device_sm_count() * 8;
        e = launch_pdl(lce_pack_weight<T>, dim3((unsigned)(blocks < most ? blocks : most)),
                       dim3(256), 0, st, reinterpret_cast<O *>(ws + l.w), w, V, D, l.w_pitch);
    }
    *g = LceArgs{};
    g->rows = rows;
    g->D = D;
    g->V = V;
    g->row_cap = l.row_cap;
    g->vc = V;
    g->q_pitch = l.q_pitch;
    g->bf16 = !std::is_same<T, __half>::value;
    g->first = g->last = 1;
    g->count = p.count;
    g->row_of = p.row_of;
    g->target = p.row_target;
    g->row_lse = p.row_lse;
    g->row_up = p.row_up;
    g->unscale = p.unscale;
    return e;
}

template <typename T>
cudaError_t launch_linear_ce_fw(float *loss, float *lse, const T *x, const T *w,
                                const int32_t *target, int64_t rows, int64_t D, int64_t V,
                                void *workspace, cudaStream_t st) {
    const LceLayout l = lce_layout(false, rows, D, V, sizeof(T));
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    LceArgs g;
    const void *wp;
    cudaError_t e = lce_prepare<T>(&g, &wp, l, false, ws, x, w, target, nullptr, nullptr, loss,
                                   lse, nullptr, rows, D, V, st);
    if (e != cudaSuccess) return e;
    g.row_hit = reinterpret_cast<float *>(ws + l.row_hit);
    g.part = reinterpret_cast<float2 *>(ws + l.part);
    CUtensorMap mx, mw;
    e = lce_map(&mx, true, ws + l.x, g.bf16, l.pitch, l.row_cap, l.planes, l.pitch,
                l.row_cap * l.pitch);
    if (e == cudaSuccess)
        e = lce_map(&mw, true, wp, g.bf16, l.w_pitch, V, l.planes, l.w_pitch, V * l.w_pitch);
    // (both 16-bit types share the kernel)
    using S = typename std::conditional<sizeof(T) == 4, float, __half>::type;
    if (e == cudaSuccess) e = lce_launch<kLceStats, S>(mx, mw, mx, mw, g, st);
    if (e != cudaSuccess) return e;
    const int64_t blocks = ceil_div(rows, 32), most = (int64_t)device_sm_count() * 8;
    return launch_pdl(lce_join, dim3((unsigned)(blocks < most ? blocks : most)),
                      dim3(32 * kLceJoin), 0, st, loss, lse, g, 2 * ceil_div(V, kLceN));
}

template <typename T>
cudaError_t launch_linear_ce_bw(T *dx, T *dw, const T *x, const T *w, const int32_t *target,
                                const float *lse, const float *dloss, int64_t rows, int64_t D,
                                int64_t V, void *workspace, cudaStream_t st) {
    const LceLayout l = lce_layout(true, rows, D, V, sizeof(T));
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    LceArgs g;
    const void *wp;
    cudaError_t e = lce_prepare<T>(&g, &wp, l, true, ws, x, w, target, lse, dloss, nullptr,
                                   nullptr, dx, rows, D, V, st);
    if (e != cudaSuccess) return e;
    g.q = ws + l.q;
    g.dx_sum = reinterpret_cast<float *>(ws + l.dx_sum);
    g.dx = dx;
    g.dw = dw;
    g.with_dw = dw != nullptr;
    g.splits = l.splits;
    g.split_k = l.split_k;
    g.sum_pitch = round_up(D, 8);
    g.aligned = D * sizeof(T) % 16 == 0 && reinterpret_cast<uintptr_t>(dx) % 16 == 0 &&
                reinterpret_cast<uintptr_t>(dw) % 16 == 0;
    CUtensorMap x_k, x_n, w_k, w_n, q_k, q_n;  // along K, and not
    const int64_t x_plane = l.row_cap * l.pitch, q_plane = l.row_cap * l.q_pitch;
    for (const bool k : {true, false}) {
        if (e == cudaSuccess)
            e = lce_map(k ? &x_k : &x_n, k, ws + l.x, g.bf16, l.pitch, l.row_cap, l.planes, l.pitch,
                        x_plane);
        if (e == cudaSuccess)
            e = lce_map(k ? &q_k : &q_n, k, ws + l.q, g.bf16, l.q_pitch, l.row_cap, l.planes,
                        l.q_pitch, q_plane);
    }
    for (int64_t i = 0; i < l.pieces && e == cudaSuccess; ++i) {
        g.v0 = i * l.vc;
        g.vc = V - g.v0 < l.vc ? V - g.v0 : l.vc;
        g.first = i == 0;
        g.last = i == l.pieces - 1;
        // rows of W from the piece on
        for (const bool k : {true, false})
            if (e == cudaSuccess)
                e = lce_map(k ? &w_k : &w_n, k,
                            static_cast<const uint8_t *>(wp) + g.v0 * l.w_pitch * 2, g.bf16,
                            l.w_pitch, V - g.v0, l.planes, l.w_pitch, V * l.w_pitch);
        if (e == cudaSuccess) e = lce_launch<kLceQ, T>(x_k, w_k, x_k, w_k, g, st);
        const int64_t nk = ceil_div(g.vc, kLceK);  // (the last piece may be shorter)
        g.split_k = ceil_div(nk, l.splits);
        if (e == cudaSuccess) e = lce_launch<kLceGrads, T>(q_k, w_n, q_n, x_n, g, st);
    }
    if (e != cudaSuccess || l.splits == 1 || rows == 0) return e;
    const int64_t most = (int64_t)device_sm_count() * 8;
    return launch_pdl(lce_join_dx<T>, dim3((unsigned)(rows < most ? rows : most)), dim3(256), 0,
                      st, g);
}

#define LSR_LCE_INSTANTIATE(T)                                                                  \
    template cudaError_t launch_linear_ce_fw<T>(float *, float *, const T *, const T *,         \
                                                const int32_t *, int64_t, int64_t, int64_t,     \
                                                void *, cudaStream_t);                          \
    template cudaError_t launch_linear_ce_bw<T>(T *, T *, const T *, const T *, const int32_t *, \
                                                const float *, const float *, int64_t, int64_t, \
                                                int64_t, void *, cudaStream_t);
LSR_LCE_INSTANTIATE(float)
LSR_LCE_INSTANTIATE(__half)
LSR_LCE_INSTANTIATE(__nv_bfloat16)
#undef LSR_LCE_INSTANTIATE

}  // namespace lsr
