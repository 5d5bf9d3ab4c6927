// C ABI of the operators around the mixer in a serving step (include/gdn.h): the
// norms between blocks, 8-bit projections, beam selection and state reordering.
// Argument checks and launches; the kernels are in the headers named below.
#include "gdn.h"

#include <algorithm>
#include <cstring>

#include "beam.cuh"
#include "block_norm.cuh"
#include "device.cuh"
#include "gemm_i8.cuh"
#include "host.cuh"
#include "quant.cuh"
#include "reorder.cuh"

namespace {

using namespace gdn::host;

// Lifts a kernel's shared-memory limit, once per device.
template <auto Kernel>
cudaError_t allow_smem(size_t bytes) {
    static bool done[64];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 64 && done[dev]) return cudaSuccess;
    e = cudaFuncSetAttribute(Kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
    if (e == cudaSuccess && dev < 64) done[dev] = true;
    return e;
}

struct Span {
    uintptr_t lo, hi;
};
Span span(const void* p, int64_t bytes) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(p);
    return {a, a + (p ? (uintptr_t)bytes : 0)};
}
bool overlap(const Span& a, const Span& b) { return a.lo < b.hi && b.lo < a.hi; }

bool float_dtype(int32_t d) { return d == GDN_BF16 || d == GDN_F32; }
int64_t elem(int32_t d) { return d == GDN_F32 ? 4 : d == GDN_BF16 ? 2 : 1; }

// Every kernel here is launched so that it may start while the kernel before it on the
// stream still runs (its set-up then costs no time of its own), and waits for that
// kernel's end before it reads or writes any tensor; so whoever waits for one of them to
// end has waited for all before it.  The one exception is a product's weights, behind
// the rows that the same call makes 8-bit (I8Args::w_ready).
struct Launch {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    Launch(unsigned grid, unsigned block, size_t smem, cudaStream_t st) {
        cfg.gridDim = dim3(grid, 1, 1);
        cfg.blockDim = dim3(block, 1, 1);
        cfg.dynamicSmemBytes = smem;
        cfg.stream = st;
        cfg.attrs = attr;
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        cfg.numAttrs = 1;
    }
    template <typename... P, typename... A>
    cudaError_t operator()(void (*kernel)(P...), const A&... args) {
        return cudaLaunchKernelEx(&cfg, kernel, P(args)...);
    }
    Launch& cluster(unsigned n) {
        if (n > 1) {
            attr[cfg.numAttrs].id = cudaLaunchAttributeClusterDimension;
            attr[cfg.numAttrs].val.clusterDim.x = n;
            attr[cfg.numAttrs].val.clusterDim.y = 1;
            attr[cfg.numAttrs++].val.clusterDim.z = 1;
        }
        return *this;
    }
};

// ---------------------------------------------------------------------------
// Block norms
// ---------------------------------------------------------------------------
template <typename TA, typename TR, bool kI8, int WARPS, int NV>
cudaError_t launch_norm(const gdn::bnorm::Args& a, int64_t T, cudaStream_t st) {
    return Launch((unsigned)T, WARPS * 32, 0, st)(gdn::bnorm::block_norm_kernel<TA, TR, kI8, WARPS, NV>, a);
}

template <typename TA, typename TR, bool kI8>
cudaError_t norm_by_size(const gdn::bnorm::Args& a, int64_t T, cudaStream_t st) {
    const int nv = a.D / 8;
    if (T <= 2 * sm_count()) {   // few rows: the lowest latency
        if (nv <= 512) return launch_norm<TA, TR, kI8, 16, 1>(a, T, st);
        if (nv <= 1024) return launch_norm<TA, TR, kI8, 16, 2>(a, T, st);
    } else {
        if (nv <= 64) return launch_norm<TA, TR, kI8, 2, 1>(a, T, st);
        if (nv <= 128) return launch_norm<TA, TR, kI8, 4, 1>(a, T, st);
        if (nv <= 192) return launch_norm<TA, TR, kI8, 6, 1>(a, T, st);
        if (nv <= 256) return launch_norm<TA, TR, kI8, 8, 1>(a, T, st);
        if (nv <= 384) return launch_norm<TA, TR, kI8, 4, 3>(a, T, st);
        if (nv <= 512) return launch_norm<TA, TR, kI8, 4, 4>(a, T, st);
        if (nv <= 1024) return launch_norm<TA, TR, kI8, 8, 4>(a, T, st);
    }
    return launch_norm<TA, TR, kI8, 16, 4>(a, T, st);
}

template <typename TA, typename TR>
cudaError_t norm_by_output(const gdn::bnorm::Args& a, int64_t T, cudaStream_t st) {
    return a.y_scale ? norm_by_size<TA, TR, true>(a, T, st) : norm_by_size<TA, TR, false>(a, T, st);
}

// ---------------------------------------------------------------------------
// 8-bit rows
// ---------------------------------------------------------------------------
template <typename T>
cudaError_t launch_quantize(const void* x, int64_t rows, int32_t cols, int8_t* q, float* scale, cudaStream_t st) {
    using namespace gdn::quant;
    const T* xt = static_cast<const T*>(x);
    const unsigned grid = (unsigned)rows;
    const int nv = cols / 8;
    // Few rows: a vector per thread, the lowest latency.  Many: the fewest warps that hold the
    // row, with several vectors each.  168 M elements in bf16, us (floor 78; blocks of 2 warps
    // and 5 vectors / 4 and 6 / 8 and 4): 1040 columns 170 / 211 / 293, 1536 116 / 152 / 207,
    // 2560 79 / 113 / 150, then - / 115 / 152 at 2576, 4096 - / 90 / 112, 6144 - / 80 / 94; from
    // fp32 (floor 130) 170 / 281 / 385 at 1040, 125 / 151 / 197 at 2560, - / 123 / 125 at 6144.
    // Up to 1024 columns every form takes 1.05 ns a row, the rate at which blocks start (1024:
    // 172 us, 512: 340), and the last one any length.
    if (nv <= 128) return Launch(grid, 128, 0, st)(quantize_rows_kernel<T, 4, 1>, xt, cols, q, scale);
    if (nv <= 320 && rows <= 2 * sm_count()) return Launch(grid, 320, 0, st)(quantize_rows_kernel<T, 10, 1>, xt, cols, q, scale);
    if (nv <= 320) return Launch(grid, 64, 0, st)(quantize_rows_kernel<T, 2, 5>, xt, cols, q, scale);
    if (nv <= 768) return Launch(grid, 128, 0, st)(quantize_rows_kernel<T, 4, 6>, xt, cols, q, scale);
    if (nv <= 1024) return Launch(grid, 256, 0, st)(quantize_rows_kernel<T, 8, 4>, xt, cols, q, scale);
    return Launch(grid, 512, 0, st)(quantize_rows_kernel<T, 16, 0>, xt, cols, q, scale);
}

gdn_status run_quantize(const void* x, int32_t x_dtype, int64_t rows, int32_t cols, int8_t* q, float* scale,
                        cudaStream_t st) {
    return cuda_status(x_dtype == GDN_BF16 ? launch_quantize<__nv_bfloat16>(x, rows, cols, q, scale, st)
                                           : launch_quantize<float>(x, rows, cols, q, scale, st));
}

// ---------------------------------------------------------------------------
// 8-bit projections
// ---------------------------------------------------------------------------
// 2-D map over a row-major [rows][K] int8 matrix: boxes of 128 (K) x box_rows,
// 128-byte swizzle; elements past K or rows read as zero.
bool i8_map(CUtensorMap* m, const void* base, int64_t rows, int K, int box_rows) {
    auto enc = tensor_map_encoder();
    if (!enc) return false;
    cuuint64_t dims[2] = {(cuuint64_t)K, (cuuint64_t)rows};
    cuuint64_t strides[1] = {(cuuint64_t)K};
    cuuint32_t box[2] = {(cuuint32_t)gdn::gemm::BK8, (cuuint32_t)box_rows};
    cuuint32_t estr[2] = {1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Clusters of `size` CTAs of a kernel that the device holds at once, asked of the
// runtime once per device and size.
template <auto Kernel>
int resident_clusters(int size, unsigned threads, size_t smem) {
    static int known[64][4];
    int dev = 0, n = 0;
    const int slot = size == 1 ? 0 : size == 2 ? 1 : size == 4 ? 2 : 3;
    if (cudaGetDevice(&dev) != cudaSuccess) return 1;
    if (dev < 64 && known[dev][slot]) return known[dev][slot];
    Launch l((unsigned)(sm_count() / size * size), threads, smem, nullptr);
    l.cfg.numAttrs = 0;
    l.cluster((unsigned)size);
    if (size == 1) n = sm_count();
    else if (cudaOccupancyMaxActiveClusters(&n, Kernel, &l.cfg) != cudaSuccess || n <= 0) {
        (void)cudaGetLastError();
        n = std::max(1, sm_count() / size);
    }
    if (dev < 64) known[dev][slot] = n;
    return n;
}

template <int BN>
cudaError_t launch_i8_pair(const void* x, const void* w, gdn::gemm::I8Args a, cudaStream_t st) {
    using S = gdn::gemm::Shape2<BN>;
    using Op = gdn::gemm::I8Op;
    constexpr auto kernel = gdn::gemm::linear_pair_kernel<BN, Op>;
    constexpr unsigned threads = 64 + 32 * Op::kEpiWarps;
    constexpr size_t smem = S::SMEM + 16 + Op::kEpiSmem;
    static_assert(smem <= 227 * 1024, "shared memory");
    CUtensorMap tm_x, tm_w;
    if (!i8_map(&tm_x, x, a.M, a.K, gdn::gemm::BM) || !i8_map(&tm_w, w, a.N, a.K, BN / 2)) return cudaErrorInvalidValue;
    a.n_blocks = (a.N + BN - 1) / BN;
    a.tiles = (a.M + 2 * gdn::gemm::BM - 1) / (2 * gdn::gemm::BM) * a.n_blocks;
    cudaError_t e = allow_smem<kernel>(smem);
    if (e != cudaSuccess) return e;
    const int pairs = (int)std::min<int64_t>(a.tiles, resident_clusters<kernel>(2, threads, smem));
    return Launch((unsigned)(2 * pairs), threads, smem, st)(kernel, tm_x, tm_w, a);   // (the kernel names its cluster size)
}

// Pair tile width for M > 128, over the widths that kind::i8 has at M = 256: fewest
// waves x (operand bytes of a k-block, 128 x (256 + BN) of a pair).  The bytes from L2 bound
// a k-block, not the MMA: 4096 x 16480 x 2560 at 256 (15 waves) 127 us, at 224 (16) 131, at 192
// (19) 142; the bf16 form's rule took 224.
// *cost: those bytes of one CTA in units of 128 times K's k-blocks, as for the other form.
int pick_bn_i8(int64_t M, int N, int pairs, int64_t* cost_out) {
    static const int cand[] = {256, 224, 192, 160, 128};
    const int64_t mp = (M + 2 * gdn::gemm::BM - 1) / (2 * gdn::gemm::BM);
    int best = 256;
    int64_t best_cost = -1;
    for (int bn : cand) {
        const int64_t tiles = mp * ((N + bn - 1) / bn);
        const int64_t cost = (tiles + pairs - 1) / pairs * (256 + bn);
        if (best_cost < 0 || cost < best_cost) {
            best = bn;
            best_cost = cost;
        }
    }
    *cost_out = best_cost / 2;
    return best;
}

constexpr int kMinTileRows = 96, kJoinCost = 250, kBlocksCost = 950;
constexpr int64_t kMaxRowsM = 148 * 128;   // more blocks of tokens than SMs need no plan

template <int BT, int kSplits, int XQ>
struct RowsForm {
    using S = gdn::gemm::RowsShape<BT, XQ>;
    static constexpr auto kernel = gdn::gemm::linear_i8_rows_kernel<BT, kSplits, XQ>;
    static int at_once() {   // (the runtime counts what the kernel is allowed)
        return allow_smem<kernel>(S::SMEM) == cudaSuccess ? resident_clusters<kernel>(kSplits, gdn::gemm::NT, S::SMEM) : 0;
    }
    static cudaError_t launch(const CUtensorMap& tm_x, const CUtensorMap& tm_w, const gdn::gemm::I8Args& a,
                              cudaStream_t st) {
        const cudaError_t e = allow_smem<kernel>(S::SMEM);
        if (e != cudaSuccess) return e;
        const int tiles = a.n_blocks * a.m_blocks, grid = kSplits > 1 ? tiles * kSplits : std::min(tiles, sm_count());
        return Launch((unsigned)grid, gdn::gemm::NT, S::SMEM, st).cluster(kSplits)(kernel, tm_x, tm_w, a);
    }
};

// Tile height and split of K: the fewest bytes (of 128) that one CTA loads, over the
// clusters that run at once; a split (one tile per cluster) pays for its join.  Heights
// below 128 even out the waves (64 rows x 64,000 outputs x 2560: 29.7 us, 31.7 with 128).
// Sets a's tile height and counts; returns log2 of the split and the cost, or -1 where the
// tokens take several blocks and their tiles do not all run at once.
template <int BT>
int plan_i8_rows(gdn::gemm::I8Args& a, int64_t* cost_out = nullptr) {
    const int64_t m_blocks = (a.M + BT - 1) / BT;
    const int kb = (a.K + gdn::gemm::BK8 - 1) / gdn::gemm::BK8;
    const int at_once[4] = {sm_count(), RowsForm<BT, 2, 0>::at_once(), RowsForm<BT, 4, 0>::at_once(),
                            RowsForm<BT, 8, 0>::at_once()};
    int best = -1;
    int64_t best_cost = INT64_MAX;
    for (int i = 0; i < 4 && (1 << i) <= kb; ++i) {
        if (at_once[i] <= 0) break;
        for (int rows = 128; rows >= kMinTileRows; rows -= 8) {
            const int n_blocks = (a.N + rows - 1) / rows;
            const int64_t tiles = n_blocks * m_blocks;
            if ((i > 0 || m_blocks > 1) && tiles > at_once[i]) break;
            const int64_t cost = (tiles + at_once[i] - 1) / at_once[i] * (rows + BT) * ((kb + (1 << i) - 1) >> i) +
                                 (i > 0 ? kJoinCost : 0);
            if (cost < best_cost) {
                best_cost = cost;
                best = i;
                a.tile_rows = rows;
                a.n_blocks = n_blocks;
                a.m_blocks = (int)m_blocks;
            }
        }
    }
    if (cost_out) *cost_out = best_cost;
    return best;
}

template <int BT, int XQ>
cudaError_t launch_i8_rows_planned(const void* x, const void* w, const gdn::gemm::I8Args& a, int split, cudaStream_t st) {
    CUtensorMap tm_x, tm_w;
    if (!i8_map(&tm_w, w, a.N, a.K, a.tile_rows)) return cudaErrorInvalidValue;
    if (XQ > 0) tm_x = tm_w;   // (not used)
    else if (!i8_map(&tm_x, x, a.M, a.K, BT)) return cudaErrorInvalidValue;
    switch (split) {
        case 0: return RowsForm<BT, 1, XQ>::launch(tm_x, tm_w, a, st);
        case 1: return RowsForm<BT, 2, XQ>::launch(tm_x, tm_w, a, st);
        case 2: return RowsForm<BT, 4, XQ>::launch(tm_x, tm_w, a, st);
        default: return RowsForm<BT, 8, XQ>::launch(tm_x, tm_w, a, st);
    }
}

template <int BT>
cudaError_t launch_i8_rows(const void* x, const void* w, gdn::gemm::I8Args a, cudaStream_t st) {
    const int split = plan_i8_rows<BT>(a);
    return launch_i8_rows_planned<BT, 0>(x, w, a, split, st);
}

// One or two rows in bf16 or fp32, by one launch: true if the form takes them (the rows' 8-bit
// k-blocks fit beside the ring).
bool launch_i8_raw_rows(const void* w, gdn::gemm::I8Args a, cudaStream_t st, cudaError_t* e) {
    const int kb = (a.K + gdn::gemm::BK8 - 1) / gdn::gemm::BK8;
    if (a.M <= gdn::gemm::RawShape<24>::ROWS && kb <= 24) {
        const int split = plan_i8_rows<16>(a);
        *e = launch_i8_rows_planned<16, 24>(nullptr, w, a, split, st);
    } else if (a.M <= gdn::gemm::RawShape<48>::ROWS && kb <= 48) {
        const int split = plan_i8_rows<16>(a);
        *e = launch_i8_rows_planned<16, 48>(nullptr, w, a, split, st);
    } else {
        return false;
    }
    return true;
}

// 8-bit rows, then their scales, in the workspace.
size_t i8_scale_off(int64_t M, int32_t K) { return align_up((size_t)M * (size_t)K, 256); }

gdn_status run_linear_i8(const void* x, int32_t x_dtype, const float* x_scale, const int8_t* w, const float* w_scale,
                         int64_t M, int32_t N, int32_t K, int32_t out_dtype, const gdn_out_segment* segs,
                         int32_t n_segs, void* workspace, size_t workspace_bytes, void* stream) {
    if (M < 0 || N <= 0 || K <= 0 || !segs || n_segs <= 0) return GDN_ERR_INVALID_ARG;
    if ((x_dtype != GDN_I8 && !float_dtype(x_dtype)) || !float_dtype(out_dtype)) return GDN_ERR_INVALID_ARG;
    if (n_segs > GDN_LINEAR_MAX_SEGMENTS) return GDN_ERR_UNSUPPORTED;
    if (N % 8 != 0 || K % 16 != 0 || K > 131056) return GDN_ERR_UNSUPPORTED;
    // Row coordinates are int32, the end of a tile past the last row too (tiles have up to 256).
    if (M > 0x7fffffffLL - 256 || N > 0x7fffffff - 256) return GDN_ERR_UNSUPPORTED;
    gdn::gemm::I8Args a = {};
    a.M = M;
    a.N = N;
    a.K = K;
    a.n_segs = n_segs;
    a.out_f32 = out_dtype == GDN_F32;
    int n0 = 0;
    for (int i = 0; i < n_segs; ++i) {
        const gdn_out_segment& g = segs[i];
        if (g.width <= 0 || g.width % 8 != 0 || g.width > N - n0) return GDN_ERR_INVALID_ARG;
        a.seg[i].dst = static_cast<__nv_bfloat16*>(g.dst);
        a.seg[i].n0 = n0;
        a.seg[i].width = g.width;
        n0 += g.width;
    }
    if (n0 != N) return GDN_ERR_INVALID_ARG;
    if (M == 0) return GDN_OK;
    for (int i = 0; i < n_segs; ++i)
        if (!segs[i].dst || !aligned(segs[i].dst, 16)) return GDN_ERR_INVALID_ARG;
    if (!x || !w || !w_scale || !aligned(x, 16) || !aligned(w, 16) || !aligned(w_scale, 16))
        return GDN_ERR_INVALID_ARG;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const bool quantize = x_dtype != GDN_I8;
    const size_t ws_need = quantize ? gdn_linear_i8_workspace_size(M, K) : 0;
    // what is written (the workspace last), what is read
    Span outs[GDN_LINEAR_MAX_SEGMENTS + 1];
    for (int i = 0; i < n_segs; ++i) outs[i] = span(segs[i].dst, M * segs[i].width * elem(out_dtype));
    outs[n_segs] = quantize ? span(workspace, (int64_t)ws_need) : Span{0, 0};
    const Span ins[4] = {span(x, M * K * elem(x_dtype)), span(x_scale, M * 4), span(w, (int64_t)N * K), span(w_scale, (int64_t)N * 4)};
    for (int i = 0; i <= n_segs; ++i) {
        for (int j = i + 1; j <= n_segs; ++j)
            if (overlap(outs[i], outs[j])) return GDN_ERR_INVALID_ARG;
        for (const Span& in : ins)
            if (overlap(outs[i], in)) return GDN_ERR_INVALID_ARG;
    }
    if (quantize) {
        if (x_scale || !workspace || !aligned(workspace, 256)) return GDN_ERR_INVALID_ARG;
        if (workspace_bytes < ws_need) return GDN_ERR_WORKSPACE;
        a.x_raw = x;
        a.x_f32 = x_dtype == GDN_F32;
        a.w_scale = w_scale;
        cudaError_t e;
        if (launch_i8_raw_rows(w, a, st, &e)) return cuda_status(e);
        int8_t* q = static_cast<int8_t*>(workspace);
        float* scale = reinterpret_cast<float*>(q + i8_scale_off(M, K));
        const gdn_status s = run_quantize(x, x_dtype, M, K, q, scale, st);
        if (s != GDN_OK) return s;
        x = q;
        x_scale = scale;
    } else if (!x_scale || !aligned(x_scale, 4)) {
        return GDN_ERR_INVALID_ARG;
    }
    a.x_scale = x_scale;
    a.w_scale = w_scale;
    a.w_ready = quantize;
    cudaError_t e;
    if (M <= 16) e = launch_i8_rows<16>(x, w, a, st);
    else if (M <= 32) e = launch_i8_rows<32>(x, w, a, st);
    else if (M <= 64) e = launch_i8_rows<64>(x, w, a, st);
    else if (M <= 128) e = launch_i8_rows<128>(x, w, a, st);
    else {
        // Several blocks of 128 tokens in the form for few rows where its tiles, with K split,
        // all run at once and load fewer bytes a CTA than pair tiles do by more than its longer
        // epilogue: 252 x 1728 x 3616 7.8 us, 11.1 in pair tiles; 256 x 2560 x 6144 12.4 and
        // 16.0; but 3841 x 152 x 1504 7.8 and 7.2, 1000 x 520 x 1040 7.5 and 6.7.
        int64_t rows_cost = 0, pair_cost = 0;
        gdn::gemm::I8Args r = a;
        const int bn = pick_bn_i8(M, N, std::max(1, sm_count() / 2), &pair_cost);
        const int split = M <= kMaxRowsM ? plan_i8_rows<128>(r, &rows_cost) : -1;
        if (split >= 0 && rows_cost + kBlocksCost < pair_cost * ((K + gdn::gemm::BK8 - 1) / gdn::gemm::BK8)) {
            e = launch_i8_rows_planned<128, 0>(x, w, r, split, st);
        } else {
            switch (bn) {
                case 256: e = launch_i8_pair<256>(x, w, a, st); break;
                case 224: e = launch_i8_pair<224>(x, w, a, st); break;
                case 192: e = launch_i8_pair<192>(x, w, a, st); break;
                case 160: e = launch_i8_pair<160>(x, w, a, st); break;
                default: e = launch_i8_pair<128>(x, w, a, st); break;
            }
        }
    }
    return cuda_status(e);
}

// ---------------------------------------------------------------------------
// Beam selection
// ---------------------------------------------------------------------------
constexpr int kBeamTiles = 2;
// The slice warps that a B200 holds: fixed, not asked of the device, since the workspace's
// size follows from it and may be asked for where there is none.
constexpr int kBeamWarps = 148 * 32;

struct BeamLayout {
    int slices, tiles;
    size_t cand_off, total;
};

// GDN_OK and the layout, or what is wrong with the sizes.
gdn_status beam_layout(int32_t n_groups, int32_t n_beams, int32_t vocab, int32_t n_out, int32_t dtype, BeamLayout* L) {
    if (n_groups < 0 || n_beams <= 0 || vocab <= 0 || n_out <= 0 || !float_dtype(dtype)) return GDN_ERR_INVALID_ARG;
    if (n_beams > GDN_BEAM_MAX_BEAMS || n_out > GDN_BEAM_MAX_OUT || vocab > GDN_BEAM_MAX_VOCAB)
        return GDN_ERR_UNSUPPORTED;
    // Tiles of a slice: at least kBeamTiles (shorter ones spend more on their selection and
    // leave the merge more lists) and n / 16 (a tile has 32 maxima for n of them to be
    // among); longer ones where the slices fill the GPU's warps anyway.
    const int len = gdn::beam::tile_len(elem(dtype));
    L->tiles = (vocab + len - 1) / len;
    const int64_t rows = std::max<int64_t>((int64_t)n_groups * n_beams, 1);
    int64_t each = std::max<int64_t>(rows * L->tiles / kBeamWarps + 1, std::max(kBeamTiles, (n_out + 15) / 16));
    each = std::min<int64_t>(each, gdn::beam::TILES);
    L->slices = std::max((int)(L->tiles / each), 1);
    L->slices = std::max(L->slices, (L->tiles + gdn::beam::TILES - 1) / gdn::beam::TILES);
    // (a merge block holds a list head per slice of the group)
    L->slices = std::min(L->slices, gdn::beam::kMaxLists / n_beams);
    static_assert(GDN_BEAM_MAX_VOCAB / gdn::beam::tile_len(4) <= gdn::beam::kMaxLists / GDN_BEAM_MAX_BEAMS * gdn::beam::TILES,
                  "tiles of a slice");
    const int64_t lists = (int64_t)n_groups * n_beams * L->slices;
    if (lists > 0x7fffffffLL) return GDN_ERR_UNSUPPORTED;   // (their numbers are 32 bits)
    L->cand_off = align_up((size_t)lists * sizeof(gdn::beam::Stat), 256);
    // The workspace asked for is that of the most lists that this many rows or fewer, of this
    // length or shorter, make (there are fewer of them where more rows take longer slices), so
    // that one for the largest call serves every smaller one: slices of `each` tiles are fewer
    // than kBeamWarps in all (each > rows tiles / kBeamWarps) and each >= kBeamTiles, but a
    // row has one slice at least, and one for every TILES tiles.
    const int64_t most = std::max(std::min<int64_t>(kBeamWarps, rows * L->tiles / kBeamTiles),
                                  rows * ((L->tiles + gdn::beam::TILES - 1) / gdn::beam::TILES));
    L->total = align_up((size_t)most * sizeof(gdn::beam::Stat), 256) + align_up((size_t)most * n_out * sizeof(uint64_t), 256);
    return GDN_OK;
}

// ---------------------------------------------------------------------------
// State reordering
// ---------------------------------------------------------------------------
// Whether two buffers of n states each share a byte.  Equal strides: where the states
// of one fall between those of the other, modulo the stride.  Different strides: by
// what the buffers span.
bool buffers_collide(const gdn_state_buffer& a, const gdn_state_buffer& b, int64_t n) {
    const Span sa = span(a.base, (n - 1) * a.stride + a.bytes), sb = span(b.base, (n - 1) * b.stride + b.bytes);
    if (!overlap(sa, sb)) return false;
    if (a.stride != b.stride) return true;
    const int64_t d = (int64_t)(sb.lo - sa.lo);   // b's first state after a's (or before it)
    const int64_t m = ((d % a.stride) + a.stride) % a.stride;
    return m < a.bytes || m + b.bytes > a.stride;
}

template <int WMAX, int U>
cudaError_t launch_reorder(gdn::reorder::Args a, int64_t n_groups, cudaStream_t st) {
    const int per_item = gdn::reorder::NT * U;
    int32_t items = 0;
    for (int i = 0; i < a.n_buffers; ++i) {
        a.buf[i].item0 = items;
        items += (a.buf[i].vecs + per_item - 1) / per_item;
    }
    a.items = items;
    a.total = (int64_t)items * n_groups;
    const unsigned grid = (unsigned)std::min<int64_t>(a.total, 0x7fffffff);
    return Launch(grid, gdn::reorder::NT, 0, st)(gdn::reorder::reorder_kernel<WMAX, U>, a);
}

}  // namespace

namespace gdn {
cudaError_t take_serve_error_word(unsigned int* word) { return take_error_word(word); }
}  // namespace gdn

extern "C" {

void gdn_norm_config_default(gdn_norm_config* cfg) {
    if (!cfg) return;
    cfg->dim = 2560;
    cfg->eps = 1e-6f;
    cfg->res_scale = 1.0f;
    cfg->gate = GDN_GATE_NONE;
    cfg->gate_sigmoid = 0;
    cfg->act_dtype = GDN_BF16;
    cfg->res_dtype = GDN_BF16;
}

gdn_status gdn_block_norm(const gdn_norm_config* cfg, const void* o, const void* x, const void* gate,
                          const float* w_post, const float* w_pre, int64_t T, void* r, void* y, float* y_scale,
                          void* stream) {
    if (!cfg || cfg->dim <= 0 || !(cfg->eps >= 0.f) || !std::isfinite(cfg->eps) || !std::isfinite(cfg->res_scale))
        return GDN_ERR_INVALID_ARG;
    if (!float_dtype(cfg->act_dtype) || !float_dtype(cfg->res_dtype)) return GDN_ERR_INVALID_ARG;
    if (cfg->gate < GDN_GATE_NONE || cfg->gate > GDN_GATE_FULL || T < 0) return GDN_ERR_INVALID_ARG;
    if (cfg->dim % 8 != 0 || cfg->dim > GDN_NORM_MAX_DIM || T > 0x7fffffffLL) return GDN_ERR_UNSUPPORTED;
    if (T == 0) return GDN_OK;
    // what goes with what
    if (!o && (w_post || gate || r || cfg->gate != GDN_GATE_NONE)) return GDN_ERR_INVALID_ARG;
    if (!y && (w_pre || y_scale)) return GDN_ERR_INVALID_ARG;
    if ((cfg->gate == GDN_GATE_NONE) != !gate) return GDN_ERR_INVALID_ARG;
    if (!x || (o && !r) || (y && !w_pre) || (!o && !y)) return GDN_ERR_INVALID_ARG;
    const void* a16[] = {o, x, r, y, w_post, w_pre, cfg->gate == GDN_GATE_TOKEN ? nullptr : gate};
    for (const void* p : a16)
        if (!aligned(p, 16)) return GDN_ERR_INVALID_ARG;   // null passes
    const int ab = elem(cfg->act_dtype), rb = elem(cfg->res_dtype);
    if (!aligned(gate, ab) || !aligned(y_scale, 4)) return GDN_ERR_INVALID_ARG;
    const int64_t n = T * cfg->dim;
    const Span outs[3] = {span(r, n * rb), span(y, n * (y_scale ? 1 : ab)), span(y_scale, T * 4)};
    const int64_t gate_bytes = cfg->gate == GDN_GATE_FULL ? n * ab : cfg->gate == GDN_GATE_TOKEN ? T * ab : cfg->dim * 4;
    const Span ins[5] = {span(x, n * rb), span(o, n * ab), span(gate, gate_bytes), span(w_post, cfg->dim * 4),
                         span(w_pre, cfg->dim * 4)};
    for (int i = 0; i < 3; ++i) {
        for (int j = i + 1; j < 3; ++j)
            if (overlap(outs[i], outs[j])) return GDN_ERR_INVALID_ARG;
        for (int j = 0; j < 5; ++j) {
            const bool in_place = (i == 0 && j == 0 && r == x) || (i == 1 && j == 1 && y == o && !y_scale);
            if (!in_place && overlap(outs[i], ins[j])) return GDN_ERR_INVALID_ARG;
        }
    }
    gdn::bnorm::Args a;
    a.o = o; a.x = x; a.gate = gate;
    a.w_post = w_post; a.w_pre = w_pre;
    a.r = r; a.y = y; a.y_scale = y_scale;
    a.D = cfg->dim;
    a.gate_kind = cfg->gate;
    a.gate_sigmoid = cfg->gate_sigmoid;
    a.eps = cfg->eps;
    a.res_scale = cfg->res_scale;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const bool abf = cfg->act_dtype == GDN_BF16, rbf = cfg->res_dtype == GDN_BF16;
    cudaError_t e;
    if (abf && rbf) e = norm_by_output<__nv_bfloat16, __nv_bfloat16>(a, T, st);
    else if (abf) e = norm_by_output<__nv_bfloat16, float>(a, T, st);
    else if (rbf) e = norm_by_output<float, __nv_bfloat16>(a, T, st);
    else e = norm_by_output<float, float>(a, T, st);
    return cuda_status(e);
}

gdn_status gdn_quantize_rows(const void* x, int32_t x_dtype, int64_t rows, int32_t cols, int8_t* q, float* scale,
                             void* stream) {
    if (rows < 0 || cols <= 0 || !float_dtype(x_dtype)) return GDN_ERR_INVALID_ARG;
    if (cols % 16 != 0 || rows > 0x7fffffffLL) return GDN_ERR_UNSUPPORTED;
    if (rows == 0) return GDN_OK;
    if (!x || !q || !scale || !aligned(x, 16) || !aligned(q, 16) || !aligned(scale, 4)) return GDN_ERR_INVALID_ARG;
    const int64_t n = rows * cols;
    const Span in = span(x, n * elem(x_dtype)), oq = span(q, n), os = span(scale, rows * 4);
    if (overlap(in, oq) || overlap(in, os) || overlap(oq, os)) return GDN_ERR_INVALID_ARG;
    return run_quantize(x, x_dtype, rows, cols, q, scale, static_cast<cudaStream_t>(stream));
}

size_t gdn_linear_i8_workspace_size(int64_t M, int32_t K) {
    if (M < 0 || K <= 0) return 0;
    return i8_scale_off(M, K) + align_up((size_t)M * sizeof(float), 256);
}

gdn_status gdn_linear_i8(const void* x, int32_t x_dtype, const float* x_scale, const int8_t* w, const float* w_scale,
                         int64_t M, int32_t N, int32_t K, int32_t out_dtype, const gdn_out_segment* segs,
                         int32_t n_segs, void* workspace, size_t workspace_bytes, void* stream) {
    return run_linear_i8(x, x_dtype, x_scale, w, w_scale, M, N, K, out_dtype, segs, n_segs, workspace, workspace_bytes,
                         stream);
}

gdn_status gdn_in_proj_i8(const gdn_config* cfg, const void* hidden, int32_t x_dtype, const float* x_scale,
                          const int8_t* w_in, const float* w_scale, int64_t T, int32_t d_model, void* q, void* k,
                          void* v, void* z, void* a, void* b, void* workspace, size_t workspace_bytes, void* stream) {
    gdn_status s = check_config(cfg);
    if (s != GDN_OK) return s;
    if (T < 0 || d_model <= 0) return GDN_ERR_INVALID_ARG;
    const int qk = cfg->n_k_heads * cfg->d_k, vz = cfg->n_v_heads * cfg->d_v, ab = cfg->n_v_heads;
    if (ab % 8 != 0) return GDN_ERR_UNSUPPORTED;
    const gdn_out_segment segs[6] = {{q, qk}, {k, qk}, {v, vz}, {z, vz}, {a, ab}, {b, ab}};
    return run_linear_i8(hidden, x_dtype, x_scale, w_in, w_scale, T, 2 * qk + 2 * vz + 2 * ab, d_model, GDN_BF16, segs,
                         6, workspace, workspace_bytes, stream);
}

gdn_status gdn_out_proj_i8(const gdn_config* cfg, const void* o, int32_t x_dtype, const float* x_scale,
                           const int8_t* w_out, const float* w_scale, int64_t T, int32_t d_model, void* y,
                           void* workspace, size_t workspace_bytes, void* stream) {
    gdn_status s = check_config(cfg);
    if (s != GDN_OK) return s;
    if (T < 0 || d_model <= 0) return GDN_ERR_INVALID_ARG;
    const gdn_out_segment seg = {y, d_model};
    return run_linear_i8(o, x_dtype, x_scale, w_out, w_scale, T, d_model, cfg->n_v_heads * cfg->d_v, GDN_BF16, &seg, 1,
                         workspace, workspace_bytes, stream);
}

size_t gdn_beam_workspace_size(int32_t n_groups, int32_t n_beams, int32_t vocab, int32_t n_out, int32_t logits_dtype) {
    BeamLayout L;
    return beam_layout(n_groups, n_beams, vocab, n_out, logits_dtype, &L) == GDN_OK ? std::max<size_t>(L.total, 256) : 0;
}

gdn_status gdn_beam_select(const void* logits, int32_t logits_dtype, int64_t ld, const float* scores,
                           const uint8_t* finished, int32_t n_groups, int32_t n_beams, int32_t vocab, int32_t n_out,
                           int32_t pad_token, int32_t* parents, int32_t* tokens, float* out_scores, void* workspace,
                           size_t workspace_bytes, void* stream) {
    BeamLayout L;
    const gdn_status s = beam_layout(n_groups, n_beams, vocab, n_out, logits_dtype, &L);
    if (s != GDN_OK) return s;
    if (ld < vocab || pad_token < 0 || pad_token >= vocab) return GDN_ERR_INVALID_ARG;
    if (n_groups == 0) return GDN_OK;
    if (!logits || !scores || !parents || !tokens || !out_scores || !workspace) return GDN_ERR_INVALID_ARG;
    if (!aligned(logits, elem(logits_dtype)) || !aligned(scores, 4) || !aligned(parents, 4) || !aligned(tokens, 4) ||
        !aligned(out_scores, 4) || !aligned(workspace, 256))
        return GDN_ERR_INVALID_ARG;
    const int64_t rows = (int64_t)n_groups * n_beams, res = (int64_t)n_groups * n_out;
    if (ld > (INT64_MAX / 8) / rows) return GDN_ERR_INVALID_ARG;
    const Span outs[4] = {span(parents, res * 4), span(tokens, res * 4), span(out_scores, res * 4),
                          span(workspace, (int64_t)L.total)};
    const Span ins[3] = {span(logits, ((rows - 1) * ld + vocab) * elem(logits_dtype)), span(scores, rows * 4),
                         span(finished, rows)};
    for (int i = 0; i < 4; ++i) {
        for (int j = i + 1; j < 4; ++j)
            if (overlap(outs[i], outs[j])) return GDN_ERR_INVALID_ARG;
        for (int j = 0; j < 3; ++j) {
            const bool in_place = i == 2 && j == 1 && out_scores == scores && n_out == n_beams;
            if (!in_place && overlap(outs[i], ins[j])) return GDN_ERR_INVALID_ARG;
        }
    }
    if (workspace_bytes < L.total) return GDN_ERR_WORKSPACE;
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    gdn::beam::Args a;
    a.logits = logits;
    a.ld = ld;
    a.scores = scores;
    a.finished = finished;
    a.W = n_beams; a.V = vocab; a.n = n_out; a.pad = pad_token;
    a.slices = L.slices; a.tiles = L.tiles;
    a.keys_in_smem = gdn::beam::merge_key_bytes(n_beams, L.slices, n_out) <= gdn::beam::kMaxKeyBytes;
    a.stats = reinterpret_cast<gdn::beam::Stat*>(ws);
    a.cand = reinterpret_cast<uint64_t*>(ws + L.cand_off);
    a.parents = parents;
    a.tokens = tokens;
    a.out_scores = out_scores;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    a.total = (unsigned)(rows * L.slices);
    const unsigned grid = (a.total + gdn::beam::WARPS - 1) / gdn::beam::WARPS, block = 32 * gdn::beam::WARPS;
    cudaError_t e = logits_dtype == GDN_BF16 ? Launch(grid, block, 0, st)(gdn::beam::slice_kernel<__nv_bfloat16>, a)
                                             : Launch(grid, block, 0, st)(gdn::beam::slice_kernel<float>, a);
    if (e != cudaSuccess) return cuda_status(e);
    e = allow_smem<gdn::beam::merge_kernel>(gdn::beam::kMaxMergeSmem);
    if (e != cudaSuccess) return cuda_status(e);
    return cuda_status(Launch((unsigned)n_groups, gdn::beam::MT, gdn::beam::merge_smem(n_beams, L.slices, n_out), st)(
        gdn::beam::merge_kernel, a));
}

gdn_status gdn_reorder_states(const int32_t* parents, int32_t n_groups, int32_t n_beams,
                              const gdn_state_buffer* buffers, int32_t n_buffers, void* stream) {
    if (n_groups < 0 || n_beams <= 0 || n_buffers < 0) return GDN_ERR_INVALID_ARG;
    if (n_beams > GDN_REORDER_MAX_BEAMS || n_buffers > GDN_REORDER_MAX_BUFFERS) return GDN_ERR_UNSUPPORTED;
    if (n_groups == 0 || n_buffers == 0) return GDN_OK;
    if (!parents || !buffers || !aligned(parents, 4)) return GDN_ERR_INVALID_ARG;
    const int64_t n = (int64_t)n_groups * n_beams;
    gdn::reorder::Args a = {};
    a.parents = parents;
    a.W = n_beams;
    a.n_buffers = n_buffers;
    const Span par = span(parents, n * 4);
    for (int i = 0; i < n_buffers; ++i) {
        const gdn_state_buffer& b = buffers[i];
        if (!b.base || !aligned(b.base, 16) || b.bytes <= 0 || b.bytes % 16 != 0 || b.stride % 16 != 0 ||
            b.stride < b.bytes || b.stride > INT64_MAX / n)
            return GDN_ERR_INVALID_ARG;
        if (b.bytes > ((int64_t)16 << 30)) return GDN_ERR_UNSUPPORTED;   // 16-byte units are int32
        if (overlap(par, span(b.base, (n - 1) * b.stride + b.bytes))) return GDN_ERR_INVALID_ARG;
        for (int j = 0; j < i; ++j)
            if (buffers_collide(buffers[j], b, n)) return GDN_ERR_INVALID_ARG;
        a.buf[i].base = static_cast<uint4*>(b.base);
        a.buf[i].stride = b.stride / 16;
        a.buf[i].vecs = (int32_t)(b.bytes / 16);
    }
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    cudaError_t e;
    if (n_beams <= 2) e = launch_reorder<2, 8>(a, n_groups, st);
    else if (n_beams <= 4) e = launch_reorder<4, 4>(a, n_groups, st);
    else if (n_beams <= 8) e = launch_reorder<8, 2>(a, n_groups, st);
    else if (n_beams <= 16) e = launch_reorder<16, 2>(a, n_groups, st);
    else e = launch_reorder<32, 1>(a, n_groups, st);
    return cuda_status(e);
}

}  // extern "C"
