// Dense projections in 8-bit integers on the 5th-generation tensor cores:
//   y[m][n] = x_scale[m] * w_scale[n] * sum_k x[m][k] w[n][k]
// kind::i8 multiplies int8 pairs and adds them in int32, so the sum is exact
// whatever its order; it meets the scales in fp32 in the epilogue.
//
// Two forms:
//   - M > 128 (prefill): the CTA-pair kernel of gemm.cuh with 128 bytes of K per
//     k-block = 128 int8, i.e. twice the K of the bf16 form for the same operand
//     bytes and MMA time.  Bound by those bytes from L2 (MMA pipe 83% busy at
//     4096 x 16480 x 2560), in long runs by the power cap.
//   - M <= 128 (decode), and more tokens where few outputs leave that form's pairs idle
//     and all tiles run at once: linear_i8_rows_kernel below, bound by reading the weights.
#pragma once

#include "gemm.cuh"
#include "quant.cuh"

namespace gdn {
namespace gemm {

// D format s32, A and B int8 (signed), both K-major.
__host__ __device__ constexpr uint32_t idesc_i8(int M, int N) {
    return (2u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

constexpr int BK8 = 128;   // 128 int8 = one 128-byte swizzle row along K

struct I8Args : Args {
    const float* x_scale;
    const float* w_scale;
    int out_f32;           // destinations are fp32 (else bf16)
    int w_ready;           // the kernel before this one does not write w
    int tile_rows;         // channels of a tile (rows kernel): a multiple of 8, at most 128
    const void* x_raw;     // rows that the rows kernel makes 8-bit itself, bf16 or fp32
    int x_f32;
};

#define GDN_ELECT "{\n\t.reg .pred e;\n\t.reg .b32 ex;\n\telect.sync ex|e, 0xffffffff;\n\t"
__device__ __forceinline__ void mma_i8_w(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                         uint32_t accumulate) {
    asm volatile(GDN_ELECT ".reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
                 "@e tcgen05.mma.cta_group::1.kind::i8 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
                 "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
                 : "memory");
}
__device__ __forceinline__ void mma_i8_pair_w(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                              uint32_t accumulate) {
    asm volatile(GDN_ELECT ".reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
                 "@e tcgen05.mma.cta_group::2.kind::i8 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
                 "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
                 : "memory");
}
#undef GDN_ELECT

// The output segment that holds column n.
__device__ __forceinline__ const Seg& segment_of(const Args& p, int n) {
    int j = 0;
    while (j + 1 < p.n_segs && n >= p.seg[j + 1].n0) ++j;
    return p.seg[j];
}

struct I8Op {
    using Args = I8Args;
    static constexpr int BK = BK8;
    static constexpr bool kOverlapped = true;
    static __host__ __device__ constexpr uint32_t idesc(int M, int N) { return idesc_i8(M, N); }
    static __device__ __forceinline__ void mma_pair(uint32_t d, uint64_t a, uint64_t b, uint32_t id, uint32_t acc) {
        mma_i8_pair_w(d, a, b, id, acc);
    }
    // A tile's main loop is half as long as the bf16 form's, so its epilogue has half the
    // time: twice the warps, the scales fetched while the accumulator is still at work, and
    // rows turned in shared memory so that a store fills whole sectors (16 bytes of each of
    // 32 rows at a time took 38 us more at 4096 x 16480 x 2560).
    static constexpr int kEpiWarps = 8;
    static constexpr int kEpiWarpSmem = 128 * 4 + 32 * 64;   // w_scale of up to four 32-column chunks; 32 rows of 64 bytes
    static constexpr int kEpiSmem = kEpiWarps * kEpiWarpSmem;
    template <int BN>
    static __device__ __forceinline__ float prepare(const Args& p, int64_t m, int n0, int part, int lane, void* own) {
        float* ws = static_cast<float*>(own);
        __syncwarp();   // (the tile before this one is done with ws)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int c = part + 2 * i, n = n0 + c * 32 + lane;
            if (c < BN / 32) ws[i * 32 + lane] = n < p.N ? p.w_scale[n] : 0.0f;
        }
        __syncwarp();
        return m < p.M ? p.x_scale[m] : 0.0f;
    }
    // This thread's 64 bytes of row m from column n on, stored by the warp four rows' worth
    // of lanes at a time: piece k (16 bytes) of lane r's row passes through position
    // k ^ (r / 2 % 4) of row r, which keeps both directions free of bank conflicts.
    static __device__ __forceinline__ void store64(const uint4 (&v)[4], uint8_t* rows, const Args& p, int64_t m, int n,
                                                   int elem) {
        const int lane = threadIdx.x & 31, k = lane & 3;
        __syncwarp();   // (the rows before are stored)
#pragma unroll
        for (int i = 0; i < 4; ++i) *reinterpret_cast<uint4*>(rows + lane * 64 + ((i ^ (lane >> 1 & 3)) << 4)) = v[i];
        __syncwarp();
        const int nk = n + k * (16 / elem);
        if (nk >= p.N) return;
        const Seg& sg = segment_of(p, nk);
        uint8_t* dst = reinterpret_cast<uint8_t*>(sg.dst) + (int64_t)(nk - sg.n0) * elem;
        const int64_t m0 = m - lane, pitch = (int64_t)sg.width * elem;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = i * 8 + (lane >> 2);
            if (m0 + r < p.M)
                *reinterpret_cast<uint4*>(dst + (m0 + r) * pitch) =
                    *reinterpret_cast<const uint4*>(rows + r * 64 + ((k ^ (r >> 1 & 3)) << 4));
        }
    }
    template <int BN>
    static __device__ __forceinline__ void store(uint32_t taddr, const Args& p, int64_t m, int n0, int part, float xs,
                                                 void* own) {
        const float* ws = static_cast<const float*>(own);
        uint8_t* rows = static_cast<uint8_t*>(own) + 128 * 4;
#pragma unroll 1
        for (int i = 0; 2 * i + part < BN / 32; ++i) {
            const int c = 2 * i + part;
            uint32_t r[32];
            tmem_ld32(taddr + c * 32, r);
#pragma unroll
            for (int j = 0; j < 32; j += 4) {
                const float4 w = *reinterpret_cast<const float4*>(ws + i * 32 + j);
                r[j] = __float_as_uint((float)(int)r[j] * (xs * w.x));
                r[j + 1] = __float_as_uint((float)(int)r[j + 1] * (xs * w.y));
                r[j + 2] = __float_as_uint((float)(int)r[j + 2] * (xs * w.z));
                r[j + 3] = __float_as_uint((float)(int)r[j + 3] * (xs * w.w));
            }
            uint4 v[4];
            if (p.out_f32) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        v[j] = make_uint4(r[16 * h + 4 * j], r[16 * h + 4 * j + 1], r[16 * h + 4 * j + 2], r[16 * h + 4 * j + 3]);
                    store64(v, rows, p, m, n0 + c * 32 + 16 * h, 4);
                }
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    v[j] = make_uint4(pack_bf16(r[8 * j], r[8 * j + 1]), pack_bf16(r[8 * j + 2], r[8 * j + 3]),
                                      pack_bf16(r[8 * j + 4], r[8 * j + 5]), pack_bf16(r[8 * j + 6], r[8 * j + 7]));
                store64(v, rows, p, m, n0 + c * 32, 2);
            }
        }
        __syncwarp();
    }
};

// ---------------------------------------------------------------------------
// Few tokens: the weights' rows are the MMA's M (up to 128 channels a tile), the tokens
// its N (BT = 16 .. 128, rows past M read as zeros), so a tile's time is that of
// its 16 KiB of weights per k-block and the tokens cost little.  A tile takes fewer channels
// where that deals them out evenly over the SMs (the MMA's rows past them hold whatever the
// stage held and are not read).  One persistent
// CTA per SM with the roles of linear_kernel: TMA producer, MMA issuer, 4 epilogue
// warps over two TMEM accumulators; the ring holds about 200 KiB in flight, several
// times what an SM needs to draw its share of HBM.
// When there are fewer tiles than SMs, a cluster of S CTAs shares a tile: each
// takes a range of K, leaves its int32 sums in its shared memory, and adds up the
// tokens that fall to it over the cluster (exact, so the split changes no bit): one token
// x 2560 x 6144 in 6.3 us over 20 tiles of 4 CTAs.
// Launched behind the kernel that makes the 8-bit rows: the weights, which that
// kernel does not write, are fetched while it still runs.
// ---------------------------------------------------------------------------
// One bf16 or fp32 token, or two short ones (XQ > 0: the most k-blocks of a row): every CTA
// makes them 8-bit itself while its first weights are on their way, into shared memory; that
// saves the launch before.  One token x 16480 x 2560: 9.2 us, 10.4 with that launch, x 64000:
// 25.5 and 28.3; two rows of 6144 lose by it (8.5 and 7.5 for 2560 outputs), and so do more
// rows.
template <int BT, int XQ>
struct RowsShape {
    static_assert(BT % 16 == 0 && BT >= 16 && BT <= 128, "tokens a tile");
    static constexpr int W_BYTES = 128 * BK8;
    static constexpr int X_BYTES = XQ ? 0 : BT * BK8;
    static constexpr int STAGE = W_BYTES + X_BYTES;
    static constexpr int XQ_BYTES = XQ * BT * BK8;
    static constexpr int STAGES = (200 * 1024 - XQ_BYTES) / STAGE;
    static constexpr int OFF_XQ = STAGES * STAGE;
    static constexpr int OFF_BAR = OFF_XQ + XQ_BYTES;
    static constexpr int N_BARS = 2 * STAGES + 6;   // full, empty, acc_full[2], acc_empty[2], drain, x_ready
    static constexpr int OFF_XS = (OFF_BAR + N_BARS * 8 + 8 + 15) & ~15;   // x_scale of the BT tokens
    static constexpr int SMEM = OFF_XS + BT * 4 + 1024;
    static constexpr uint32_t TMEM_COLS = 2 * BT < 32 ? 32 : 2 * BT;
    static_assert(STAGE % 1024 == 0 && XQ_BYTES % 1024 == 0, "swizzle atoms");
    static_assert(SMEM <= 227 * 1024, "shared memory");
    static_assert(STAGES * STAGE >= BT * 128 * 4, "partial sums fit where the stages were");
};
// What a thread of the 128 holds of the raw rows in registers.
template <int XQ>
struct RawShape {
    static constexpr int ROWS = XQ <= 24 ? 2 : 1, VECS = XQ / 8;
};

// All rows of x (at most R, of at most 1024 NV elements) as 8-bit integers, k-blocks
// [k_lo, k_lo + kb_n) of them into shared memory in the layout that a load by tensor map
// leaves, by the four epilogue warps (thread t of 128).  xs: the rows' scales; its upper half
// is scratch.
template <typename T, int R, int NV>
__device__ __forceinline__ void raw_rows_to_i8(const T* x, int M, int K, int k_lo, int kb_n, uint8_t* xq, int tile_bytes,
                                               float* xs, int t) {
    constexpr int kVecs = BK8 / 8;   // of a k-block
    const int nv = K / 8;
    uint32_t* part = reinterpret_cast<uint32_t*>(xs + 8);
    quant::Raw8<T> v[R][NV];
#pragma unroll
    for (int m = 0; m < R; ++m)
#pragma unroll
        for (int j = 0; j < NV; ++j)
            if (m < M && t + j * 128 < nv) v[m][j].load(x + (int64_t)m * K + 8 * (t + j * 128));
#pragma unroll
    for (int m = 0; m < R; ++m) {
        uint32_t amax = 0;
#pragma unroll
        for (int j = 0; j < NV; ++j)
            if (m < M && t + j * 128 < nv) amax = max(amax, v[m][j].max_bits());
        amax = __reduce_max_sync(0xffffffffu, amax);
        if ((t & 31) == 0) part[m * 4 + (t >> 5)] = amax;
    }
    asm volatile("bar.sync 1, 128;" ::: "memory");
    const int lo = k_lo * kVecs, hi = lo + kb_n * kVecs;
#pragma unroll
    for (int m = 0; m < R; ++m) {
        if (m >= M) break;
        const uint32_t* q = part + m * 4;
        const quant::RowScale s = quant::row_scale(max(max(q[0], q[1]), max(q[2], q[3])));
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int i = t + j * 128;
            if (i >= nv || i < lo || i >= hi) continue;
            float f[8];
            v[m][j].get(f);
            const int kb = (i - lo) / kVecs, k8 = (i - lo) % kVecs;
            *reinterpret_cast<uint2*>(xq + kb * tile_bytes + swz128(m, k8 >> 1) + (k8 & 1) * 8) = quant::pack_i8(f, s);
        }
        if (t == 0) xs[m] = s.scale;
    }
}

__device__ __forceinline__ int4 ld_cluster_int4(uint32_t addr) {
    int4 v;
    asm volatile("ld.shared::cluster.v4.s32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(addr)
                 : "memory");
    return v;
}

template <int BT, int kSplits, int XQ>
__global__ void __launch_bounds__(NT, 1)
linear_i8_rows_kernel(const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_w,
                      const __grid_constant__ I8Args p) {
    using S = RowsShape<BT, XQ>;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t sb = (raw + 1023u) & ~1023u;
    uint8_t* smem = smem_raw + (sb - raw);
    const uint32_t bar0 = sb + S::OFF_BAR;
    auto full = [&](int s) { return bar0 + 8u * s; };
    auto empty = [&](int s) { return bar0 + 8u * (S::STAGES + s); };
    auto acc_full = [&](int a) { return bar0 + 8u * (2 * S::STAGES + a); };
    auto acc_empty = [&](int a) { return bar0 + 8u * (2 * S::STAGES + 2 + a); };
    const uint32_t drain = bar0 + 8u * (2 * S::STAGES + 4), x_ready = drain + 8u;
    volatile uint32_t* s_tmem = reinterpret_cast<volatile uint32_t*>(smem + S::OFF_BAR + S::N_BARS * 8);
    volatile uint32_t* s_abort = s_tmem + 1;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int s = 0; s < S::STAGES; ++s) {
            mbar_init(full(s), 1);
            mbar_init(empty(s), 1);
        }
        for (int a = 0; a < 2; ++a) {
            mbar_init(acc_full(a), 1);
            mbar_init(acc_empty(a), 4);
        }
        mbar_init(drain, 1);
        mbar_init(x_ready, 4);
        *s_abort = 0;
        fence_mbar_init();
    }
    if (warp == 0) {
        tmem_alloc(smem_u32(const_cast<uint32_t*>(s_tmem)), S::TMEM_COLS);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *s_tmem;
    grid_dependency_trigger();

    // this CTA's k-blocks [k_lo, k_lo + kb_n) and tiles first, first + step, ...
    const int rank = kSplits > 1 ? (int)cluster_rank() : 0;
    const int kb_all = (p.K + BK8 - 1) / BK8;
    const int k_lo = (int)((int64_t)kb_all * rank / kSplits);
    const int kb_n = (int)((int64_t)kb_all * (rank + 1) / kSplits) - k_lo;
    const int tiles = p.n_blocks * p.m_blocks;   // (with more than one block of tokens, one tile a CTA)
    const int first = blockIdx.x / kSplits, step = gridDim.x / kSplits;
    const int my_tiles = first < tiles ? (tiles - first + step - 1) / step : 0;
    const int m0 = first / p.n_blocks * BT, n_tile0 = first % p.n_blocks;   // first token, first tile of channels
    const int m_here = (int)min((int64_t)BT, p.M - m0);                     // tokens of the block

    if (warp == 0) {
        // ---- TMA producer (one thread) ----
        if (lane == 0) {
            prefetch_tmap(&tm_w);
            const uint32_t total = (uint32_t)my_tiles * kb_n;
            const uint32_t pre = total < (uint32_t)S::STAGES ? total : S::STAGES;
            auto load_w = [&](uint32_t it, int s) {
                const int tile = n_tile0 + (int)(it / kb_n) * step, kb = k_lo + (int)(it % kb_n);
                tma_load_2d(sb + (uint32_t)s * S::STAGE, &tm_w, kb * BK8, tile * p.tile_rows, full(s));
            };
            auto load_x = [&](uint32_t it, int s) {
                if constexpr (XQ > 0) return;
                const int kb = k_lo + (int)(it % kb_n);
                tma_load_2d(sb + (uint32_t)s * S::STAGE + S::W_BYTES, &tm_x, kb * BK8, m0, full(s));
            };
            const uint32_t bytes = (uint32_t)(p.tile_rows * BK8 + S::X_BYTES);   // of a stage
            if constexpr (XQ == 0) prefetch_tmap(&tm_x);
            if (!p.w_ready) grid_dependency_wait();
            for (uint32_t it = 0; it < pre; ++it) {
                mbar_arrive_expect_tx(full(it), bytes);
                load_w(it, it);
            }
            if (p.w_ready) grid_dependency_wait();
            for (uint32_t it = 0; it < pre; ++it) load_x(it, it);
            bool ok = true;
            uint32_t it = pre;
            for (; it < total; ++it) {
                const int s = (int)(it % S::STAGES);
                if (!mbar_wait_bounded(empty(s), ((it / S::STAGES) & 1u) ^ 1u) || *s_abort) {
                    ok = false;
                    break;
                }
                mbar_arrive_expect_tx(full(s), bytes);
                load_w(it, s);
                load_x(it, s);
            }
            if (!ok) {
                record_error(kErrCopyTimeout);
                *s_abort = 1;
            }
            // the last copy armed on each stage lands before the CTA may exit
            for (uint32_t s = 0; s < (uint32_t)S::STAGES && s < it; ++s) {
                const uint32_t last = s + (it - 1 - s) / S::STAGES * S::STAGES;
                mbar_wait_bounded(full(s), (last / S::STAGES) & 1u);
            }
        }
    } else if (warp == 1) {
        // ---- MMA issuer (converged warp, elected lane issues) ----
        // (the limits of the waits below are for this kernel's own work, not for the kernels before it)
        grid_dependency_wait();
        constexpr uint32_t ID = idesc_i8(128, BT);
        uint32_t it = 0;
        bool ok = true;
        if constexpr (XQ > 0) ok = mbar_wait_bounded(x_ready, 0);
        for (int ti = 0; ti < my_tiles && ok; ++ti) {
            const uint32_t a = ti & 1u;
            if (!mbar_wait_bounded(acc_empty(a), ((ti >> 1) & 1u) ^ 1u) || *s_abort) {
                ok = false;
                break;
            }
            tc_fence_after();
            const uint32_t d = tmem + a * BT;
            for (int kb = 0; kb < kb_n; ++kb, ++it) {
                const int s = (int)(it % S::STAGES);
                if (!mbar_wait_bounded(full(s), (it / S::STAGES) & 1u) || *s_abort) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t src = sb + (uint32_t)s * S::STAGE;
                const uint32_t xsrc = XQ > 0 ? sb + S::OFF_XQ + kb * (BT * BK8) : src + S::W_BYTES;
#pragma unroll
                for (int k = 0; k < 4; ++k)   // 32 int8 of K each
                    mma_i8_w(d, sdesc(src + k * 32, 16, 1024), sdesc(xsrc + k * 32, 16, 1024), ID, (kb | k) != 0);
                mma_commit_w(empty(s));
            }
            if (!ok) break;
            mma_commit_w(acc_full(a));
        }
        if (!ok) {
            record_error(kErrMmaTimeout);
            *s_abort = 1;
        }
        // every MMA issued here completes before TMEM and shared memory are released
        mma_commit_w(drain);
        mbar_wait_bounded(drain, 0);
    } else {
        // ---- epilogue: this thread's channel, all tokens ----
        const int q = warp & 3;
        const int row = q * 32 + lane;
        grid_dependency_wait();   // (the rows, or their scales)
        float* xs = reinterpret_cast<float*>(smem + S::OFF_XS);
        if constexpr (XQ > 0) {
            using Raw = RawShape<XQ>;
            static_assert(BT == 16 && 8 + 4 * Raw::ROWS <= BT, "scales and scratch");
            uint8_t* xq = smem + S::OFF_XQ;
            const int t = (int)threadIdx.x - 64;
            if (p.x_f32)
                raw_rows_to_i8<float, Raw::ROWS, Raw::VECS>(static_cast<const float*>(p.x_raw), (int)p.M, p.K, k_lo, kb_n,
                                                            xq, BT * BK8, xs, t);
            else
                raw_rows_to_i8<__nv_bfloat16, Raw::ROWS, Raw::VECS>(static_cast<const __nv_bfloat16*>(p.x_raw), (int)p.M,
                                                                    p.K, k_lo, kb_n, xq, BT * BK8, xs, t);
            fence_async_smem();   // (the MMA reads them)
            __syncwarp();
            if (lane == 0) arrive(x_ready);
        } else if ((int)threadIdx.x - 64 < BT) {
            xs[threadIdx.x - 64] = (int)threadIdx.x - 64 < m_here ? p.x_scale[m0 + threadIdx.x - 64] : 0.0f;
        }
        asm volatile("bar.sync 1, 128;" ::: "memory");   // (the epilogue warps)
        bool ok = true;
        for (int ti = 0; ti < my_tiles; ++ti) {
            const uint32_t a = ti & 1u;
            const int n = row < p.tile_rows ? (n_tile0 + ti * step) * p.tile_rows + row : p.N;
            const float ws = n < p.N ? p.w_scale[n] : 0.0f;
            const Seg& sg = segment_of(p, n);
            if (!mbar_wait_bounded(acc_full(a), (ti >> 1) & 1u) || *s_abort) {
                ok = false;
                break;
            }
            tc_fence_after();
            const uint32_t taddr = tmem + ((uint32_t)(q * 32) << 16) + a * BT;
#pragma unroll 1
            for (int c = 0; c < BT / 16; ++c) {
                uint32_t r[16];
                tmem_ld16(taddr + c * 16, r);
                if constexpr (kSplits > 1) {   // [token][channel] int32 over the stages, all read by now
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        asm volatile("st.shared.b32 [%0], %1;" ::"r"(sb + ((c * 16 + i) * 128 + row) * 4), "r"(r[i])
                                     : "memory");
                } else if (n < p.N) {
                    const int64_t at = (int64_t)(m0 + c * 16) * sg.width + (n - sg.n0);
                    const int left = m_here - c * 16;
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        if (i >= left) break;
                        const float y = (float)(int)r[i] * (xs[c * 16 + i] * ws);
                        if (p.out_f32) reinterpret_cast<float*>(sg.dst)[at + (int64_t)i * sg.width] = y;
                        else sg.dst[at + (int64_t)i * sg.width] = __float2bfloat16_rn(y);
                    }
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) arrive(acc_empty(a));
        }
        if (!ok && lane == 0) {
            record_error(kErrMmaTimeout);
            *s_abort = 1;
        }
    }

    if constexpr (kSplits > 1) {
        // One tile per cluster.  CTA m % kSplits adds up token m, a warp to a token and a
        // lane to four channels.
        cluster_sync();
        const int n = lane * 4 < p.tile_rows ? n_tile0 * p.tile_rows + lane * 4 : p.N;
        if (warp >= 2 && !*s_abort && my_tiles > 0 && n < p.N) {
            const float* xs = reinterpret_cast<const float*>(smem + S::OFF_XS);
            const Seg& sg = segment_of(p, n);
            const float4 ws = *reinterpret_cast<const float4*>(p.w_scale + n);
#pragma unroll 2
            for (int m = rank + (warp - 2) * kSplits; m < m_here; m += 4 * kSplits) {
                int4 v[kSplits];
#pragma unroll
                for (int r = 0; r < kSplits; ++r) v[r] = ld_cluster_int4(map_to_rank(sb + (m * 128 + lane * 4) * 4, r));
#pragma unroll
                for (int r = 1; r < kSplits; ++r) {
                    v[0].x += v[r].x;
                    v[0].y += v[r].y;
                    v[0].z += v[r].z;
                    v[0].w += v[r].w;
                }
                const float f = xs[m];
                const float4 y = make_float4((float)v[0].x * (f * ws.x), (float)v[0].y * (f * ws.y),
                                             (float)v[0].z * (f * ws.z), (float)v[0].w * (f * ws.w));
                const int64_t at = (int64_t)(m0 + m) * sg.width + (n - sg.n0);
                if (p.out_f32) {
                    *reinterpret_cast<float4*>(reinterpret_cast<float*>(sg.dst) + at) = y;
                } else {
                    *reinterpret_cast<uint2*>(sg.dst + at) =
                        make_uint2(pack_bf16(__float_as_uint(y.x), __float_as_uint(y.y)),
                                   pack_bf16(__float_as_uint(y.z), __float_as_uint(y.w)));
                }
            }
        }
        cluster_sync();   // no CTA leaves while its sums may still be read
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 0) {
        tc_fence_after();
        tmem_dealloc(tmem, S::TMEM_COLS);
    }
}

}  // namespace gemm
}  // namespace gdn
