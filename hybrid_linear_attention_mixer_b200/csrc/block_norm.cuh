// The norms between two blocks in one pass over the rows:
//   n = o / sqrt(mean(o^2) + eps) * w_post        norm after the block
//   r = x + s * g * n                             gate, residual scale and sum
//   y = r / sqrt(mean(r^2) + eps) * w_pre         norm before the next block
// with y rounded to the activation type or to 8-bit rows with a scale.
//
// Bound by memory: o, x (and a full gate) read once, r and y written once, 10 bytes
// per bf16 element; 47,200 rows of 2560 take 187 us (6.5 TB/s, the copy rate), 16 rows 2.4 us
// (4.8 in the form for many).  A row belongs to one block and stays in its registers through
// the two or three reductions it needs (sum of o^2, sum of r^2, max |y|), which is
// what keeps it to one pass; r passes to the second norm in fp32, unrounded.
//
// Two forms: for many rows a vector per thread (rows up to 2048) or 4 warps with a few, and
// the weights read from L1 when they are used (4,095 rows of 1336: 15.8 us with 6 warps and
// one vector, 17.5 with 4 warps and two); for few (fewer than the SMs hold at once, where a row's latency is
// the call's) 16 warps a row and the weights fetched together with the row.
#pragma once

#include "device.cuh"
#include "quant.cuh"

namespace gdn {
namespace bnorm {

struct Args {
    const void* o;
    const void* x;
    const void* gate;
    const float* w_post;
    const float* w_pre;
    void* r;
    void* y;
    float* y_scale;
    int D;
    int gate_kind;       // gdn_gate
    int gate_sigmoid;
    float eps, res_scale;
};

__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&f)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void store8(float* p, const float (&f)[8]) {
    reinterpret_cast<float4*>(p)[0] = make_float4(f[0], f[1], f[2], f[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(f[4], f[5], f[6], f[7]);
}

// Sum over the block; every thread gets it, added in the same order.  `slot` is a
// shared array of WARPS words that no reduction in flight uses.
template <int WARPS>
__device__ __forceinline__ float block_sum(float v, float* slot) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
    if constexpr (WARPS > 1) {
        if ((threadIdx.x & 31) == 0) slot[threadIdx.x >> 5] = v;
        __syncthreads();
        v = slot[0];
#pragma unroll
        for (int i = 1; i < WARPS; ++i) v += slot[i];
    }
    return v;
}

// 1 / (1 + exp(-g)).  __expf is off by 2 + 1.173 |g| ulp, the sum by half a one, __fdividef by 2
// (and 0 for a sum above 2^126, i.e. g < -87.33): (5 + 1.2 |g|) 2^-23 of the result, below a bf16
// rounding wherever it is not 0.
__device__ __forceinline__ float sigmoid(float g) { return __fdividef(1.0f, 1.0f + __expf(-g)); }

// Blocks an SM shall hold: 1024 threads of them where a thread's loads in flight (2 TA, 1 TR)
// and its r leave that many registers; 47,200 rows of 2560 in bf16: 186 us, 194 with the 72
// registers that the compiler takes by itself, 209 and 267 with 1280 and 1536 threads.
template <typename TA, typename TR, int WARPS, int NV>
constexpr int blocks_per_sm() {
    return NV * (int)(4 * sizeof(TA) + 2 * sizeof(TR)) <= 36 && WARPS <= 8 ? 32 / WARPS : 1;
}

// One row per block of WARPS warps, NV vectors of 8 elements per thread.
template <typename TA, typename TR, bool kI8, int WARPS, int NV>
__global__ void __launch_bounds__(WARPS * 32, blocks_per_sm<TA, TR, WARPS, NV>()) block_norm_kernel(const __grid_constant__ Args p) {
    constexpr int NT = WARPS * 32;
    constexpr bool kFew = WARPS == 16 && NV <= 2;   // weights fetched with the row
    __shared__ float slot_o[WARPS], slot_r[WARPS];
    __shared__ uint32_t slot_y[WARPS];
    grid_dependency_trigger();
    grid_dependency_wait();
    const int64_t row = blockIdx.x, base = row * p.D;
    const int nv = p.D / 8;
    const TA* o = static_cast<const TA*>(p.o);
    const TR* x = static_cast<const TR*>(p.x);
    const TA* gate = static_cast<const TA*>(p.gate);

    using quant::Raw8;
    Raw8<TR> xv[NV];
    Raw8<TA> ov[NV], gv[NV];
    Raw8<float> post[kFew ? NV : 1], pre[kFew ? NV : 1];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int v = threadIdx.x + j * NT;
        if (v >= nv) continue;
        if (o) ov[j].load(o + base + 8 * v);
        xv[j].load(x + base + 8 * v);
        if (p.gate_kind == GDN_GATE_FULL) gv[j].load(gate + base + 8 * v);
        if constexpr (kFew) {
            if (p.w_post) post[j].load(p.w_post + 8 * v);
            if (p.w_pre) pre[j].load(p.w_pre + 8 * v);
        }
    }

    float inv_o = 1.0f;
    if (p.w_post) {
        float sum = 0.0f;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            if (threadIdx.x + j * NT >= nv) continue;
            float f[8];
            ov[j].get(f);
#pragma unroll
            for (int i = 0; i < 8; ++i) sum = fmaf(f[i], f[i], sum);
        }
        inv_o = rsqrtf(block_sum<WARPS>(sum, slot_o) / (float)p.D + p.eps);
    }
    float row_factor = p.res_scale * inv_o;
    if (p.gate_kind == GDN_GATE_TOKEN) {
        const float g = to_f32(gate[row]);
        row_factor *= p.gate_sigmoid ? sigmoid(g) : g;
    }

    float f[NV][8];   // r
    float sum = 0.0f;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int v = threadIdx.x + j * NT;
        if (v >= nv) continue;
        xv[j].get(f[j]);
        if (o) {
            float n[8];
            ov[j].get(n);
#pragma unroll
            for (int i = 0; i < 8; ++i) n[i] *= row_factor;
            if (p.w_post) {
                float w[8];
                if constexpr (kFew) post[j].get(w);
                else load8(p.w_post + 8 * v, w);
#pragma unroll
                for (int i = 0; i < 8; ++i) n[i] *= w[i];
            }
            if (p.gate_kind >= GDN_GATE_CHANNEL) {
                float g[8];
                if (p.gate_kind == GDN_GATE_FULL) gv[j].get(g);
                else load8(static_cast<const float*>(p.gate) + 8 * v, g);
#pragma unroll
                for (int i = 0; i < 8; ++i) n[i] *= p.gate_sigmoid ? sigmoid(g[i]) : g[i];
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) f[j][i] += n[i];
            store8(static_cast<TR*>(p.r) + base + 8 * v, f[j]);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) sum = fmaf(f[j][i], f[j][i], sum);
    }
    if (!p.y) return;
    const float inv_r = rsqrtf(block_sum<WARPS>(sum, slot_r) / (float)p.D + p.eps);

    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int v = threadIdx.x + j * NT;
        if (v >= nv) continue;
        float w[8];
        if constexpr (kFew) pre[j].get(w);
        else load8(p.w_pre + 8 * v, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) f[j][i] = f[j][i] * inv_r * w[i];
        if constexpr (kI8) m = quant::max_bits8(f[j], m);
        else store8(static_cast<TA*>(p.y) + base + 8 * v, f[j]);
    }
    if constexpr (kI8) {
        const quant::RowScale s = quant::row_scale(quant::block_max<WARPS>(m, slot_y));
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int v = threadIdx.x + j * NT;
            if (v < nv) *reinterpret_cast<uint2*>(static_cast<int8_t*>(p.y) + base + 8 * v) = quant::pack_i8(f[j], s);
        }
        if (threadIdx.x == 0) p.y_scale[row] = s.scale;
    }
}

}  // namespace bnorm
}  // namespace gdn
