// Rows in 8-bit integers with one scale each:
//   scale = max|x| / 127,  q = rint(127 x / max|x|).
//
// 127 x is exact in fp32 for a bf16 x (8 + 7 bits) and the division is correctly
// rounded, so for bf16 rows q is the rounding of the real quotient (ties to even):
// the quotient of a 15-bit by an 8-bit integer that is no tie is at least 2^-9 of
// itself away from one.  Multiplying by 127 / max|x| instead moves ties (x = max / 2)
// to either side.
//
// Bound by memory: 2 (or 4) bytes read and 1 written per element.  A row belongs to
// one block and stays in its registers between the maximum and the rounding.
#pragma once

#include "device.cuh"

namespace gdn {
namespace quant {

constexpr uint32_t kInfBits = 0x7f800000u;

// What a row's elements are divided by.  The largest |x| comes as its bit pattern,
// which orders finite < infinity < NaN.
struct RowScale {
    float num, den;   // q = rint(x * num / den)
    float scale;      // 0 / NaN: the row is all zeros / not finite, and q is zero
    bool zero;
};

__device__ __forceinline__ RowScale row_scale(uint32_t amax_bits) {
    RowScale s;
    const float amax = __uint_as_float(amax_bits);
    // a power of two keeps 127 x in range at both ends of fp32; it is exact
    const float c = amax > 0x1p100f ? 0x1p-64f : amax < 0x1p-60f ? 0x1p60f : 1.0f;
    s.num = 127.0f * c;
    s.den = amax * c;
    s.zero = amax_bits == 0 || amax_bits >= kInfBits;
    s.scale = amax_bits >= kInfBits ? __uint_as_float(0x7fffffffu) : __fdiv_rn(amax, 127.0f);
    return s;
}

__device__ __forceinline__ int to_i8(float x, const RowScale& s) {
    return __float2int_rn(__fdiv_rn(x * s.num, s.den));
}

// Eight values -> eight int8 in two words.
__device__ __forceinline__ uint2 pack_i8(const float (&f)[8], const RowScale& s) {
    if (s.zero) return make_uint2(0u, 0u);
    uint32_t w[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const uint32_t a = (uint32_t)to_i8(f[4 * h], s) & 0xffu, b = (uint32_t)to_i8(f[4 * h + 1], s) & 0xffu;
        const uint32_t c = (uint32_t)to_i8(f[4 * h + 2], s) & 0xffu, d = (uint32_t)to_i8(f[4 * h + 3], s);
        w[h] = a | (b << 8) | (c << 16) | (d << 24);
    }
    return make_uint2(w[0], w[1]);
}

__device__ __forceinline__ uint32_t max_bits8(const float (&f)[8], uint32_t m) {
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(f[i]) & 0x7fffffffu);
    return m;
}

// Largest value over the block's WARPS warps; every thread gets it.  `slot` is a
// shared array of WARPS words that no reduction in flight uses.
template <int WARPS>
__device__ __forceinline__ uint32_t block_max(uint32_t m, uint32_t* slot) {
    m = __reduce_max_sync(0xffffffffu, m);
    if constexpr (WARPS > 1) {
        if ((threadIdx.x & 31) == 0) slot[threadIdx.x >> 5] = m;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < WARPS; ++i) m = max(m, slot[i]);
    }
    return m;
}

// One row per block.  NV > 0: the row's 8-element vectors fit in NV per thread and
// stay in registers; NV == 0: a longer row is read twice (the second time from L2).
template <typename T, int WARPS, int NV>
__global__ void __launch_bounds__(WARPS * 32)
quantize_rows_kernel(const T* __restrict__ x, int cols, int8_t* __restrict__ q, float* __restrict__ scale) {
    constexpr int NT = WARPS * 32;
    __shared__ uint32_t slot[WARPS];
    // (a product launched behind this kernel may start on its weights)
    grid_dependency_trigger();
    const int64_t row = blockIdx.x;
    const T* xr = x + row * cols;
    int8_t* qr = q + row * cols;
    const int nv = cols / 8;
    uint32_t m = 0;
    if constexpr (NV > 0) {
        float f[NV][8];
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int v = threadIdx.x + j * NT;
            if (v < nv) {
                load8(xr + 8 * v, f[j]);
                m = max_bits8(f[j], m);
            }
        }
        const RowScale s = row_scale(block_max<WARPS>(m, slot));
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int v = threadIdx.x + j * NT;
            if (v < nv) *reinterpret_cast<uint2*>(qr + 8 * v) = pack_i8(f[j], s);
        }
        if (threadIdx.x == 0) scale[row] = s.scale;
    } else {
        for (int v = threadIdx.x; v < nv; v += NT) {
            float f[8];
            load8(xr + 8 * v, f);
            m = max_bits8(f, m);
        }
        const RowScale s = row_scale(block_max<WARPS>(m, slot));
        for (int v = threadIdx.x; v < nv; v += NT) {
            float f[8];
            load8(xr + 8 * v, f);
            *reinterpret_cast<uint2*>(qr + 8 * v) = pack_i8(f, s);
        }
        if (threadIdx.x == 0) scale[row] = s.scale;
    }
}

}  // namespace quant
}  // namespace gdn
