// Rows in 8-bit integers with one scale each:
//   scale = max|x| / 127,  q = rint(127 x / max|x|).
//
// 127 x is exact in fp32 for a bf16 x (8 + 7 bits), and the correctly rounded quotient
// (127 x) / max|x| rounds to the same integer as the real one, ties included: the quotient
// of a 15-bit by an 8-bit integer that is no tie is at least 2^-9 of itself away from one.
// For an fp32 x the result is that of the two fp32 operations, 127 x and the quotient.
// A product with 127 / max|x| is cheaper (4096 rows of 2560 took 14 us with the division
// everywhere, profiled, XU pipe 61% busy) but moves ties (x = max / 2) to either side; it is
// within 2^-22 of the quotient, so only a value that close to a half needs the division.
//
// Bound by memory, 2 (or 4) bytes read and 1 written per element: 32,768 rows of 2560 in 47 us
// (5.4 TB/s), 4096 in 8 to 9; one row by latency, 1.6 us.  A row belongs to one block and stays
// in its registers as loaded between the maximum and the rounding.
#pragma once

#include "device.cuh"

namespace gdn {
namespace quant {

constexpr uint32_t kInfBits = 0x7f800000u;

// 16-byte loads of what is read once: they leave L1 to what is not.
__device__ __forceinline__ uint4 ld_stream(const void* p) {
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p)
                 : "memory");
    return v;
}

// Eight consecutive values of a row, kept as loaded.
template <typename T>
struct Raw8;
template <>
struct Raw8<__nv_bfloat16> {
    uint4 u;
    __device__ __forceinline__ void load(const __nv_bfloat16* p) { u = ld_stream(p); }
    __device__ __forceinline__ void get(float (&f)[8]) const {
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[2 * i] = __uint_as_float(w[i] << 16);
            f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
    // the largest |x|, as its fp32 bit pattern (which orders finite < infinity < NaN)
    __device__ __forceinline__ uint32_t max_bits() const {
        constexpr uint32_t kAbs = 0x7fff7fffu;
        const uint32_t m = __vmaxu2(__vmaxu2(u.x & kAbs, u.y & kAbs), __vmaxu2(u.z & kAbs, u.w & kAbs));
        return max(m << 16, m & 0xffff0000u);
    }
};
template <>
struct Raw8<float> {
    uint4 a, b;
    __device__ __forceinline__ void load(const float* p) {
        a = ld_stream(p);
        b = ld_stream(p + 4);
    }
    __device__ __forceinline__ void get(float (&f)[8]) const {
        const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = __uint_as_float(w[i]);
    }
    __device__ __forceinline__ uint32_t max_bits() const {
        constexpr uint32_t kAbs = 0x7fffffffu;
        return max(max(max(a.x & kAbs, a.y & kAbs), max(a.z & kAbs, a.w & kAbs)),
                   max(max(b.x & kAbs, b.y & kAbs), max(b.z & kAbs, b.w & kAbs)));
    }
};

// What a row's elements are divided by.  The largest |x| comes as its bit pattern,
// which orders finite < infinity < NaN.
struct RowScale {
    float c;          // a power of two that keeps 127 c x in range at both ends of fp32
    float den;        // c max|x|
    float inv;        // about 127 / den
    float scale;      // 0 / NaN: the row is all zeros / not finite, and q is zero
    bool zero;
};

__device__ __forceinline__ RowScale row_scale(uint32_t amax_bits) {
    RowScale s;
    const float amax = __uint_as_float(amax_bits);
    s.c = amax > 0x1p100f ? 0x1p-64f : amax < 0x1p-60f ? 0x1p60f : 1.0f;
    s.den = amax * s.c;
    s.inv = __fdividef(127.0f, s.den);
    s.zero = amax_bits == 0 || amax_bits >= kInfBits;
    s.scale = amax_bits >= kInfBits ? __uint_as_float(0x7fffffffu) : __fdiv_rn(amax, 127.0f);
    return s;
}

// Eight values -> eight int8 in two words.
__device__ __forceinline__ uint2 pack_i8(const float (&f)[8], const RowScale& s) {
    if (s.zero) return make_uint2(0u, 0u);
    constexpr float kRound = 12582912.0f;   // 1.5 * 2^23: t + kRound holds rint(t) in its low bits
    constexpr float kNear = 0.5f - 0x1p-12f;   // |t| <= 127, so t is off by 2^-14 at most
    uint32_t q[8];
    float off = 0.0f;
    auto round = [&](int i, float t) {
        const float r = t + kRound;
        off = fmaxf(off, fabsf(t - (r - kRound)));
        q[i] = __float_as_uint(r);
    };
    if (s.c == 1.0f) {
#pragma unroll
        for (int i = 0; i < 8; ++i) round(i, f[i] * s.inv);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) round(i, (f[i] * s.c) * s.inv);
    }
    if (off > kNear) {
#pragma unroll
        for (int i = 0; i < 8; ++i) q[i] = __float_as_uint(__fdiv_rn(f[i] * (127.0f * s.c), s.den) + kRound);
    }
    const uint32_t a = __byte_perm(q[0], q[1], 0x0040), b = __byte_perm(q[2], q[3], 0x0040);
    const uint32_t c = __byte_perm(q[4], q[5], 0x0040), d = __byte_perm(q[6], q[7], 0x0040);
    return make_uint2(__byte_perm(a, b, 0x5410), __byte_perm(c, d, 0x5410));
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
quantize_rows_kernel(const T* x, int cols, int8_t* q, float* scale) {
    constexpr int NT = WARPS * 32;
    __shared__ uint32_t slot[WARPS];
    // In this order: a product launched behind this kernel may read its weights as soon as
    // it starts, so what ran before this kernel (and may have written them) has to have ended.
    grid_dependency_wait();
    grid_dependency_trigger();
    const int64_t row = blockIdx.x;
    const T* xr = x + row * cols;
    int8_t* qr = q + row * cols;
    const int nv = cols / 8;
    uint32_t m = 0;
    if constexpr (NV > 0) {
        Raw8<T> v[NV];
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int i = threadIdx.x + j * NT;
            if (i < nv) v[j].load(xr + 8 * i);
        }
#pragma unroll
        for (int j = 0; j < NV; ++j)
            if (threadIdx.x + j * NT < nv) m = max(m, v[j].max_bits());
        const RowScale s = row_scale(block_max<WARPS>(m, slot));
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int i = threadIdx.x + j * NT;
            if (i >= nv) continue;
            float f[8];
            v[j].get(f);
            *reinterpret_cast<uint2*>(qr + 8 * i) = pack_i8(f, s);
        }
        if (threadIdx.x == 0) scale[row] = s.scale;
    } else {
        for (int i = threadIdx.x; i < nv; i += NT) {
            Raw8<T> v;
            v.load(xr + 8 * i);
            m = max(m, v.max_bits());
        }
        const RowScale s = row_scale(block_max<WARPS>(m, slot));
        for (int i = threadIdx.x; i < nv; i += NT) {
            Raw8<T> v;
            float f[8];
            v.load(xr + 8 * i);
            v.get(f);
            *reinterpret_cast<uint2*>(qr + 8 * i) = pack_i8(f, s);
        }
        if (threadIdx.x == 0) scale[row] = s.scale;
    }
}

}  // namespace quant
}  // namespace gdn
