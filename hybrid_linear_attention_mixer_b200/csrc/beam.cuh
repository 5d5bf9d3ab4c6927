// Beam search's selection over beams and vocabulary.
//   score(w, v) = S_w + x_wv - log sum_u exp(x_wu);  the n best of W * V, ties to the
//   lowest w * V + v.
//
// Within one row the order of the scores is the order of the logits, so one pass
// over the logits suffices: slice_kernel reads a slice of a row once, tile by tile,
// and leaves its sum of exponentials and its n largest logits; merge_kernel then joins
// a group's slices, adds the rows' offsets in fp64 and ranks the few candidates left.
// Bound by reading the logits (a small group: by the latency of the two dependent
// launches).
//
// A warp takes a slice and streams it: each lane keeps its sum of exponentials, about a
// reference of its own, and its largest logit of each tile.  Then, any bound that n of
// these maxima (or of maxima over several tiles) reach is reached by at least n logits; a
// few bisection steps find one that not many more reach.  The vectors behind the tile
// maxima that reach it are read once more (from L2), and the logits that do are ranked
// exactly, by 64-bit keys (logit, then lowest index).  Where ties make them too many (a row of
// equal logits), the bound is found exactly, over logits and then over indexes, by more such
// readings.
// Nothing synchronises warps, so one's selection runs beside the others' streams.
//
// 64 requests of 8 beams x 248,320 bf16 logits, 16 results: 63 us (4.0 TB/s), 57 of it the
// slices (without the exponentials 8 us less, without the selection 11); blocks of 8 warps
// that synchronise took 71.  One request of 4 beams: 12 us, half of it the merge.
#pragma once

#include "device.cuh"

namespace gdn {
namespace beam {

constexpr int WARPS = 4;            // slices (warps) of a slice block
constexpr int VPT = 4;              // 16-byte vectors per lane of a tile
constexpr int TILES = 32;           // most tiles of a slice
constexpr int GROUPS = 8;           // groups of its tiles, whose maxima the bound is found from
constexpr int SETS = GROUPS * 32;
constexpr int LISTED = 256;         // tile maxima that a slice follows up
constexpr int CAP = 256;            // candidates a slice ranks
constexpr int MT = 512;             // threads of a merge block
constexpr int kMaxBeams = GDN_BEAM_MAX_BEAMS;
constexpr int kMaxOut = GDN_BEAM_MAX_OUT;
static_assert(2 * kMaxOut <= SETS && 2 * kMaxOut <= CAP && kMaxOut <= MT, "candidate lists");

// A tile is 32 * VPT vectors of 16 bytes, a slice some tiles.  A row's slices and the
// elements of a lane go by element number, wherever the row starts in memory: equal rows
// have bit-equal sums, so their candidates tie.
__host__ __device__ constexpr int tile_len(int elem_bytes) { return 32 * VPT * (16 / elem_bytes); }

// The sum of exp(x) over a slice: sum * 2^c * exp(-top * kScale), or, c being NaN,
// sum * exp(top).  sum is NaN where the slice holds a NaN or +inf; top is its largest
// logit, -inf (then sum is 0 or NaN) where it holds nothing else.
struct Stat {
    double sum;
    float c, top;
};

struct Args {
    const void* logits;
    int64_t ld;
    const float* scores;
    const uint8_t* finished;   // or null
    int W, V, n, pad, slices;
    int tiles;                 // of a row; slice s has [s tiles / slices, (s + 1) tiles / slices)
    unsigned total;            // slices of all rows
    int keys_in_smem;          // the merge holds a group's candidates in shared memory
    Stat* stats;               // [rows][slices]
    uint64_t* cand;            // [rows][slices][n] keys, descending, 0 = none
    int32_t* parents;
    int32_t* tokens;
    float* out_scores;
};

// Finite logits in order as unsigned integers; +0 and -0 are one.
__device__ __forceinline__ uint32_t ordered(float x) {
    const uint32_t u = __float_as_uint(x + 0.0f);
    return u ^ ((u & 0x80000000u) ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ float from_ordered(uint32_t k) {
    return __uint_as_float(k ^ ((k & 0x80000000u) ? 0x80000000u : 0xffffffffu));
}
// (never 0: the ordered form of a finite number is not)
__device__ __forceinline__ uint64_t make_key(float x, uint32_t index) {
    return ((uint64_t)ordered(x) << 32) | (0xffffffffu - index);
}

__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
constexpr float kLog2e = 1.44269504088896341f;
constexpr double kLn2 = 0.693147180559945309417;

// Two fp32 operations in one instruction.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;"
        : "=l"(reinterpret_cast<uint64_t&>(d))
        : "l"(reinterpret_cast<uint64_t&>(a)), "l"(reinterpret_cast<uint64_t&>(b)), "l"(reinterpret_cast<uint64_t&>(c)));
    return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    float2 d;
    asm("add.rn.f32x2 %0, %1, %2;"
        : "=l"(reinterpret_cast<uint64_t&>(d))
        : "l"(reinterpret_cast<uint64_t&>(a)), "l"(reinterpret_cast<uint64_t&>(b)));
    return d;
}

// 16 bytes of logits.
template <typename T>
struct Vec;
template <>
struct Vec<__nv_bfloat16> {
    static constexpr int N = 8;
    static constexpr uint32_t kNone = 0xff80ff80u;   // -inf
    // the largest of some vectors, NaN ignored as in fmaxf
    template <int K>
    static __device__ __forceinline__ float top(const uint4 (&u)[K]) {
        __nv_bfloat162 m[4] = {as2(u[0].x), as2(u[0].y), as2(u[0].z), as2(u[0].w)};
#pragma unroll
        for (int j = 1; j < K; ++j) {
            m[0] = __hmax2(m[0], as2(u[j].x));
            m[1] = __hmax2(m[1], as2(u[j].y));
            m[2] = __hmax2(m[2], as2(u[j].z));
            m[3] = __hmax2(m[3], as2(u[j].w));
        }
        const __nv_bfloat162 c = __hmax2(__hmax2(m[0], m[1]), __hmax2(m[2], m[3]));
        return fmaxf(__low2float(c), __high2float(c));
    }
    static __device__ __forceinline__ __nv_bfloat162 as2(uint32_t w) { return reinterpret_cast<__nv_bfloat162&>(w); }
    static __device__ __forceinline__ float2 pair(uint4 u, int i) {
        const uint32_t w = i == 0 ? u.x : i == 1 ? u.y : i == 2 ? u.z : u.w;
        return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
    }
    static __device__ __forceinline__ float get(uint4 u, int i) {
        const uint32_t w = i < 2 ? u.x : i < 4 ? u.y : i < 6 ? u.z : u.w;
        return __uint_as_float((i & 1) ? (w & 0xffff0000u) : (w << 16));
    }
    static __device__ __forceinline__ void set(uint4& u, int i, __nv_bfloat16 x) {
        const uint32_t b = __bfloat16_as_ushort(x);
        uint32_t& w = i < 2 ? u.x : i < 4 ? u.y : i < 6 ? u.z : u.w;
        w = (i & 1) ? ((w & 0xffffu) | (b << 16)) : ((w & 0xffff0000u) | b);
    }
};
template <>
struct Vec<float> {
    static constexpr int N = 4;
    static constexpr uint32_t kNone = 0xff800000u;
    template <int K>
    static __device__ __forceinline__ float top(const uint4 (&u)[K]) {
        float m = -INFINITY;
#pragma unroll
        for (int j = 0; j < K; ++j)
            m = fmaxf(fmaxf(fmaxf(m, __uint_as_float(u[j].x)), fmaxf(__uint_as_float(u[j].y), __uint_as_float(u[j].z))),
                      __uint_as_float(u[j].w));
        return m;
    }
    static __device__ __forceinline__ float2 pair(uint4 u, int i) {
        return i == 0 ? make_float2(__uint_as_float(u.x), __uint_as_float(u.y))
                      : make_float2(__uint_as_float(u.z), __uint_as_float(u.w));
    }
    static __device__ __forceinline__ float get(uint4 u, int i) {
        return __uint_as_float(i == 0 ? u.x : i == 1 ? u.y : i == 2 ? u.z : u.w);
    }
    static __device__ __forceinline__ void set(uint4& u, int i, float x) {
        (i == 0 ? u.x : i == 1 ? u.y : i == 2 ? u.z : u.w) = __float_as_uint(x);
    }
};

// (coherent: the kernel before, which may have written the logits, can still run when this one starts)
__device__ __forceinline__ uint4 ld_once(const void* p) {
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}

// The 16 bytes that start `shift` bytes (2 .. 14, even) into the vector at p, which is
// 16-byte aligned: two aligned loads (a warp's second ones hit the lines of its first).
__device__ __forceinline__ uint4 ld_shifted(const uint8_t* p, int shift) {
    const uint4 a = *reinterpret_cast<const uint4*>(p), b = *reinterpret_cast<const uint4*>(p + 16);
    uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    if (shift & 8)
#pragma unroll
        for (int i = 0; i < 6; ++i) w[i] = w[i + 2];
    if (shift & 4)
#pragma unroll
        for (int i = 0; i < 5; ++i) w[i] = w[i + 1];
    if (shift & 2)
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = __funnelshift_r(w[i], w[i + 1], 16);
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// A row is live when it can give candidates from its logits.
__device__ __forceinline__ bool row_live(const Args& p, int64_t row) {
    const float score = p.scores[row];   // (both on their way at once)
    const uint8_t ended = p.finished ? p.finished[row] : 0;
    return !ended && isfinite(score);
}

// Elements [i0, i0 + N) of a row that starts `shift` bytes into a 16-byte vector; -inf
// past its end.  The loads stay within the row.
template <typename T>
__device__ __forceinline__ uint4 load_vec(const T* x, int i0, int V, int shift) {
    constexpr int N = Vec<T>::N;
    const int skew = shift / (int)sizeof(T);
    if (i0 >= skew && i0 + (skew ? 2 * N - skew : N) <= V)
        return skew ? ld_shifted(reinterpret_cast<const uint8_t*>(x + i0) - shift, shift) : ld_once(x + i0);
    uint4 u = make_uint4(Vec<T>::kNone, Vec<T>::kNone, Vec<T>::kNone, Vec<T>::kNone);
#pragma unroll
    for (int e = 0; e < N; ++e)
        if (i0 + e < V) Vec<T>::set(u, e, x[i0 + e]);
    return u;
}

// A bound that at least n of the SETS maxima reach and not many more (n + 8; where ties
// make them more, fewer than n are above it, and tied is set); each lane holds GROUPS of
// them.  -FLT_MAX where no more than n are above -inf.
__device__ __forceinline__ float find_bound(const float (&mine)[GROUPS], float top, int n, bool& tied) {
    int valid = 0;
    uint32_t least = 0xffffffffu;
#pragma unroll
    for (int i = 0; i < GROUPS; ++i) {
        if (mine[i] > -INFINITY) {
            ++valid;
            least = min(least, ordered(mine[i]));
        }
    }
    valid = __reduce_add_sync(0xffffffffu, valid);
    least = __reduce_min_sync(0xffffffffu, least);
    tied = false;
    if (valid <= n) return -3.402823466e38f;
    uint32_t lo = least, hi = ordered(top);   // at least n reach lo, fewer reach anything above hi
    int at_lo = valid;
    while (at_lo > n + 8 && hi > lo) {
        const uint32_t mid = lo + (hi - lo + 1) / 2;
        const float b = from_ordered(mid);
        int c = 0;
#pragma unroll
        for (int i = 0; i < GROUPS; ++i) c += mine[i] >= b;
        c = __reduce_add_sync(0xffffffffu, c);
        if (c >= n) {
            lo = mid;
            at_lo = c;
        } else {
            hi = mid - 1;
        }
    }
    tied = at_lo > n + 8;
    return from_ordered(lo);
}

// The fast sum: exp(x) / 2^c is 2^(x log2e - c) in one fused operation, c an integer near
// the largest x so far.  log2e in fp32 is off by 1.3e-8 of itself (too small: kScale < 0), which
// scales x: that is taken back at the slice's top, so what is left goes by the distance from it.
// kSpan: how far above c a maximum may lie; kMaxTop: the size of x up to which c is exact.
constexpr float kSpan = 32.0f, kMaxTop = 65536.0f;
constexpr double kScale = (double)kLog2e * kLn2 - 1.0;

// 2^k for an integer k <= 0 (0 below the normal numbers)
__device__ __forceinline__ double pow2(float k) {
    return k > -1000.0f ? __hiloint2double((1023 + (int)k) << 20, 0) : 0.0;
}

// A lane's sum of exponentials, in units of 2^c.
struct Running {
    float c = -2.0f * kMaxTop;
    double sum = 0.0;
    // adds a tile; returns its largest logit
    template <typename T>
    __device__ __forceinline__ float add(const uint4 (&v)[VPT]) {
        const float tm = Vec<T>::top(v);   // (NaN show in the sum)
        if (tm * kLog2e > c + kSpan) {
            const float up = ceilf(fminf(tm, kMaxTop) * kLog2e);
            sum *= pow2(c - up);
            c = up;
        }
        float2 s[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
#pragma unroll
        for (int j = 0; j < VPT; ++j)
#pragma unroll
            for (int e = 0; e < Vec<T>::N / 2; ++e) {
                const float2 y = fma2(Vec<T>::pair(v[j], e), make_float2(kLog2e, kLog2e), make_float2(-c, -c));
                s[e & 1] = add2(s[e & 1], make_float2(exp2_fast(y.x), exp2_fast(y.y)));
            }
        const float2 both = add2(s[0], s[1]);
        sum += (double)(both.x + both.y);
        return tm;
    }
};

template <typename T>
__global__ void __launch_bounds__(WARPS * 32, 32 / WARPS) slice_kernel(const __grid_constant__ Args p) {
    using X = Vec<T>;
    constexpr int N = X::N, kStep = 32 * N, kTile = kStep * VPT;
    constexpr uint32_t kAll = 0xffffffffu;
    __shared__ uint64_t s_keys[WARPS][CAP];
    __shared__ float s_tops[WARPS][TILES * 32];
    __shared__ uint16_t s_lists[WARPS][LISTED];
    __shared__ int s_counts[WARPS];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    grid_dependency_wait();
    const unsigned at = blockIdx.x * WARPS + warp;
    const unsigned row = at / (unsigned)p.slices, slice = at % (unsigned)p.slices;
    if (at >= p.total || !row_live(p, row)) {
        grid_dependency_trigger();
        return;
    }
    uint64_t* s_key = s_keys[warp];
    float* s_top = s_tops[warp] + lane;   // this lane's largest logit of tile t: s_top[32 t]
    uint16_t* s_list = s_lists[warp];
    int& s_n = s_counts[warp];
    const T* x = static_cast<const T*>(p.logits) + row * p.ld;
    const int shift = (int)(reinterpret_cast<uintptr_t>(x) & 15u);
    const int tile_lo = (int)((int64_t)p.tiles * slice / p.slices);
    const int tiles = (int)((int64_t)p.tiles * (slice + 1) / p.slices) - tile_lo;
    const int begin = tile_lo * kTile, first = begin + lane * N;   // this lane's first element
    // lane's vector j of the slice, j < tiles * VPT
    auto vec = [&](int j) { return load_vec<T>(x, first + j * kStep, p.V, shift); };
    auto load_tile = [&](uint4 (&u)[VPT], int t) {
        if (t >= tiles) return;
        const T* at = x + first + t * kTile;
        if (shift == 0 && begin + (t + 1) * kTile <= p.V) {
#pragma unroll
            for (int j = 0; j < VPT; ++j) u[j] = ld_once(at + j * kStep);
        } else if (shift != 0 && begin + t * kTile > 0 && begin + (t + 1) * kTile + N <= p.V) {
#pragma unroll
            for (int j = 0; j < VPT; ++j) u[j] = ld_shifted(reinterpret_cast<const uint8_t*>(at + j * kStep) - shift, shift);
        } else {
#pragma unroll 1
            for (int j = 0; j < VPT; ++j) {
                const uint4 a = vec(t * VPT + j);
#pragma unroll
                for (int k = 0; k < VPT; ++k)
                    if (k == j) u[k] = a;
            }
        }
    };

    // one tile's vectors are on their way while the other's are worked on
    uint4 even[VPT], odd[VPT];
    Running run;
    load_tile(even, 0);
#pragma unroll 1
    for (int t = 0; t < tiles; t += 2) {
        load_tile(odd, t + 1);
        s_top[32 * t] = run.template add<T>(even);
        if (t + 1 >= tiles) break;
        load_tile(even, t + 2);
        s_top[32 * t + 32] = run.template add<T>(odd);
    }

    float mine[GROUPS], top = -INFINITY;
#pragma unroll
    for (int i = 0; i < GROUPS; ++i) {
        mine[i] = -INFINITY;
        for (int t = i; t < tiles; t += GROUPS) mine[i] = fmaxf(mine[i], s_top[32 * t]);   // (this lane's own)
        top = fmaxf(top, mine[i]);
    }
    float c = run.c;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) {
        top = fmaxf(top, __shfl_xor_sync(kAll, top, d));
        c = fmaxf(c, __shfl_xor_sync(kAll, c, d));
    }
    double sum = run.sum * pow2(run.c - c);
    if (top > -INFINITY && !(fabsf(top) <= kMaxTop)) {
        // beyond the fast sum: about the top itself
        c = __int_as_float(0x7fffffff);
        sum = 0.0;
#pragma unroll 1
        for (int j = 0; j < tiles * VPT; ++j) {
            const uint4 u = vec(j);
            float part = 0.0f;
#pragma unroll
            for (int e = 0; e < N; ++e) part += exp2_fast((X::get(u, e) - top) * kLog2e);
            sum += (double)part;
        }
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(kAll, sum, d);
    if (lane == 0) {
        p.stats[at] = Stat{sum, c, top};
        s_n = 0;
    }

    // The tile maxima that reach the bound, and of the vectors behind them the logits that do;
    // if those are too many to hold because of ties, the ones above the bound.
    bool tied;
    float bound = find_bound(mine, top, p.n, tied);
    float low = bound;
    bool held;
#pragma unroll 1
    while (true) {
        int listed = 0;
#pragma unroll 4
        for (int t = 0; t < tiles; ++t) {
            const bool hits = s_top[32 * t] >= low;
            const uint32_t hit = __ballot_sync(kAll, hits);
            const int k = listed + __popc(hit & ((1u << lane) - 1u));
            if (hits && k < LISTED) s_list[k] = (uint16_t)(t * 32 + lane);
            listed += __popc(hit);
        }
        __syncwarp();
        for (int i = lane; i < min(listed, LISTED) * VPT; i += 32) {
            const int set = s_list[i / VPT];
            const int i0 = begin + set / 32 * kTile + i % VPT * kStep + set % 32 * N;
            const uint4 u[1] = {load_vec<T>(x, i0, p.V, shift)};
            if (X::top(u) >= low) {
#pragma unroll
                for (int e = 0; e < N; ++e) {
                    const float f = X::get(u[0], e);
                    if (f >= low) {
                        const int k = atomicAdd(&s_n, 1);
                        if (k < CAP) s_key[k] = make_key(f, i0 + e);
                    }
                }
            }
        }
        __syncwarp();
        held = listed <= LISTED && s_n <= CAP;
        if (held || !tied || low > bound) break;
        low = from_ordered(ordered(bound) + 1u);   // the next number
        __syncwarp();
        if (lane == 0) s_n = 0;
        __syncwarp();
    }
    if (low > bound) {   // of those equal to the bound, the first n
        int have = 0;   // logits equal to the bound so far
#pragma unroll 1
        for (int j = 0; j < tiles * VPT && have < p.n; ++j) {   // 32 vectors in a row
            const uint4 u = vec(j);
            int mine_eq = 0;
#pragma unroll
            for (int e = 0; e < N; ++e) mine_eq += X::get(u, e) == bound;
            int upto = mine_eq;   // this lane's and those of the lanes before
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int v = __shfl_up_sync(kAll, upto, d);
                if (lane >= d) upto += v;
            }
            int order = have + upto - mine_eq;
#pragma unroll
            for (int e = 0; e < N; ++e)
                if (X::get(u, e) == bound && order++ < p.n) {
                    const int k = atomicAdd(&s_n, 1);
                    if (k < CAP) s_key[k] = make_key(bound, first + j * kStep + e);
                }
            have += __shfl_sync(kAll, upto, 31);
        }
        __syncwarp();
        held = held && s_n <= CAP;
    }
    if (!held) {
        // Too many reach it.  The n-th largest logit itself ...
        auto each = [&](auto&& use) {   // use(value, index) for the lane's logits
#pragma unroll 1
            for (int j = 0; j < tiles * VPT; ++j) {
                const uint4 u = vec(j);
#pragma unroll
                for (int e = 0; e < N; ++e) use(X::get(u, e), first + j * kStep + e);
            }
        };
        auto count = [&](auto&& pred) {
            int n = 0;
            each([&](float f, int i) { n += pred(f, i); });
            return __reduce_add_sync(kAll, n);
        };
        uint32_t lo = ordered(bound), hi = ordered(top);
        while (hi > lo) {
            const uint32_t mid = lo + (hi - lo + 1) / 2;
            const float b = from_ordered(mid);
            if (count([&](float f, int) { return f >= b; }) >= p.n) lo = mid;
            else hi = mid - 1;
        }
        bound = from_ordered(lo);
        // ... and the index of the last one of its kind that is still among the n
        const int above = count([&](float f, int) { return f > bound; });
        int i_lo = begin, i_hi = min(p.V, begin + tiles * kTile) - 1;
        while (i_lo < i_hi) {
            const int mid = i_lo + (i_hi - i_lo) / 2;
            if (above + count([&](float f, int i) { return f == bound && i <= mid; }) >= p.n) i_hi = mid;
            else i_lo = mid + 1;
        }
        __syncwarp();
        if (lane == 0) s_n = 0;
        __syncwarp();
        each([&](float f, int i) {
            if (f > bound || (f == bound && i <= i_lo)) s_key[atomicAdd(&s_n, 1)] = make_key(f, i);
        });
        __syncwarp();
    }
    const int total = s_n;
    uint64_t* out = p.cand + (int64_t)at * p.n;
    for (int i = lane; i < total; i += 32) {
        const uint64_t k = s_key[i];
        int rank = 0;
#pragma unroll 4
        for (int j = 0; j < total; ++j) rank += s_key[j] > k;
        if (rank < p.n) out[rank] = k;
    }
    for (int i = total + lane; i < p.n; i += 32) out[i] = 0;
    grid_dependency_trigger();   // (the merge may be set up; it waits for this grid's end)
}

// fp64 scores in order as unsigned integers (never 0 for a finite one).
__device__ __forceinline__ uint64_t ordered64(double x) {
    const uint64_t u = (uint64_t)__double_as_longlong(x + 0.0);
    return u ^ ((u >> 63) ? ~0ull : (1ull << 63));
}
__device__ __forceinline__ double from_ordered64(uint64_t k) {
    return __longlong_as_double((long long)(k ^ ((k >> 63) ? (1ull << 63) : ~0ull)));
}

// One candidate of a group; better() is the order of the results.
constexpr int kTokenBits = 20;
static_assert(GDN_BEAM_MAX_VOCAB <= 1 << kTokenBits && kMaxBeams <= 1 << (32 - kTokenBits), "Cand::at");
struct Cand {
    uint64_t score;   // ordered; 0: none
    uint32_t at;      // w * 2^20 + v: in the order of w * V + v
    uint32_t logit;   // ordered
    // the score's upper half, in the same order; 0: none
    __device__ __forceinline__ uint32_t rough() const { return (uint32_t)(score >> 32); }
};
// Within a beam the logits decide: beside a score of 1e17, say, fp64 does not tell them apart.
__device__ __forceinline__ bool better(const Cand& a, const Cand& b) {
    if (a.score != b.score) return a.score > b.score;
    return a.at >> kTokenBits == b.at >> kTokenBits && a.logit != b.logit ? a.logit > b.logit : a.at < b.at;
}

// How many of c[0 .. total) are better than c[i], for the items i that the block's
// threads take: `each` threads (a power of two) share an item.  use(i, rank) runs on one.
template <typename F>
__device__ __forceinline__ void rank_all(const Cand* c, int total, F&& use) {
    int each = 1;
    while (each < 32 && each * 2 * total <= MT) each *= 2;
    const int sub = threadIdx.x % each;
    for (int i0 = 0; i0 < total; i0 += MT / each) {
        const int i = i0 + threadIdx.x / each;
        int rank = 0;
        if (i < total) {
            const Cand mine = c[i];
#pragma unroll 4
            for (int j = sub; j < total; j += each) rank += better(c[j], mine);
        }
        for (int d = each / 2; d > 0; d >>= 1) rank += __shfl_xor_sync(0xffffffffu, rank, d);
        if (i < total && sub == 0) use(i, rank);
    }
}

// A bound on the rough scores that at least n of c[0 .. total) reach and not many more
// (n + 8, but for equal ones); 1, which all candidates reach, where there are no more than
// n.  By the whole block; s is scratch in shared memory that nothing else uses.
struct Scratch {
    int valid;
    uint32_t least, most;
};
__device__ __noinline__ uint32_t block_bound(const Cand* c, int total, int n, Scratch* s) {
    const int tid = threadIdx.x;
    if (tid == 0) *s = Scratch{0, ~0u, 0};
    __syncthreads();
    uint32_t least = ~0u, most = 0;
    int valid = 0;
    for (int i = tid; i < total; i += MT) {
        const uint32_t r = c[i].rough();
        if (r) {
            ++valid;
            least = min(least, r);
            most = max(most, r);
        }
    }
    valid = __reduce_add_sync(0xffffffffu, valid);
    least = __reduce_min_sync(0xffffffffu, least);
    most = __reduce_max_sync(0xffffffffu, most);
    if (tid % 32 == 0) {
        atomicAdd(&s->valid, valid);
        atomicMin(&s->least, least);
        atomicMax(&s->most, most);
    }
    __syncthreads();
    int reach = s->valid;
    if (reach <= n) return 1;
    uint32_t lo = s->least, hi = s->most;   // at least n reach lo, fewer reach anything above hi
    while (reach > n + 8 && hi > lo) {
        const uint32_t mid = lo + (hi - lo + 1) / 2;
        int k = 0;
        for (int i = 0; i < total; i += MT) k += __syncthreads_count(i + tid < total && c[i + tid].rough() >= mid);
        if (k >= n) {
            lo = mid;
            reach = k;
        } else {
            hi = mid - 1;
        }
    }
    return lo;
}

// Shared memory of a merge block: list heads, candidates, then the group's keys if they
// are held there (up to kMaxKeyBytes).
constexpr size_t kMaxKeyBytes = 64 * 1024;
constexpr int kFew = 96;               // candidates that are ranked as they are
constexpr int kMaxLists = 4096;        // of a group
constexpr size_t kMaxMergeSmem = (kMaxLists + (size_t)kMaxOut * kMaxOut) * sizeof(Cand) + kMaxKeyBytes;
static_assert(kMaxMergeSmem <= 210 * 1024, "shared memory of the merge");
__host__ __device__ constexpr int merge_cap(int n) { return n * n < 512 ? 512 : n * n; }   // candidates
inline size_t merge_key_bytes(int W, int slices, int n) { return (size_t)W * slices * n * sizeof(uint64_t); }
inline size_t merge_smem(int W, int slices, int n) {
    const size_t keys = merge_key_bytes(W, slices, n);
    return ((size_t)W * slices + merge_cap(n)) * sizeof(Cand) + (keys <= kMaxKeyBytes ? keys : 0);
}

// One block per group.
__global__ void __launch_bounds__(MT) merge_kernel(const __grid_constant__ Args p) {
    extern __shared__ __align__(16) uint8_t smem[];
    Cand* head = reinterpret_cast<Cand*>(smem);
    Cand* cand = head + p.W * p.slices;
    // a row's candidates have the score (logit - ref) + offset; a finished beam's one: offset
    __shared__ double ref[kMaxBeams], offset[kMaxBeams];
    __shared__ uint8_t kind[kMaxBeams];    // 0: no candidates, 1: from the logits, 2: finished
    __shared__ int sel[kMaxOut];           // the lists of the n best heads, best first
    __shared__ int s_n, s_few, s_lists;
    __shared__ uint16_t s_list[kMaxLists]; // the lists whose heads reach the bound
    __shared__ Scratch scratch[2];
    __shared__ Cand few[kFew];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t row0 = (int64_t)blockIdx.x * p.W;
    const int lists = p.W * p.slices;
    if (tid == 0) s_n = s_few = s_lists = 0;
    grid_dependency_trigger();
    grid_dependency_wait();
    const uint64_t* keys = p.cand + row0 * p.slices * p.n;
    // The group's keys, on their way while the rows' sums are formed (of rows that left none
    // too: whatever is there is not used).
    constexpr int kAhead = 4;
    const int n_keys = p.keys_in_smem ? lists * p.n : 0;
    uint64_t ahead[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
        if (tid + i * MT < n_keys) ahead[i] = keys[tid + i * MT];

    for (int w = warp; w < p.W; w += MT / 32) {
        const int64_t row = row0 + w;
        const Stat* st = p.stats + row * p.slices;
        Stat mine = lane < p.slices ? st[lane] : Stat{0.0, -INFINITY, -INFINITY};   // (used only if the row is live)
        const float score = p.scores[row];
        const bool fin = p.finished && p.finished[row];
        double off = score;
        float top = -INFINITY;
        if (!fin && isfinite(score)) {
            // sums of exp(x) / (2^c exp(-top kScale)), or, some c being NaN, / exp(top)
            float c = mine.c;
            top = mine.top;
            bool fast = !isnan(mine.c);
            for (int s = lane + 32; s < p.slices; s += 32) {
                top = fmaxf(top, st[s].top);
                c = fmaxf(c, st[s].c);
                fast &= !isnan(st[s].c);
            }
#pragma unroll
            for (int d = 16; d > 0; d >>= 1) {
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
                c = fmaxf(c, __shfl_xor_sync(0xffffffffu, c, d));
            }
            fast = __all_sync(0xffffffffu, fast);
            double sum = 0.0;
            for (int s = lane;;) {
                // (no logits: the sum is 0, or the NaN that has to show)
                double f = 1.0;
                if (mine.top > -INFINITY)
                    f = fast ? pow2(mine.c - c) * (1.0 - ((double)mine.top - (double)top) * kScale)   // (exp of 1e-6 at most where it matters)
                             : exp((isnan(mine.c) ? (double)mine.top : (double)mine.c * kLn2 - (double)mine.top * kScale) -
                                   (double)top);
                sum += mine.sum * f;
                if ((s += 32) >= p.slices) break;
                mine = st[s];
            }
#pragma unroll
            for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
            // off + (logit - top) is the score
            off -= log(sum);   // (nothing but -inf: +inf; a NaN or +inf among the logits: NaN)
            if (fast && top > -INFINITY) off += (double)top * (1.0 + kScale) - (double)c * kLn2;
        }
        if (lane == 0) {
            ref[w] = top;
            offset[w] = off;
            kind[w] = !isfinite(off) ? 0 : fin ? 2 : 1;
        }
    }
    if (p.keys_in_smem) {
        uint64_t* mine = reinterpret_cast<uint64_t*>(cand + merge_cap(p.n));
#pragma unroll
        for (int i = 0; i < kAhead; ++i)
            if (tid + i * MT < n_keys) mine[tid + i * MT] = ahead[i];
        for (int i = tid + kAhead * MT; i < n_keys; i += MT) mine[i] = keys[i];
        keys = mine;
    }
    __syncthreads();
    // Entry e of list l, which is beam w's.  A finished beam's one entry is the first of its
    // first list.
    auto entry = [&](int l, int w, int e) {
        double score = offset[w];
        Cand c{0, (uint32_t)(w << kTokenBits | p.pad), 0};
        if (kind[w] == 1) {
            const uint64_t k = keys[l * p.n + e];
            if (!k) return c;
            c.logit = (uint32_t)(k >> 32);
            score += (double)from_ordered(c.logit) - ref[w];
            c.at = (uint32_t)w << kTokenBits | (0xffffffffu - (uint32_t)k);
        } else if (kind[w] == 0 || l != w * p.slices || e != 0) {
            return c;
        }
        c.score = ordered64(score);
        return c;
    };
    // What n heads reach, the n best candidates reach: they are collected, and narrowed down
    // once more, since one beam's may be most of them.
    for (int l = tid; l < lists; l += MT) head[l] = entry(l, l / p.slices, 0);
    __syncthreads();
    const uint32_t bound = block_bound(head, lists, p.n, &scratch[0]);
    auto collect = [&](const Cand& c) {
        const int k = atomicAdd(&s_n, 1);
        if (k < merge_cap(p.n)) cand[k] = c;
    };
    for (int l = tid; l < lists; l += MT)
        if (head[l].rough() >= bound) {
            collect(head[l]);
            s_list[atomicAdd(&s_lists, 1)] = (uint16_t)l;
        }
    __syncthreads();
    const int bits = 32 - __clz(p.n - 1);   // n <= 2^bits
    for (int i = tid; i < s_lists << bits; i += MT) {
        const int l = s_list[i >> bits], e = i & ((1 << bits) - 1);
        if (e == 0 || e >= p.n) continue;
        const Cand c = entry(l, head[l].at >> kTokenBits, e);
        if (c.rough() >= bound) collect(c);
    }
    __syncthreads();
    if (s_n > merge_cap(p.n)) {
        // Ties make them too many: from the lists of exactly the n best heads, what is not
        // behind the n-th of them.
        rank_all(head, lists, [&](int l, int rank) {
            if (rank < p.n && head[l].score) sel[rank] = l;
        });
        __syncthreads();
        if (tid == 0) s_n = 0;
        const Cand last = head[sel[p.n - 1]];
        __syncthreads();
        for (int i = tid; i < p.n * p.n; i += MT) {
            const int l = sel[i / p.n];
            const Cand c = entry(l, head[l].at >> kTokenBits, i % p.n);
            if (c.score && !better(last, c)) cand[atomicAdd(&s_n, 1)] = c;
        }
        __syncthreads();
    }
    int total = s_n;
    const Cand* from = cand;
    if (total > kFew) {
        const uint32_t closer = block_bound(cand, total, p.n, &scratch[1]);
        for (int i = tid; i < total; i += MT)
            if (cand[i].rough() >= closer) {
                const int k = atomicAdd(&s_few, 1);
                if (k < kFew) few[k] = cand[i];
            }
        __syncthreads();
        if (s_few <= kFew) {   // (else: ties)
            from = few;
            total = s_few;
        }
    }
    const int64_t out = (int64_t)blockIdx.x * p.n;
    rank_all(from, total, [&](int i, int rank) {
        if (rank >= p.n) return;
        p.parents[out + rank] = (int32_t)(from[i].at >> kTokenBits);
        p.tokens[out + rank] = (int32_t)(from[i].at & ((1u << kTokenBits) - 1u));
        p.out_scores[out + rank] = (float)from_ordered64(from[i].score);
    });
    for (int i = total + tid; i < p.n; i += MT) {
        p.parents[out + i] = -1;
        p.tokens[out + i] = -1;
        p.out_scores[out + i] = -INFINITY;
    }
}

}  // namespace beam
}  // namespace gdn
