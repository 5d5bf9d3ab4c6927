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
// The slice is streamed without synchronisation: each thread keeps its largest logit and
// its sum of exponentials about a reference of its own.  Then, any bound that n thread
// maxima reach is reached by at least n logits; a few bisection steps find one that not
// many more reach.  The threads that reach it read their vectors once more (from L2), and
// the logits that do are ranked exactly, by 64-bit keys (logit, then lowest index).  Where
// ties make them too many (a row of equal logits), the bound is found exactly, over logits
// and then over indexes, by more such readings.
#pragma once

#include "device.cuh"

namespace gdn {
namespace beam {

constexpr int NT = 256;             // threads of a slice block
constexpr int VPT = 4;              // 16-byte vectors per thread of a tile
constexpr int CAP = 512;            // candidates a slice ranks
constexpr int MT = 512;             // threads of a merge block
constexpr int kMaxBeams = GDN_BEAM_MAX_BEAMS;
constexpr int kMaxOut = GDN_BEAM_MAX_OUT;
static_assert(kMaxOut <= NT && kMaxOut <= MT, "candidate lists");

// A tile is NT * VPT vectors of 16 bytes, a slice some tiles.  A row's slices and the
// elements of a thread go by element number, wherever the row starts in memory: equal
// rows have bit-equal sums, so their candidates tie.
__host__ __device__ constexpr int tile_len(int elem_bytes) { return NT * VPT * (16 / elem_bytes); }

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
    int W, V, n, pad, slices, tiles;   // tiles of a slice
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

__device__ __forceinline__ uint4 ld_once(const void* p) {
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
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

// Block-wide sum of small counts (every thread gets it).
__device__ __forceinline__ int block_count(int c, int* slot) {
    c = __reduce_add_sync(0xffffffffu, c);
    __syncthreads();   // the slots' last readers are done
    if ((threadIdx.x & 31) == 0) slot[threadIdx.x >> 5] = c;
    __syncthreads();
    int t = 0;
#pragma unroll
    for (int i = 0; i < NT / 32; ++i) t += slot[i];
    return t;
}

// A row is live when it can give candidates from its logits.
__device__ __forceinline__ bool row_live(const Args& p, int64_t row) {
    return !(p.finished && p.finished[row]) && isfinite(p.scores[row]);
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

// A bound that at least n of the NT thread maxima reach and not many more, by one warp
// that holds NT / 32 of them per lane; found only if more than n are above -inf.
__device__ __forceinline__ bool find_bound(const float (&mine)[NT / 32], float top, int n, float* bound) {
    int valid = 0;
    uint32_t least = 0xffffffffu;
#pragma unroll
    for (int i = 0; i < NT / 32; ++i) {
        if (mine[i] > -INFINITY) {
            ++valid;
            least = min(least, ordered(mine[i]));
        }
    }
    valid = __reduce_add_sync(0xffffffffu, valid);
    least = __reduce_min_sync(0xffffffffu, least);
    if (valid <= n) return false;
    uint32_t lo = least, hi = ordered(top);   // at least n reach lo, fewer reach anything above hi
    int at_lo = valid;
    while (at_lo > n + 8 && hi > lo) {
        const uint32_t mid = lo + (hi - lo + 1) / 2;
        const float b = from_ordered(mid);
        int c = 0;
#pragma unroll
        for (int i = 0; i < NT / 32; ++i) c += mine[i] >= b;
        c = __reduce_add_sync(0xffffffffu, c);
        if (c >= n) {
            lo = mid;
            at_lo = c;
        } else {
            hi = mid - 1;
        }
    }
    *bound = from_ordered(lo);
    return true;
}

// The fast sum: exp(x) / 2^c is 2^(x log2e - c) in one fused operation, c an integer near
// the largest x so far.  log2e in fp32 is 1.3e-8 (kScale) too large, which scales x: that
// is taken back at the slice's top, so what is left goes by the distance from it.
// kSpan: how far above c a maximum may lie; kMaxTop: the size of x up to which c is exact.
constexpr float kSpan = 32.0f, kMaxTop = 65536.0f;
constexpr double kScale = (double)kLog2e * kLn2 - 1.0;

// 2^k for an integer k <= 0 (0 below the normal numbers)
__device__ __forceinline__ double pow2(float k) {
    return k > -1000.0f ? __hiloint2double((1023 + (int)k) << 20, 0) : 0.0;
}

// A thread's largest logit and its sum of exponentials, in units of 2^c.
struct Running {
    float m = -INFINITY, c = -2.0f * kMaxTop;
    double sum = 0.0;
    template <typename T>
    __device__ __forceinline__ void add(const uint4 (&v)[VPT]) {
        const float tm = Vec<T>::top(v);   // (NaN show in the sum)
        m = fmaxf(m, tm);
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
    }
};

template <typename T>
__global__ void __launch_bounds__(NT, 4) slice_kernel(const __grid_constant__ Args p) {
    using X = Vec<T>;
    constexpr int N = X::N, kStep = NT * N, kTile = kStep * VPT;
    __shared__ float s_max[NT], s_c[NT / 32];
    __shared__ double s_sum[NT / 32];
    __shared__ int s_count[NT / 32];
    __shared__ int s_list[NT];       // first elements of the threads that reach the bound
    __shared__ uint64_t s_key[CAP];
    __shared__ int s_listed, s_n;
    __shared__ float s_bound;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t row = blockIdx.x / (unsigned)p.slices;
    const int slice = blockIdx.x % (unsigned)p.slices;
    if (!row_live(p, row)) {
        grid_dependency_trigger();
        return;
    }
    const T* x = static_cast<const T*>(p.logits) + row * p.ld;
    const int first = slice * p.tiles * kTile + tid * N;   // this thread's first element
    const int tiles = min(p.tiles, (p.V - slice * p.tiles * kTile + kTile - 1) / kTile);
    const int shift = (int)(reinterpret_cast<uintptr_t>(x) & 15u);

    auto load_tile = [&](uint4 (&u)[VPT], int t) {
        if (t >= tiles) return;
        const int i0 = first + t * kTile, tile0 = (slice * p.tiles + t) * kTile;
        if (shift == 0 && tile0 + kTile <= p.V) {
#pragma unroll
            for (int j = 0; j < VPT; ++j) u[j] = ld_once(x + i0 + j * kStep);
        } else {
#pragma unroll 1
            for (int j = 0; j < VPT; ++j) {
                const uint4 a = load_vec<T>(x, i0 + j * kStep, p.V, shift);
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
        run.add<T>(even);
        if (t + 1 >= tiles) break;
        load_tile(even, t + 2);
        run.add<T>(odd);
    }

    s_max[tid] = run.m;
    if (tid == 0) {
        s_listed = s_n = 0;
        s_bound = -3.402823466e38f;
    }
    float c = run.c;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) c = fmaxf(c, __shfl_xor_sync(0xffffffffu, c, d));
    double sum = run.sum * pow2(run.c - c);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
    if (lane == 0) {
        s_sum[warp] = sum;
        s_c[warp] = c;
    }
    __syncthreads();
    float mine[NT / 32], top = -INFINITY;
#pragma unroll
    for (int i = 0; i < NT / 32; ++i) {
        mine[i] = s_max[i * 32 + lane];
        top = fmaxf(top, mine[i]);
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
    const bool redo_sum = top > -INFINITY && !(fabsf(top) <= kMaxTop);
    const int finder = blockIdx.x % (NT / 32);   // (spreads this work over the schedulers)
    if (warp == finder) {
        float b;
        if (find_bound(mine, top, p.n, &b) && lane == 0) s_bound = b;
    } else if (warp == (finder + 1) % (NT / 32) && lane == 0 && !redo_sum) {
        float most = s_c[0];
        for (int i = 1; i < NT / 32; ++i) most = fmaxf(most, s_c[i]);
        double t = 0.0;
        for (int i = 0; i < NT / 32; ++i) t += s_sum[i] * pow2(s_c[i] - most);
        p.stats[row * p.slices + slice] = Stat{t, most, top};
    }
    __syncthreads();
    float bound = s_bound;
    auto each_vec = [&](auto&& use) {   // use(vector, index) for the thread's vectors of the slice
#pragma unroll 1
        for (int t = 0; t < tiles; ++t)
#pragma unroll 1
            for (int j = 0; j < VPT; ++j) {
                const int i0 = first + t * kTile + j * kStep;
                use(load_vec<T>(x, i0, p.V, shift), i0);
            }
    };
    if (redo_sum) {   // about the top itself
        sum = 0.0;
        each_vec([&](uint4 u, int) {
            float part = 0.0f;
#pragma unroll
            for (int e = 0; e < N; ++e) part += exp2_fast((X::get(u, e) - top) * kLog2e);
            sum += (double)part;
        });
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
        if (lane == 0) s_sum[warp] = sum;
        __syncthreads();
        if (tid == 0) {
            double t = 0.0;
            for (int i = 0; i < NT / 32; ++i) t += s_sum[i];
            p.stats[row * p.slices + slice] = Stat{t, __int_as_float(0x7fffffff), top};
        }
    }

    // the threads that reach the bound, and of their vectors the logits that do
    if (run.m >= bound) s_list[atomicAdd(&s_listed, 1)] = first;
    __syncthreads();
    const int per = tiles * VPT;
    for (int i = tid; i < s_listed * per; i += NT) {
        const int i0 = s_list[i / per] + i % per * kStep;   // (kTile is VPT kStep)
        const uint4 u[1] = {load_vec<T>(x, i0, p.V, shift)};
        if (X::top(u) >= bound) {
#pragma unroll
            for (int e = 0; e < N; ++e) {
                const float f = X::get(u[0], e);
                if (f >= bound) {
                    const int at = atomicAdd(&s_n, 1);
                    if (at < CAP) s_key[at] = make_key(f, i0 + e);
                }
            }
        }
    }
    __syncthreads();
    if (s_n > CAP) {
        // Too many reach it.  The n-th largest logit itself ...
        auto each = [&](auto&& use) {   // use(value, index)
            each_vec([&](uint4 u, int i0) {
#pragma unroll
                for (int e = 0; e < N; ++e) use(X::get(u, e), i0 + e);
            });
        };
        auto count = [&](auto&& pred) {
            int n = 0;
            each([&](float f, int i) { n += pred(f, i); });
            return block_count(n, s_count);
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
        int i_lo = slice * p.tiles * kTile, i_hi = min(p.V, i_lo + tiles * kTile) - 1;
        while (i_lo < i_hi) {
            const int mid = i_lo + (i_hi - i_lo) / 2;
            if (above + count([&](float f, int i) { return f == bound && i <= mid; }) >= p.n) i_hi = mid;
            else i_lo = mid + 1;
        }
        if (tid == 0) s_n = 0;
        __syncthreads();
        each([&](float f, int i) {
            if (f > bound || (f == bound && i <= i_lo)) s_key[atomicAdd(&s_n, 1)] = make_key(f, i);
        });
        __syncthreads();
    }
    grid_dependency_trigger();   // (the merge may be set up; it waits for this grid's end)
    const int total = s_n;
    uint64_t* out = p.cand + (row * p.slices + slice) * p.n;
    for (int i = tid; i < total; i += NT) {
        const uint64_t k = s_key[i];
        int rank = 0;
        for (int j = 0; j < total; ++j) rank += s_key[j] > k;
        if (rank < p.n) out[rank] = k;
    }
    for (int i = total + tid; i < p.n; i += NT) out[i] = 0;
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
struct Cand {
    uint64_t score;   // ordered; 0: none
    uint32_t at;      // w * V + v
    uint32_t unused;
};
__device__ __forceinline__ bool better(const Cand& a, const Cand& b) {
    return a.score > b.score || (a.score == b.score && a.at < b.at);
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

// Shared memory of a merge block: list heads, candidates, then the group's keys if they
// are held there (up to kMaxKeyBytes).
constexpr size_t kMaxKeyBytes = 64 * 1024;
constexpr int kMaxLists = 4096;        // of a group
constexpr size_t kMaxMergeSmem = (kMaxLists + (size_t)kMaxOut * kMaxOut) * sizeof(Cand) + kMaxKeyBytes;
static_assert(kMaxMergeSmem <= 225 * 1024, "shared memory of the merge");
inline size_t merge_key_bytes(int W, int slices, int n) { return (size_t)W * slices * n * sizeof(uint64_t); }
inline size_t merge_smem(int W, int slices, int n) {
    const size_t keys = merge_key_bytes(W, slices, n);
    return ((size_t)W * slices + (size_t)n * n) * sizeof(Cand) + (keys <= kMaxKeyBytes ? keys : 0);
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
    __shared__ int s_n;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t row0 = (int64_t)blockIdx.x * p.W;
    const int lists = p.W * p.slices;
    if (tid < kMaxOut) sel[tid] = -1;
    if (tid == 0) s_n = 0;
    grid_dependency_wait();
    const uint64_t* keys = p.cand + row0 * p.slices * p.n;
    if (p.keys_in_smem) {   // (of rows that left none too: whatever is there is not used)
        uint64_t* mine = reinterpret_cast<uint64_t*>(cand + p.n * p.n);
        for (int i = tid; i < lists * p.n; i += MT) mine[i] = keys[i];
        keys = mine;
    }

    for (int w = warp; w < p.W; w += MT / 32) {
        const int64_t row = row0 + w;
        const float score = p.scores[row];
        const bool fin = p.finished && p.finished[row];
        double off = score;
        float top = -INFINITY;
        if (!fin && isfinite(score)) {
            const Stat* st = p.stats + row * p.slices;
            float c = -INFINITY;
            bool fast = true;
            for (int s = lane; s < p.slices; s += 32) {
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
            double sum = 0.0;   // of exp(x) / (2^c exp(-top kScale)), or / exp(top)
            for (int s = lane; s < p.slices; s += 32) {
                const Stat t = st[s];
                double f = 0.0;   // (no logits: t.sum is 0, or the NaN that has to show)
                if (!(t.top > -INFINITY)) f = 1.0;
                else if (fast)   // (exp of a number below 2e-3, and of 1e-6 where it matters)
                    f = pow2(t.c - c) * (1.0 - ((double)t.top - (double)top) * kScale);
                else f = exp((isnan(t.c) ? (double)t.top : (double)t.c * kLn2 - (double)t.top * kScale) - (double)top);
                sum += t.sum * f;
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
    __syncthreads();
    // Entry e of list l: beam l / slices, slice l % slices.  A finished beam's one entry is
    // the first of its first list.
    auto entry = [&](int l, int e) {
        const int w = l / p.slices;
        Cand c{0, 0, 0};
        if (kind[w] == 1) {
            const uint64_t k = keys[l * p.n + e];
            if (k) {
                c.score = ordered64(((double)from_ordered((uint32_t)(k >> 32)) - ref[w]) + offset[w]);
                c.at = (uint32_t)w * p.V + (0xffffffffu - (uint32_t)k);
            }
        } else if (kind[w] == 2 && l % p.slices == 0 && e == 0) {
            c.score = ordered64(offset[w]);
            c.at = (uint32_t)w * p.V + p.pad;
        }
        return c;
    };
    for (int l = tid; l < lists; l += MT) head[l] = entry(l, 0);
    __syncthreads();

    // The n best heads: the n best candidates are in their lists, at or above the n-th of them.
    rank_all(head, lists, [&](int l, int rank) {
        if (rank < p.n && head[l].score) sel[rank] = l;
    });
    __syncthreads();
    // (fewer lists than results: no bound)
    const Cand least = sel[p.n - 1] < 0 ? Cand{0, 0xffffffffu, 0} : head[sel[p.n - 1]];
    for (int i = tid; i < p.n * p.n; i += MT) {
        const int l = sel[i / p.n];
        if (l < 0) continue;
        const Cand c = entry(l, i % p.n);
        if (c.score && !better(least, c)) cand[atomicAdd(&s_n, 1)] = c;
    }
    __syncthreads();
    const int total = s_n;
    const int64_t out = (int64_t)blockIdx.x * p.n;
    rank_all(cand, total, [&](int i, int rank) {
        if (rank >= p.n) return;
        p.parents[out + rank] = (int32_t)(cand[i].at / (uint32_t)p.V);
        p.tokens[out + rank] = (int32_t)(cand[i].at % (uint32_t)p.V);
        p.out_scores[out + rank] = (float)from_ordered64(cand[i].score);
    });
    for (int i = total + tid; i < p.n; i += MT) {
        p.parents[out + i] = -1;
        p.tokens[out + i] = -1;
        p.out_scores[out + i] = -INFINITY;
    }
}

}  // namespace beam
}  // namespace gdn
