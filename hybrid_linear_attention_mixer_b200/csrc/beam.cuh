// Beam search's selection over beams and vocabulary.
//   score(w, v) = S_w + x_wv - log sum_u exp(x_wu);  the n best of W * V, ties to the
//   lowest w * V + v.
//
// Within one row the order of the scores is the order of the logits, so one pass
// over the logits suffices: slice_kernel reads a slice of a row once, keeps it in
// registers, and leaves its sum of exponentials and its n largest logits;
// merge_kernel then joins a group's slices, adds the rows' offsets in fp64 and ranks
// the few candidates left.  Bound by reading the logits (a small group: by the
// latency of the two dependent launches).
//
// The selection in a slice: with every thread's largest logit known, any bound that
// n thread maxima reach is reached by at least n logits; a few bisection steps find
// one that not many more reach.  The vectors that reach it go to shared memory, where
// their logits are ranked exactly, by 64-bit keys (logit, then lowest index).  Where
// ties make that too many (a row of equal logits) the bound is found exactly, over
// logits and then over indexes, from a second reading of the slice.
#pragma once

#include "device.cuh"

namespace gdn {
namespace beam {

constexpr int NT = 256;             // threads of a slice block
constexpr int VECS = 256;           // 16-byte vectors a slice collects
constexpr int CAP = 512;            // candidates a slice ranks
constexpr int MT = 512;             // threads of a merge block
constexpr int kMaxBeams = GDN_BEAM_MAX_BEAMS;
constexpr int kMaxOut = GDN_BEAM_MAX_OUT;
static_assert(kMaxOut <= NT && NT <= CAP && kMaxOut <= MT, "candidate lists");

// A slice is NT * VPT vectors of 16 bytes.  A row's slices and the elements of a thread
// go by element number, wherever the row starts in memory: equal rows have bit-equal
// sums, so their candidates tie.
__host__ __device__ constexpr int slice_len(int elem_bytes, int vpt) { return NT * vpt * (16 / elem_bytes); }

// sum of exp(x) over a slice = sum * exp(ref).  sum is NaN where the slice holds a NaN or
// +inf, and 0 with ref = -inf where it holds nothing else than -inf.
struct Stat {
    double sum, ref;
};

struct Args {
    const void* logits;
    int64_t ld;
    const float* scores;
    const uint8_t* finished;   // or null
    int W, V, n, pad, slices;
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
    // (a maximum that ignores NaN, like fmaxf)
    static __device__ __forceinline__ float top(uint4 u) {
        const __nv_bfloat162 a = __hmax2(as2(u.x), as2(u.y)), b = __hmax2(as2(u.z), as2(u.w)), c = __hmax2(a, b);
        return __bfloat162float(__hmax(c.x, c.y));
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
    static __device__ __forceinline__ float top(uint4 u) {
        return fmaxf(fmaxf(__uint_as_float(u.x), __uint_as_float(u.y)), fmaxf(__uint_as_float(u.z), __uint_as_float(u.w)));
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

template <typename T, int VPT>
__global__ void __launch_bounds__(NT, 4) slice_kernel(const __grid_constant__ Args p) {
    using X = Vec<T>;
    constexpr int N = X::N;
    __shared__ float s_max[NT];
    __shared__ double s_sum[NT / 32];
    __shared__ int s_count[NT / 32];
    __shared__ uint4 s_vec[VECS];
    __shared__ int s_at[VECS];
    __shared__ uint64_t s_key[CAP];
    __shared__ int s_vecs, s_n;
    __shared__ float s_bound;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t row = blockIdx.x / p.slices;
    const int slice = blockIdx.x % p.slices;
    if (!row_live(p, row)) {
        grid_dependency_trigger();
        return;
    }
    const T* x = static_cast<const T*>(p.logits) + row * p.ld;
    const int first = slice * slice_len(sizeof(T), VPT) + tid * N;   // this thread's first element
    const int shift = (int)(reinterpret_cast<uintptr_t>(x) & 15u);
    constexpr int kStep = NT * N;

    uint4 v[VPT];
#pragma unroll
    for (int j = 0; j < VPT; ++j) v[j] = load_vec<T>(x, first + j * kStep, p.V, shift);
    float m = X::top(v[0]);
#pragma unroll
    for (int j = 1; j < VPT; ++j) m = fmaxf(m, X::top(v[j]));
    m = fmaxf(m, -INFINITY);   // (only NaN: they show in the sum)
    s_max[tid] = m;
    if (tid == 0) s_vecs = s_n = 0;
    __syncthreads();
    float mine[NT / 32], top = -INFINITY;
#pragma unroll
    for (int i = 0; i < NT / 32; ++i) {
        mine[i] = s_max[i * 32 + lane];
        top = fmaxf(top, mine[i]);
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));

    if (warp == 0) {   // a bound that at least n thread maxima reach and not many more
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
        uint32_t lo = ordered(-3.402823466e38f);
        if (valid > p.n) {   // at least n maxima reach lo, fewer reach anything above hi
            const int enough = p.n + 8;
            uint32_t hi = ordered(top);
            int at_lo = valid;
            lo = least;
            while (at_lo > enough && hi > lo) {
                const uint32_t mid = lo + (hi - lo + 1) / 2;
                const float b = from_ordered(mid);
                int c = 0;
#pragma unroll
                for (int i = 0; i < NT / 32; ++i) c += mine[i] >= b;
                c = __reduce_add_sync(0xffffffffu, c);
                if (c >= p.n) {
                    lo = mid;
                    at_lo = c;
                } else {
                    hi = mid - 1;
                }
            }
        }
        if (lane == 0) s_bound = from_ordered(lo);
    }

    // The slice's sum of exponentials, about a reference near its top.  exp(x - ref) is
    // 2^(x log2e - c), c an integer, in one fused operation for tops of ordinary size:
    // log2e in fp32 is 1.3e-8 off, which scales x; (x - top) log2e for others, whose x
    // that would move too far.
    double ref;
    float2 s2[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
    if (fabsf(top) <= 64.0f) {
        const float c = ceilf(top * kLog2e);
        ref = (double)c * kLn2;
#pragma unroll
        for (int j = 0; j < VPT; ++j)
#pragma unroll
            for (int e = 0; e < N / 2; ++e) {
                const float2 t = fma2(X::pair(v[j], e), make_float2(kLog2e, kLog2e), make_float2(-c, -c));
                s2[e & 1] = add2(s2[e & 1], make_float2(exp2_fast(t.x), exp2_fast(t.y)));
            }
    } else {
        ref = top;
#pragma unroll
        for (int j = 0; j < VPT; ++j)
#pragma unroll
            for (int e = 0; e < N / 2; ++e) {
                const float2 t = X::pair(v[j], e);
                // (-inf and nothing else: no sum, but a NaN has to show)
                s2[0].x += top > -INFINITY || isnan(t.x) ? exp2_fast((t.x - top) * kLog2e) : 0.0f;
                s2[0].y += top > -INFINITY || isnan(t.y) ? exp2_fast((t.y - top) * kLog2e) : 0.0f;
            }
    }
    double sum = ((double)s2[0].x + (double)s2[0].y) + ((double)s2[1].x + (double)s2[1].y);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
    if (lane == 0) s_sum[warp] = sum;
    __syncthreads();

    // the vectors that reach the bound, then their logits that do
    float bound = s_bound;
    if (m >= bound) {
#pragma unroll
        for (int j = 0; j < VPT; ++j)
            if (X::top(v[j]) >= bound) {
                const int k = atomicAdd(&s_vecs, 1);
                if (k < VECS) {
                    s_vec[k] = v[j];
                    s_at[k] = first + j * kStep;
                }
            }
    }
    if (tid == 0) {
        double t = 0.0;
        for (int i = 0; i < NT / 32; ++i) t += s_sum[i];
        p.stats[row * p.slices + slice] = Stat{t, ref};
    }
    __syncthreads();
    const int vecs = s_vecs;
    if (vecs <= VECS) {
        for (int i = tid; i < vecs * N; i += NT) {
            const int k = i / N, e = i % N;
            const float f = to_f32(reinterpret_cast<const T*>(&s_vec[k])[e]);
            if (f >= bound) {
                const int at = atomicAdd(&s_n, 1);
                if (at < CAP) s_key[at] = make_key(f, s_at[k] + e);
            }
        }
    }
    __syncthreads();
    if (vecs > VECS || s_n > CAP) {
        // Too many reach it.  The n-th largest logit itself ...
        auto count = [&](auto&& pred) {   // logits of the slice that pred(value, index) takes
            int c = 0;
#pragma unroll 1
            for (int j = 0; j < VPT; ++j) {
                const int i0 = first + j * kStep;
                const uint4 u = load_vec<T>(x, i0, p.V, shift);
#pragma unroll
                for (int e = 0; e < N; ++e) c += pred(X::get(u, e), i0 + e);
            }
            return block_count(c, s_count);
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
        int i_lo = 0, i_hi = p.V - 1;
        while (i_lo < i_hi) {
            const int mid = i_lo + (i_hi - i_lo) / 2;
            if (above + count([&](float f, int i) { return f == bound && i <= mid; }) >= p.n) i_hi = mid;
            else i_lo = mid + 1;
        }
        if (tid == 0) s_n = 0;
        __syncthreads();
#pragma unroll 1
        for (int j = 0; j < VPT; ++j) {
            const int i0 = first + j * kStep;
            const uint4 u = load_vec<T>(x, i0, p.V, shift);
#pragma unroll
            for (int e = 0; e < N; ++e) {
                const float f = X::get(u, e);
                if (f > bound || (f == bound && i0 + e <= i_lo)) s_key[atomicAdd(&s_n, 1)] = make_key(f, i0 + e);
            }
        }
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

// Shared memory of a merge block: list heads, then candidates.
inline size_t merge_smem(int W, int slices, int n) {
    return ((size_t)W * slices + (size_t)n * n) * sizeof(Cand);
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

    for (int w = warp; w < p.W; w += MT / 32) {
        const int64_t row = row0 + w;
        const float score = p.scores[row];
        const bool fin = p.finished && p.finished[row];
        double off = score, top = -INFINITY;
        if (!fin && isfinite(score)) {
            const Stat* st = p.stats + row * p.slices;
            for (int s = lane; s < p.slices; s += 32) top = fmax(top, st[s].ref);
#pragma unroll
            for (int d = 16; d > 0; d >>= 1) top = fmax(top, __shfl_xor_sync(0xffffffffu, top, d));
            double sum = 0.0;
            for (int s = lane; s < p.slices; s += 32)
                sum += st[s].ref > -INFINITY ? st[s].sum * exp(st[s].ref - top) : st[s].sum;
#pragma unroll
            for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
            off -= log(sum);   // (nothing but -inf: +inf; a NaN or +inf among the logits: NaN)
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
            const uint64_t k = p.cand[((row0 + w) * p.slices + l % p.slices) * p.n + e];
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
