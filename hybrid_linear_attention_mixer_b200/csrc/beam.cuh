// Beam search's selection over beams and vocabulary.
//   score(w, v) = S_w + x_wv - log sum_u exp(x_wu);  the n best of W * V, ties to the
//   lowest w * V + v.
//
// Within one row the order of the scores is the order of the logits, so one pass
// over the logits suffices: slice_kernel reads a slice of a row once, keeps it in
// registers, and leaves its (max, sum of exponentials) and its n largest logits;
// merge_kernel then joins a group's slices, adds the rows' offsets in fp64 and ranks
// the few candidates left.  Bound by reading the logits (a small group: by the
// latency of the two dependent launches).
//
// The selection in a slice: with every thread's largest logit known, any bound that
// n thread maxima reach is reached by at least n logits; a few bisection steps find
// one that not many more reach.  What reaches it is collected and ranked exactly, by
// 64-bit keys (logit, then lowest index).  Where ties make that too many (a row of
// equal logits) the bound is found exactly, over logits and then over indexes.
#pragma once

#include "device.cuh"

namespace gdn {
namespace beam {

constexpr int NT = 256;             // threads of a slice block
constexpr int VPT = 8;              // 16-byte vectors per thread
constexpr int CAP = 512;            // candidates a slice ranks directly
constexpr int MT = 1024;            // threads of a merge block
constexpr int kMaxBeams = GDN_BEAM_MAX_BEAMS;
constexpr int kMaxOut = GDN_BEAM_MAX_OUT;
static_assert(kMaxOut <= NT && NT <= CAP, "candidate lists");

template <typename T>
__host__ __device__ constexpr int slice_len() { return NT * VPT * (16 / (int)sizeof(T)); }

// A row's slices and the elements of a thread go by element number, wherever the
// row starts in memory: equal rows have bit-equal sums, so their candidates tie.
template <typename T>
__host__ __device__ constexpr int n_slices(int V) {
    return (V + slice_len<T>() - 1) / slice_len<T>();
}

struct Stat {      // of a slice
    double sum;    // sum of exp(x - max); NaN where the slice holds a NaN or +inf
    float max;
    float unused;
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

// 16 bytes of logits as loaded.
template <typename T>
struct Vec;
template <>
struct Vec<__nv_bfloat16> {
    static constexpr int N = 8;
    uint4 u;
    __device__ __forceinline__ float get(int i) const {
        const uint32_t w = i < 2 ? u.x : i < 4 ? u.y : i < 6 ? u.z : u.w;
        return __uint_as_float((i & 1) ? (w & 0xffff0000u) : (w << 16));
    }
    __device__ __forceinline__ void set_none() { u = make_uint4(0xff80ff80u, 0xff80ff80u, 0xff80ff80u, 0xff80ff80u); }
    __device__ __forceinline__ void set(int i, __nv_bfloat16 x) {
        const uint32_t b = __bfloat16_as_ushort(x);
        uint32_t& w = i < 2 ? u.x : i < 4 ? u.y : i < 6 ? u.z : u.w;
        w = (i & 1) ? ((w & 0xffffu) | (b << 16)) : ((w & 0xffff0000u) | b);
    }
};
template <>
struct Vec<float> {
    static constexpr int N = 4;
    uint4 u;
    __device__ __forceinline__ float get(int i) const {
        return __uint_as_float(i == 0 ? u.x : i == 1 ? u.y : i == 2 ? u.z : u.w);
    }
    __device__ __forceinline__ void set_none() { u = make_uint4(0xff800000u, 0xff800000u, 0xff800000u, 0xff800000u); }
    __device__ __forceinline__ void set(int i, float x) {
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

template <typename T>
__global__ void __launch_bounds__(NT) slice_kernel(const __grid_constant__ Args p) {
    constexpr int EPV = Vec<T>::N;
    __shared__ float s_max[NT];
    __shared__ double s_sum[NT / 32];
    __shared__ int s_count[NT / 32];
    __shared__ uint64_t s_key[CAP];
    __shared__ int s_n;
    __shared__ float s_bound;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t row = blockIdx.x / p.slices;
    const int slice = blockIdx.x % p.slices;
    if (!row_live(p, row)) {
        grid_dependency_trigger();
        return;
    }
    const T* x = static_cast<const T*>(p.logits) + row * p.ld;
    const int first = slice * slice_len<T>() + tid * EPV;   // this thread's first element
    const int shift = (int)(reinterpret_cast<uintptr_t>(x) & 15u);
    const int skew = shift / (int)sizeof(T);

    Vec<T> v[VPT];
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
        const int i0 = first + j * NT * EPV;
        if (i0 >= skew && i0 + (skew ? 2 * EPV - skew : EPV) <= p.V) {   // the loads stay within the row
            v[j].u = skew ? ld_shifted(reinterpret_cast<const uint8_t*>(x + i0) - shift, shift) : ld_once(x + i0);
        } else {
            v[j].set_none();
#pragma unroll
            for (int e = 0; e < EPV; ++e)
                if (i0 + e < p.V) v[j].set(e, x[i0 + e]);
        }
    }
    float m = -INFINITY;
#pragma unroll
    for (int j = 0; j < VPT; ++j)
#pragma unroll
        for (int e = 0; e < EPV; ++e) m = fmaxf(m, v[j].get(e));   // (a NaN shows in the sum)
    // The thread's sum of exp(x - m); where m = -inf, zero, or the NaN that is there.
    float sum = 0.0f;
    if (m > -INFINITY) {
#pragma unroll
        for (int j = 0; j < VPT; ++j)
#pragma unroll
            for (int e = 0; e < EPV; ++e) sum += exp2_fast((v[j].get(e) - m) * kLog2e);
    } else {
#pragma unroll
        for (int j = 0; j < VPT; ++j)
#pragma unroll
            for (int e = 0; e < EPV; ++e)
                if (isnan(v[j].get(e))) sum = v[j].get(e);
    }
    s_max[tid] = m;
    if (tid == 0) s_n = 0;
    __syncthreads();
    float top = -INFINITY;
#pragma unroll
    for (int i = 0; i < NT / 32; ++i) top = fmaxf(top, s_max[i * 32 + lane]);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
    // (m - top in fp32 is exact enough: it scales a sum that is below 2^-24 of the whole
    // where the difference is large)
    double part = m > -INFINITY ? (double)sum * (double)exp2f((m - top) * kLog2e) : (double)sum;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) part += __shfl_xor_sync(0xffffffffu, part, d);
    if (lane == 0) s_sum[warp] = part;

    // warp 0: a bound that at least n thread maxima reach and not many more
    if (warp == 0) {
        float mine[NT / 32];
        int valid = 0;
        uint32_t least = 0xffffffffu;
#pragma unroll
        for (int i = 0; i < NT / 32; ++i) {
            mine[i] = s_max[i * 32 + lane];
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
    __syncthreads();
    if (tid == 0) {
        double t = 0.0;
        for (int i = 0; i < NT / 32; ++i) t += s_sum[i];
        const int64_t at = row * p.slices + slice;
        p.stats[at] = Stat{t, top, 0.0f};
    }

    float bound = s_bound;
    int reach = 0;
    if (m >= bound) {
#pragma unroll
        for (int j = 0; j < VPT; ++j)
#pragma unroll
            for (int e = 0; e < EPV; ++e) reach += v[j].get(e) >= bound;
    }
    int total = block_count(reach, s_count);
    int last = 0x7fffffff;   // of the logits equal to the bound, those up to this index count
    if (total > CAP) {
        // the n-th largest logit itself ...
        uint32_t lo = ordered(bound), hi = ordered(top);
        while (hi > lo) {
            const uint32_t mid = lo + (hi - lo + 1) / 2;
            const float b = from_ordered(mid);
            int c = 0;
#pragma unroll
            for (int j = 0; j < VPT; ++j)
#pragma unroll
                for (int e = 0; e < EPV; ++e) c += v[j].get(e) >= b;
            if (block_count(c, s_count) >= p.n) lo = mid;
            else hi = mid - 1;
        }
        bound = from_ordered(lo);
        // ... and the index of the last one of its kind that is still among the n
        int above = 0;
#pragma unroll
        for (int j = 0; j < VPT; ++j)
#pragma unroll
            for (int e = 0; e < EPV; ++e) above += v[j].get(e) > bound;
        above = block_count(above, s_count);
        int i_lo = 0, i_hi = p.V - 1;
        while (i_lo < i_hi) {
            const int mid = i_lo + (i_hi - i_lo) / 2;
            int c = 0;
#pragma unroll
            for (int j = 0; j < VPT; ++j)
#pragma unroll
                for (int e = 0; e < EPV; ++e) c += v[j].get(e) == bound && first + j * NT * EPV + e <= mid;
            if (above + block_count(c, s_count) >= p.n) i_hi = mid;
            else i_lo = mid + 1;
        }
        last = i_lo;
    }
    if (m >= bound) {
#pragma unroll
        for (int j = 0; j < VPT; ++j)
#pragma unroll
            for (int e = 0; e < EPV; ++e) {
                const float f = v[j].get(e);
                const int i = first + j * NT * EPV + e;
                if (f > bound || (f == bound && i <= last)) s_key[atomicAdd(&s_n, 1)] = make_key(f, i);
            }
    }
    __syncthreads();
    grid_dependency_trigger();   // (the merge may be set up; it waits for this grid's end)
    total = s_n;
    uint64_t* out = p.cand + (row * p.slices + slice) * p.n;
    for (int i = tid; i < total; i += NT) {
        const uint64_t k = s_key[i];
        int rank = 0;
        for (int j = 0; j < total; ++j) rank += s_key[j] > k;
        if (rank < p.n) out[rank] = k;
    }
    for (int i = total + tid; i < p.n; i += NT) out[i] = 0;
}

// One candidate of a group: better() is the order of the results.
struct Cand {
    double score;
    int64_t at;   // w * V + v; -1: none
};
__device__ __forceinline__ bool better(const Cand& a, const Cand& b) {
    return a.score > b.score || (a.score == b.score && a.at < b.at);
}

// Shared memory of a merge block: list heads, then candidates.
inline size_t merge_smem(int W, int slices, int n) {
    return ((size_t)W * slices + (size_t)n * n) * sizeof(Cand);
}

// Entry e of list l (beam l / slices, slice l % slices) of the group.
__device__ __forceinline__ Cand list_entry(const Args& p, int64_t row0, int l, int e, const double* offset,
                                           const uint8_t* ended) {
    const int w = l / p.slices;
    Cand c{-INFINITY, -1};
    if (ended[w]) {   // one candidate, in its first slice's list
        if (l % p.slices == 0 && e == 0 && isfinite(offset[w])) c = Cand{offset[w], (int64_t)w * p.V + p.pad};
        return c;
    }
    if (!isfinite(offset[w])) return c;
    const uint64_t k = p.cand[((row0 + w) * p.slices + l % p.slices) * p.n + e];
    if (k) c = Cand{offset[w] + (double)from_ordered((uint32_t)(k >> 32)), (int64_t)w * p.V + (0xffffffffu - (uint32_t)k)};
    return c;
}

// One block per group.
__global__ void __launch_bounds__(MT) merge_kernel(const __grid_constant__ Args p) {
    extern __shared__ __align__(16) uint8_t smem[];
    Cand* head = reinterpret_cast<Cand*>(smem);
    Cand* cand = head + p.W * p.slices;
    __shared__ double offset[kMaxBeams];   // score - log-sum-exp, or the score of a finished beam
    __shared__ uint8_t ended[kMaxBeams];
    __shared__ int sel[kMaxOut];           // the lists of the n best heads, best first
    __shared__ int s_n;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t row0 = (int64_t)blockIdx.x * p.W;
    const int lists = p.W * p.slices;
    grid_dependency_wait();

    for (int w = warp; w < p.W; w += MT / 32) {
        const int64_t row = row0 + w;
        const bool fin = p.finished && p.finished[row];
        double off = p.scores[row];
        if (!fin && row_live(p, row)) {
            float top = -INFINITY;
            for (int s = lane; s < p.slices; s += 32) top = fmaxf(top, p.stats[row * p.slices + s].max);
#pragma unroll
            for (int d = 16; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
            double sum = 0.0;
            for (int s = lane; s < p.slices; s += 32) {
                const Stat t = p.stats[row * p.slices + s];
                sum += t.max > -INFINITY ? t.sum * exp((double)t.max - (double)top) : t.sum;
            }
#pragma unroll
            for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
            off -= (double)top + log(sum);   // (top = +-inf or a NaN in the sum: not finite)
        }
        if (lane == 0) {
            offset[w] = off;
            ended[w] = fin;
        }
    }
    if (tid < kMaxOut) sel[tid] = -1;
    if (tid == 0) s_n = 0;
    __syncthreads();
    for (int l = tid; l < lists; l += MT) head[l] = list_entry(p, row0, l, 0, offset, ended);
    __syncthreads();

    // The n best heads: the n best candidates are in their lists, at or above the n-th of them.
    for (int l = tid; l < lists; l += MT) {
        const Cand c = head[l];
        if (c.at < 0) continue;
        int rank = 0;
        for (int j = 0; j < lists && rank < p.n; ++j) rank += better(head[j], c);
        if (rank < p.n) sel[rank] = l;
    }
    __syncthreads();
    const bool all = sel[p.n - 1] < 0;   // fewer lists than results: no bound
    const Cand least = all ? Cand{-INFINITY, -1} : head[sel[p.n - 1]];
    for (int i = tid; i < p.n * p.n; i += MT) {
        const int l = sel[i / p.n];
        if (l < 0) continue;
        const Cand c = list_entry(p, row0, l, i % p.n, offset, ended);
        if (c.at >= 0 && (all || !better(least, c))) cand[atomicAdd(&s_n, 1)] = c;
    }
    __syncthreads();
    const int total = s_n;
    const int64_t out = (int64_t)blockIdx.x * p.n;
    for (int i = tid; i < total; i += MT) {
        const Cand c = cand[i];
        int rank = 0;
        for (int j = 0; j < total && rank < p.n; ++j) rank += better(cand[j], c);
        if (rank < p.n) {
            p.parents[out + rank] = (int32_t)(c.at / p.V);
            p.tokens[out + rank] = (int32_t)(c.at % p.V);
            p.out_scores[out + rank] = (float)c.score;
        }
    }
    for (int i = total + tid; i < p.n; i += MT) {
        p.parents[out + i] = -1;
        p.tokens[out + i] = -1;
        p.out_scores[out + i] = -INFINITY;
    }
}

}  // namespace beam
}  // namespace gdn
