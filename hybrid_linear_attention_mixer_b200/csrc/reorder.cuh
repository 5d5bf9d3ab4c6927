// Reordering of per-sequence states after a beam selection, in place: in each group
// of W sequences, slot w takes what slot parent[w] held.
//
// A block takes the same bytes of all W slots of one group in one buffer, so each
// thread reads the W sources of its 16-byte column into registers and then writes
// the slots that change: no slot is overwritten before it is read, whatever the
// parents, with no second buffer and no synchronisation.  Slots that keep their
// state are neither read nor written; a source that several slots take is read from
// HBM once (its further reads hit L1).  Bound by memory: 2 to 16 beams of 3 MiB states
// move at 4.5 to 6.5 TB/s of unique reads and writes (8 beams: 79 us; blocks of 256
// threads, with as many registers each, 123 us: too few of them fit on an SM).  Two beams
// take 8 vectors a thread (35 us, 56 with 4), since often only one slot moves.
#pragma once

#include "device.cuh"

namespace gdn {
namespace reorder {

constexpr int NT = 128;
constexpr int kMaxBuffers = GDN_REORDER_MAX_BUFFERS;

struct Buffer {
    uint4* base;
    int64_t stride;   // 16-byte units between sequences
    int32_t vecs;     // 16-byte units of a sequence's state
    int32_t item0;    // work items of the buffers before this one (per group)
};

struct Args {
    const int32_t* parents;
    int32_t W, n_buffers, items;   // items: work items of one group over all buffers
    int64_t total;                 // items x groups
    Buffer buf[kMaxBuffers];
};

// A parent: a coherent load (the selection before, which writes them, can still run when this
// kernel starts), issued in order (left to the compiler, two beams of one layer took up to
// 0.4 us more of 1.8).
__device__ __forceinline__ int ld_parent(const int32_t* p) {
    int v;
    asm volatile("ld.global.s32 %0, [%1];" : "=r"(v) : "l"(p));
    return v;
}

// Work item: NT * U vectors of one group's slots in one buffer.
template <int WMAX, int U>
__global__ void __launch_bounds__(NT) reorder_kernel(const __grid_constant__ Args p) {
    grid_dependency_trigger();
    grid_dependency_wait();
    for (int64_t it = blockIdx.x; it < p.total; it += gridDim.x) {
        const int64_t group = it / p.items;
        const int item = (int)(it % p.items);
        int par[WMAX];
        bool bad = false;
#pragma unroll
        for (int w = 0; w < WMAX; ++w) {
            par[w] = w < p.W ? ld_parent(p.parents + group * p.W + w) : -1;
            bad |= par[w] < -1 || par[w] >= p.W;
            if (par[w] == w) par[w] = -1;   // nothing to do
        }
        if (bad) {   // the same for the whole block, and for all blocks of the group
            if (threadIdx.x == 0) record_error(kErrIndex);
            continue;
        }
        int lo = 0, hi = p.n_buffers - 1;   // the last buffer whose items start at or before this one
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (p.buf[mid].item0 <= item) lo = mid;
            else hi = mid - 1;
        }
        const Buffer& b = p.buf[lo];
        const int v0 = (item - b.item0) * (NT * U) + threadIdx.x;
        uint4* slot = b.base + group * p.W * b.stride;
        uint4 val[U][WMAX];
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int w = 0; w < WMAX; ++w)
                if (par[w] >= 0 && v0 + u * NT < b.vecs) val[u][w] = slot[par[w] * b.stride + v0 + u * NT];
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int w = 0; w < WMAX; ++w)
                if (par[w] >= 0 && v0 + u * NT < b.vecs) slot[w * b.stride + v0 + u * NT] = val[u][w];
    }
}

}  // namespace reorder
}  // namespace gdn
