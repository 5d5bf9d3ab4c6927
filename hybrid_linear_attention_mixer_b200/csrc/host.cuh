// Host-side helpers shared by the library's translation units: argument checks,
// the calling thread's last CUDA error, driver entry points, device properties.
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <cmath>
#include <mutex>

#include "gdn.h"

namespace gdn {
namespace host {

inline bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
inline size_t align_up(size_t x, size_t a) { return (x + a - 1) / a * a; }

inline bool dim_ok(int d) { return d == 32 || d == 64 || d == 128; }

// The CUDA error behind this thread's most recent GDN_ERR_CUDA (gdn_last_cuda_error).
inline thread_local cudaError_t t_last_cuda_error = cudaSuccess;

// GDN_OK for cudaSuccess; otherwise remembers e for this thread and returns GDN_ERR_CUDA.
// (The runtime's own last error is taken, or the next launch would be said to have failed.)
inline gdn_status cuda_status(cudaError_t e) {
    if (e == cudaSuccess) return GDN_OK;
    t_last_cuda_error = e;
    (void)cudaGetLastError();
    return GDN_ERR_CUDA;
}

// The prefill chunk gdn_config.chunk has to name (the intra-chunk kernel's row count).
constexpr int kChunkTokens = 64;

inline gdn_status check_config(const gdn_config* c) {
    if (!c) return GDN_ERR_INVALID_ARG;
    if (c->n_k_heads <= 0 || c->n_v_heads <= 0 || c->d_k <= 0 || c->d_v <= 0) return GDN_ERR_INVALID_ARG;
    if (!(c->l2_eps >= 0.f) || !(c->norm_eps >= 0.f) || !std::isfinite(c->l2_eps) ||
        !std::isfinite(c->norm_eps))
        return GDN_ERR_INVALID_ARG;
    if (c->act_dtype != GDN_BF16 && c->act_dtype != GDN_F32) return GDN_ERR_INVALID_ARG;
    if (c->out_dtype != GDN_BF16 && c->out_dtype != GDN_F32) return GDN_ERR_INVALID_ARG;
    if (c->state_dtype != GDN_BF16 && c->state_dtype != GDN_F32) return GDN_ERR_INVALID_ARG;
    if (c->n_v_heads % c->n_k_heads != 0) return GDN_ERR_UNSUPPORTED;
    if (!dim_ok(c->d_k) || !dim_ok(c->d_v)) return GDN_ERR_UNSUPPORTED;
    if (c->conv_kernel != 4 || c->chunk != kChunkTokens) return GDN_ERR_UNSUPPORTED;
    if (c->prefill_segments < GDN_PREFILL_SPLIT || c->prefill_segments > GDN_PREFILL_MAX_SEGMENTS)
        return GDN_ERR_INVALID_ARG;
    return GDN_OK;
}

// cuCtxGetCurrent, fetched once from the driver through the runtime.
inline PFN_cuCtxGetCurrent_v4000 ctx_getter() {
    static PFN_cuCtxGetCurrent_v4000 fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void* f = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPoint("cuCtxGetCurrent", &f, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<PFN_cuCtxGetCurrent_v4000>(f);
    });
    return fn;
}

// cuTensorMapEncodeTiled, fetched once from the driver through the runtime.  It
// is a driver call and needs a current context, which a host thread that has
// made no runtime call yet does not have: the current device's primary context
// is made current first in that case.
inline PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder() {
    static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void* f = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &f, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
    });
    CUcontext ctx = nullptr;
    auto get_ctx = ctx_getter();
    if (!get_ctx || get_ctx(&ctx) != CUDA_SUCCESS) return nullptr;
    if (!ctx) {
        int dev = 0;
        if (cudaGetDevice(&dev) != cudaSuccess || cudaSetDevice(dev) != cudaSuccess) return nullptr;
    }
    return fn;
}

// Streaming multiprocessors of the current device (cached per device).
inline int sm_count() {
    static int count[64];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return 148;
    if (dev < 64 && count[dev]) return count[dev];
    int n = 0;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0) n = 148;
    if (dev < 64) count[dev] = n;
    return n;
}

}  // namespace host

// serve.cu's half of gdn_check_device_error: reads and clears that module's
// device error word (the caller has synchronised the stream).
cudaError_t take_serve_error_word(unsigned int* word);

}  // namespace gdn
