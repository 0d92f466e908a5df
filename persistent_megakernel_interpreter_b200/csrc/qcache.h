// The 8-bit cache's geometry, shared by its kernels and entry points.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include <atomic>

#include "mk_internal.h"

namespace mk {

constexpr int kQBlock = MK_QCACHE_BLOCK;  // tokens that share one scale (of one head, of keys or of values)
constexpr int kQMaxHeads = 32;    // KV heads at most
constexpr int kQSms = 148;        // B200: sizes grids and workspaces without asking the device
// A block whose largest magnitude is below 2^-60 is held as zeros (scale 0): the
// attention divides by scales, and 127 / amax has to stay finite.
constexpr float kQNoBlock = 8.673617379884035e-19f;

// True the first time it is asked on the calling thread's current device (per flag word): for
// settings of a kernel that last as long as the process. Two threads may both be told so.
inline bool first_on_device(std::atomic<uint64_t>& seen) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev > 63) return true;
    return !(seen.load(std::memory_order_acquire) >> dev & 1);
}
inline void seen_on_device(std::atomic<uint64_t>& seen) {
    int dev = 0;
    if (cudaGetDevice(&dev) == cudaSuccess && dev >= 0 && dev < 64) seen.fetch_or(1ull << dev, std::memory_order_release);
}

#ifdef __CUDACC__
// A kernel that may be placed while the one before it in the stream still ends; each waits for
// all of it (cudaGridDependencySynchronize) before it reads or writes anything.
template <class... P, class... A>
cudaError_t launch_behind(void (*kernel)(P...), dim3 grid, int block, int smem, cudaStream_t st, A&&... args) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)block);
    cfg.dynamicSmemBytes = (size_t)smem;
    cfg.stream = st;
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}
#endif

inline int qcache_blocks(int max_seq) { return (max_seq + kQBlock - 1) / kQBlock; }

// MK_OK, or why the cache described by c is refused.
inline mk_status qcache_check(const mk_qcache* c) {
    if (!c || !c->k_codes || !c->v_codes || !c->k_scale || !c->v_scale || !c->k_tail || !c->v_tail)
        return MK_ERR_INVALID_ARG;
    if (c->n_layers < 1 || c->n_layers > kMaxLayers || c->max_batch < 1 || c->max_batch > kMaxBatch ||
        c->n_kv_heads < 1 || c->n_kv_heads > kQMaxHeads || c->max_seq < 1 || c->max_seq > (1 << 20) ||
        (c->head_dim != 64 && c->head_dim != 128))
        return MK_ERR_UNSUPPORTED;
    const uintptr_t wide = reinterpret_cast<uintptr_t>(c->k_codes) | reinterpret_cast<uintptr_t>(c->v_codes) |
                           reinterpret_cast<uintptr_t>(c->k_tail) | reinterpret_cast<uintptr_t>(c->v_tail);
    const uintptr_t narrow = reinterpret_cast<uintptr_t>(c->k_scale) | reinterpret_cast<uintptr_t>(c->v_scale);
    if ((wide & 15) || (narrow & 3)) return MK_ERR_INVALID_ARG;
    return MK_OK;
}

// A decode step on the 8-bit cache (baseline.cu): the step's parameters with the cache's
// one-slot buffers for the new key and value in kc / vc ([layer][sequence][head][dim]).
struct QcacheStep {
    Params params;
    const mk_qcache* cache;
    int32_t* positions;           // device [B], written by the step's checks
    int32_t* status_out;          // device or NULL
    void* attn_workspace;
    size_t attn_workspace_bytes;
};

}  // namespace mk
