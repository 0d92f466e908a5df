// The multi-kernel "bubble" baseline: the same decode step as one ordinary
// kernel per op and layer (about six launches per layer), the structure the
// megakernel write-ups measure against (the "Look Ma, No Bubbles" summaries,
// section "Memory Pipeline Bubbles Explained": every kernel boundary waits for
// stragglers, pays launch and teardown, and cannot prefetch the next op's
// weights). It uses the very same tile, epilogue and attention routines as the
// megakernel, with weights read straight from global memory, so the two give
// bit-identical results. Capturable in a CUDA graph.
#include <cuda_runtime.h>

#include "mk_device.cuh"
#include "qcache.h"

namespace mk {

constexpr int kBaseWarps = 8;
constexpr int kBaseThreads = 32 * kBaseWarps;
static_assert(kBaseThreads == kNT, "the block-level input routines assume the megakernel's compute warps");

__device__ __forceinline__ bool step_failed(const Params& p) {
    return ld_volatile_u32(&p.ctl->status) != 0u;
}

// Token and position checks, once per step, before any other kernel.
__global__ void k_validate(const __grid_constant__ Params p) {
    if (threadIdx.x != 0 || step_failed(p)) return;
    for (int b = 0; b < p.B; ++b) {
        const int tok = p.tokens[b], pos = p.positions[b];
        uint32_t code = 0;
        if (tok < 0 || tok >= p.V) code = MK_ERR_BAD_TOKEN;
        else if (pos < 0 || pos >= p.max_seq || pos + 1 > p.max_ctx) code = MK_ERR_BAD_POSITION;
        if (code) {
            if (atomicCAS(&p.ctl->status, 0u, code) == 0u) {
                p.ctl->info[0] = 0xffffffffu;
                p.ctl->info[1] = b;
                p.ctl->info[2] = (uint32_t)tok;
                p.ctl->info[3] = (uint32_t)pos;
            }
            return;
        }
    }
}

// The same checks for a step on the 8-bit cache, whose control block and status start
// here. `ok` receives the positions the cache's kernels go by: a failed step's are -1 for
// every row, which stores nothing.
__global__ void k_validate_qcache(const __grid_constant__ Params p, int cache_seq, int32_t* ok, int32_t* status_out) {
    if (threadIdx.x != 0) return;
    uint32_t code = 0;
    for (int b = 0; b < p.B && code == 0; ++b) {
        const int tok = p.tokens[b], pos = p.positions[b];
        if (tok < 0 || tok >= p.V) code = MK_ERR_BAD_TOKEN;
        else if (pos < 0 || pos >= p.max_seq || pos >= cache_seq || pos >= p.max_ctx) code = MK_ERR_BAD_POSITION;
    }
    for (int b = 0; b < p.B; ++b) ok[b] = code ? -1 : p.positions[b];
    p.ctl->status = code;
    if (status_out) *status_out = (int32_t)code;
}

__device__ __forceinline__ const uint8_t* op_tiles(const Params& p, int op, int l) {
    const size_t lb = p.off_layer0 + (size_t)l * p.layer_stride;
    switch (op) {
        case MK_OP_QKV: return p.packed + lb + p.rel_qkv;
        case MK_OP_OPROJ: return p.packed + lb + p.rel_o;
        case MK_OP_GATEUP: return p.packed + lb + p.rel_gu;
        default: return p.packed;  // LM head: the embedding table
    }
}

// One matvec op of one layer. The CTA first builds each sequence's input vector
// in shared memory (RMSNorm where the op has one) with the same block routine as
// the megakernel; then each warp takes tiles.
//
// STEP_KV: the new key and value go to slot 0 of a one-slot buffer (p.max_seq == 1)
// instead of the cache slot of their position.
template <int OP, int KC, int HD, bool STEP_KV = false>
__global__ void __launch_bounds__(kBaseThreads) k_tiles(const __grid_constant__ Params p, int l,
                                                        uint32_t ntiles, uint32_t tile_bytes) {
    if (step_failed(p)) return;
    extern __shared__ __align__(16) float xs_all[];  // [B][KC*256], then kConsumerWarps floats
    constexpr int N = KC * 256;
    const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
    float* red = xs_all + (size_t)p.B * N;
    auto bar = []() {
        __syncthreads();
        return true;
    };
    for (int b = 0; b < p.B; ++b) {
        const float* sf = nullptr;
        const uint16_t* sh = nullptr;
        const uint16_t* w = nullptr;
        if (OP == MK_OP_QKV) {
            w = norm_ptr(p, p.off_norms + (size_t)(2 * l) * p.H * 2);
            if (l == 0) sh = embed_row(p, b);
            else sf = p.x + (size_t)b * p.H;
        } else if (OP == MK_OP_GATEUP) {
            w = norm_ptr(p, p.off_norms + (size_t)(2 * l + 1) * p.H * 2);
            sf = p.x + (size_t)b * p.H;
        } else if (OP == MK_OP_OPROJ) {
            sf = p.attn + (size_t)b * p.Q;
        } else {
            w = norm_ptr(p, p.off_norms + (size_t)(2 * p.L) * p.H * 2);
            sf = p.x + (size_t)b * p.H;
        }
        block_input_plain(sf, sh, w, p.eps, N, xs_all + (size_t)b * N, red, t, warp, lane, bar);
    }
    const uint32_t gw = blockIdx.x * kBaseWarps + warp;
    const uint32_t nw = gridDim.x * kBaseWarps;
    const uint64_t pol = l2_evict_first_policy();
    const uint8_t* base = op_tiles(p, OP, l);
    for (uint32_t tl = gw; tl < ntiles; tl += nw) {
        for (int b = 0; b < p.B; ++b) {
            float4* v = reinterpret_cast<float4*>(xs_all + (size_t)b * N);
            const XSmem<KC> x{v, v + KC * 32};
            float acc[4];
            dot4<KC, false>(base + (size_t)tl * tile_bytes, x, acc, lane, pol);
            RopeRow rr{nullptr, nullptr, 0};
            if constexpr (OP == MK_OP_QKV) rr = rope_row_global(p, b);
            if constexpr (STEP_KV) rr.pos = 0;
            tile_epilogue<OP, HD>(p, l, b, tl, acc, lane, rr);
        }
    }
}

template <int KF>
__global__ void __launch_bounds__(kBaseThreads) k_down(const __grid_constant__ Params p, int l) {
    if (step_failed(p)) return;
    const int lane = threadIdx.x & 31;
    const uint32_t gw = blockIdx.x * kBaseWarps + (threadIdx.x >> 5);
    const uint32_t nw = gridDim.x * kBaseWarps;
    const uint64_t pol = l2_evict_first_policy();
    const uint8_t* base = p.packed + p.off_layer0 + (size_t)l * p.layer_stride + p.rel_down;
    const uint32_t nrb = p.H / 4;
    for (uint32_t rb = gw; rb < nrb; rb += nw) {
        for (int b = 0; b < p.B; ++b) {
            float tot[4];
            XRegs<KF> x;
            for (int c = 0; c < 4; ++c) {
                load_vec<KF>(p.hbuf + (size_t)b * p.F + (size_t)c * (p.F / 4), x, lane);
                float acc[4];
                dot4<KF, false>(base + ((size_t)rb * 4 + c) * p.tile_f, x, acc, lane, pol);
#pragma unroll
                for (int k = 0; k < 4; ++k) tot[k] = (c == 0) ? acc[k] : tot[k] + acc[k];
            }
            residual_epilogue(p, false, b, rb, tot, lane);
        }
    }
}

// Rows of one item in the baseline's shared memory: kpad is the partition
// length rounded up to 16 keys (a multiple of every key-class count). All rows,
// the key at pos included, are read from the cache, in the same order of
// arithmetic as the megakernel's rows (whose last row, the key at pos, comes
// from the step's own k/v).
__host__ __device__ inline int attn_kpad(int part_keys) { return (part_keys + 15) / 16 * 16; }

template <int HD>
__host__ __device__ inline size_t attn_item_smem(int G, int kpad) {
    return (size_t)align16((uint32_t)(G * HD * 4)) + 2 * (size_t)kpad * HD * 2 + (size_t)attn_scratch_floats(HD) * 4;
}

// One attention item per CTA: the item's rows (keys first .. first + n - 1, the
// key at pos included, which the QKV kernel has written) are copied into shared
// memory as one fill, then the same four phases as the megakernel run on them.
template <int HD>
__global__ void __launch_bounds__(kBaseThreads) k_attn_item(const __grid_constant__ Params p, int l) {
    if (step_failed(p)) return;
    extern __shared__ __align__(16) uint8_t sm[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int j = blockIdx.x % p.n_parts, g = (blockIdx.x / p.n_parts) % p.nkv;
    const int b = blockIdx.x / (p.n_parts * p.nkv);
    const int G = p.group, kpad = attn_kpad(p.part_keys);
    float* qs = reinterpret_cast<float*>(sm);
    uint16_t* rows = reinterpret_cast<uint16_t*>(sm + align16((uint32_t)(G * HD * 4)));
    float* sc = reinterpret_cast<float*>(rows + 2 * (size_t)kpad * HD);
    const int pos = p.positions[b];
    const int first = j * p.part_keys;
    const int count = min(p.part_keys, p.max_ctx - first);
    const int n = min(count, pos + 1 - first);
    const float* qsrc = p.q + (size_t)b * p.Q + (size_t)g * G * HD;
    for (int e = threadIdx.x * 4; e < G * HD; e += kBaseThreads * 4)
        *reinterpret_cast<uint4*>(qs + e) = ld_cg_v4(qsrc + e);
    const size_t base = kv_off(p, l, b, g, first);
    for (int i = threadIdx.x; i < n * (HD / 8); i += kBaseThreads) {
        reinterpret_cast<uint4*>(rows)[i] = ld_cg_v4(p.kc + base + (size_t)i * 8);
        reinterpret_cast<uint4*>(rows + (size_t)kpad * HD)[i] = ld_cg_v4(p.vc + base + (size_t)i * 8);
    }
    __syncthreads();
    // one fill of kpad rows; no row is special (knew / vnew only stand in for
    // rows past the item)
    const AttnRows<HD> R{reinterpret_cast<const uint8_t*>(rows), 0u, 1, 0, kpad, n, -1, rows,
                         rows + (size_t)kpad * HD};
    auto bar = []() {
        __syncthreads();
        return true;
    };
    if (p.n_parts == 1) {
        float* out = p.attn + (size_t)b * p.Q + (size_t)g * G * HD;
        attn_item_block<HD>(R, qs, G, sc, warp, lane, bar, [](int) {},
                            [&](int h, int d, float o, float, float l) { out[h * HD + d] = __fdiv_rn(o, l); });
    } else {
        attn_item_block<HD>(R, qs, G, sc, warp, lane, bar, [](int) {}, [&](int h, int d, float o, float m, float l) {
            const size_t hp = ((size_t)b * p.nq + (size_t)(g * G + h)) * p.n_parts + j;
            p.part_o[hp * HD + d] = o;
            if (d == 0) {
                p.part_ml[hp * 2] = m;
                p.part_ml[hp * 2 + 1] = l;
            }
        });
    }
}

template <int HD>
__global__ void __launch_bounds__(kBaseThreads) k_attn_merge(const __grid_constant__ Params p) {
    if (step_failed(p)) return;
    const int lane = threadIdx.x & 31;
    const int gw = blockIdx.x * kBaseWarps + (threadIdx.x >> 5);
    if (gw >= p.B * p.nq) return;
    const int b = gw / p.nq, head = gw % p.nq;
    float* out = p.attn + (size_t)b * p.Q;
    attn_merge_heads<HD, 1>(p, b, head, 1, p.nq, lane, [&](int e, float x) { out[e] = x; });
}

// ------------------------------------------------------------------ host-side launch

// CTAs of a matvec kernel over `units` tiles.
static uint32_t matvec_blocks(uint32_t units, int n_sm) {
    const uint32_t warps_cap = (uint32_t)n_sm * 16;
    const uint32_t w = units < warps_cap ? units : warps_cap;
    return (w + kBaseWarps - 1) / kBaseWarps;
}

// A layer's ops behind its attention output.
template <int KH, int KO, int KF, int HD>
static void launch_after_attention(const Params& p, int l, cudaStream_t st, int n_sm) {
    const size_t in_h = (size_t)p.B * KH * 256 * 4 + 4 * kConsumerWarps;
    const size_t in_o = (size_t)p.B * KO * 256 * 4 + 4 * kConsumerWarps;
    const uint32_t no = (uint32_t)p.H / 4;
    k_tiles<MK_OP_OPROJ, KO, HD><<<matvec_blocks(no, n_sm), kBaseThreads, in_o, st>>>(p, l, no, p.tile_o);
    const uint32_t ng = (uint32_t)p.F / 2;
    k_tiles<MK_OP_GATEUP, KH, HD><<<matvec_blocks(ng, n_sm), kBaseThreads, in_h, st>>>(p, l, ng, p.tile_h);
    k_down<KF><<<matvec_blocks((uint32_t)p.H / 4, n_sm), kBaseThreads, 0, st>>>(p, l);
}

template <int KH, int HD>
static void launch_lm_head(const Params& p, cudaStream_t st, int n_sm) {
    const size_t in_h = (size_t)p.B * KH * 256 * 4 + 4 * kConsumerWarps;
    const uint32_t nl = (uint32_t)p.V / 4;
    k_tiles<MK_OP_LMHEAD, KH, HD><<<matvec_blocks(nl, n_sm), kBaseThreads, in_h, st>>>(p, 0, nl, p.tile_h);
}

template <int KH, int KO, int KF, int HD>
static cudaError_t launch_all(const Params& p, cudaStream_t st, int n_sm) {
    const size_t attn_smem = attn_item_smem<HD>(p.group, attn_kpad(p.part_keys));
    const size_t in_h = (size_t)p.B * KH * 256 * 4 + 4 * kConsumerWarps;
    k_validate<<<1, 32, 0, st>>>(p);
    const uint32_t tpg = (uint32_t)(p.group + 2) * (HD / 4);
    for (int l = 0; l < p.L; ++l) {
        const uint32_t nq = (uint32_t)p.nkv * tpg;
        k_tiles<MK_OP_QKV, KH, HD><<<matvec_blocks(nq, n_sm), kBaseThreads, in_h, st>>>(p, l, nq, p.tile_h);
        const uint32_t na = (uint32_t)(p.B * p.nkv * p.n_parts);
        k_attn_item<HD><<<na, kBaseThreads, attn_smem, st>>>(p, l);
        if (p.n_parts > 1) {
            const uint32_t nm = (uint32_t)(p.B * p.nq);
            k_attn_merge<HD><<<(nm + kBaseWarps - 1) / kBaseWarps, kBaseThreads, 0, st>>>(p);
        }
        launch_after_attention<KH, KO, KF, HD>(p, l, st, n_sm);
    }
    launch_lm_head<KH, HD>(p, st, n_sm);
    return cudaGetLastError();
}

// The step on the 8-bit cache: the QKV kernel leaves the new key and value in a
// one-slot buffer, the cache stores them (the block they fill is quantised), and its
// attention reads the cache, the new token included.
template <int KH, int KO, int KF, int HD>
static mk_status launch_all_qcache(const QcacheStep& s, cudaStream_t st, int n_sm) {
    Params p = s.params;
    p.max_batch = p.B;
    p.max_seq = 1;
    const size_t in_h = (size_t)p.B * KH * 256 * 4 + 4 * kConsumerWarps;
    const int64_t kv_row = (int64_t)p.nkv * p.d;
    const int64_t strides[4] = {p.B * kv_row, kv_row, p.d, p.d};
    k_validate_qcache<<<1, 32, 0, st>>>(s.params, s.cache->max_seq, s.positions, s.status_out);
    const uint32_t nq = (uint32_t)p.nkv * (uint32_t)(p.group + 2) * (HD / 4);
    for (int l = 0; l < p.L; ++l) {
        k_tiles<MK_OP_QKV, KH, HD, true><<<matvec_blocks(nq, n_sm), kBaseThreads, in_h, st>>>(p, l, nq, p.tile_h);
        const size_t at = (size_t)l * p.B * p.nkv * p.d;
        mk_status r = mk_qcache_append(s.cache, l, 1, p.B, 1, p.kc + at, p.vc + at, strides, s.positions, nullptr, st);
        if (r == MK_OK)
            r = mk_qcache_attention(s.cache, l, p.B, p.nq, p.max_ctx, p.q, s.positions, p.attn, s.attn_workspace,
                                    s.attn_workspace_bytes, st);
        if (r != MK_OK) return r;
        launch_after_attention<KH, KO, KF, HD>(p, l, st, n_sm);
    }
    launch_lm_head<KH, HD>(p, st, n_sm);
    return cudaGetLastError() == cudaSuccess ? MK_OK : MK_ERR_CUDA;
}

// Shared memory of the matvec kernels, for the largest batch: the limit belongs to the
// kernel, not to a handle, so a smaller handle must not lower it under a larger one.
template <int KH, int KO, int HD>
static cudaError_t prepare_tiles() {
    const int in_h = (int)((size_t)kMaxBatch * KH * 256 * 4 + 4 * kConsumerWarps);
    const int in_o = (int)((size_t)kMaxBatch * KO * 256 * 4 + 4 * kConsumerWarps);
    cudaError_t e = cudaFuncSetAttribute(k_tiles<MK_OP_QKV, KH, HD>, cudaFuncAttributeMaxDynamicSharedMemorySize, in_h);
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(k_tiles<MK_OP_GATEUP, KH, HD>, cudaFuncAttributeMaxDynamicSharedMemorySize, in_h);
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(k_tiles<MK_OP_LMHEAD, KH, HD>, cudaFuncAttributeMaxDynamicSharedMemorySize, in_h);
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(k_tiles<MK_OP_OPROJ, KO, HD>, cudaFuncAttributeMaxDynamicSharedMemorySize, in_o);
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(k_tiles<MK_OP_QKV, KH, HD, true>, cudaFuncAttributeMaxDynamicSharedMemorySize, in_h);
    return e;
}

static cudaError_t prepare_matvecs(const Params& p) {
    const int KH = p.H / 256, KO = p.Q / 256;
    if (KH == 2 && KO == 2 && p.d == 64) return prepare_tiles<2, 2, 64>();
    if (KH == 8 && KO == 8 && p.d == 64) return prepare_tiles<8, 8, 64>();
    if (KH == 12 && KO == 12 && p.d == 128) return prepare_tiles<12, 12, 128>();
    return cudaErrorInvalidValue;
}

// Once per schedule, outside any stream capture.
cudaError_t baseline_prepare(const Params& p) {
    const cudaError_t e = prepare_matvecs(p);
    if (e != cudaSuccess) return e;
    const int kpad = attn_kpad(p.part_keys);
    if (p.d == 64)
        return cudaFuncSetAttribute(k_attn_item<64>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    (int)attn_item_smem<64>(p.group, kpad));
    if (p.d == 128)
        return cudaFuncSetAttribute(k_attn_item<128>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    (int)attn_item_smem<128>(p.group, kpad));
    return cudaErrorInvalidValue;
}

cudaError_t baseline_launch(const Params& p, cudaStream_t stream, int n_sm) {
    const int KH = p.H / 256, KO = p.Q / 256, KF = p.F / 1024;
    if (KH == 2 && KO == 2 && KF == 2 && p.d == 64) return launch_all<2, 2, 2, 64>(p, stream, n_sm);
    if (KH == 8 && KO == 8 && KF == 8 && p.d == 64) return launch_all<8, 8, 8, 64>(p, stream, n_sm);
    if (KH == 12 && KO == 12 && KF == 8 && p.d == 128) return launch_all<12, 12, 8, 128>(p, stream, n_sm);
    return cudaErrorInvalidValue;
}

mk_status qcache_step_launch(const QcacheStep& s, cudaStream_t stream, int n_sm) {
    const Params& p = s.params;
    // no schedule has set the limits; asking again at every step costs nothing that its host time shows (38 us with
    // and without)
    if (prepare_matvecs(p) != cudaSuccess) return MK_ERR_CUDA;
    const int KH = p.H / 256, KO = p.Q / 256, KF = p.F / 1024;
    if (KH == 2 && KO == 2 && KF == 2 && p.d == 64) return launch_all_qcache<2, 2, 2, 64>(s, stream, n_sm);
    if (KH == 8 && KO == 8 && KF == 8 && p.d == 64) return launch_all_qcache<8, 8, 8, 64>(s, stream, n_sm);
    if (KH == 12 && KO == 12 && KF == 8 && p.d == 128) return launch_all_qcache<12, 12, 8, 128>(s, stream, n_sm);
    return MK_ERR_UNSUPPORTED;
}

}  // namespace mk
