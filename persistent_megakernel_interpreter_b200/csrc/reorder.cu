// Reordering of slot caches: row r of the batch goes on from what row parents[r]
// holds (beam search's survivors, a prompt forked into several rows, live rows
// moved down over finished ones).
//
//   cache[layer][r][head][slot] := cache[layer][parents[r]][head][slot]
//       for starts[r] <= slot < lengths[parents[r]], all rows at once.
//
// The rows are a permutation with repeats, done in place. A 16-byte column (one
// piece of one slot of one head and layer) is independent of every other column,
// so one thread takes the column of all rows: it loads what each moving row needs
// from its parent and only then stores, which needs no second buffer, no order
// among rows and no barrier. Bound by HBM: each distinct source slot is read once
// (a second row with the same parent finds it in L1) and each changed slot written
// once.
#include <cuda_runtime.h>

#include "qcache.h"

namespace mk {
namespace {

constexpr int kThreadsRe = 256;
constexpr int kRows = kMaxBatch;

// One tensor [planes outer][rows][planes inner][slots][slot_bytes]; the slots that
// move are the closed blocks' (codes, scales), the open block's (tails) or all.
enum Span { kSpanAll, kSpanClosed, kSpanClosedBlocks, kSpanOpen };
struct MoveTensor {
    uint8_t* base;
    uint32_t slot_bytes;
    uint32_t slots;
    int span;
};
struct MoveArgs {
    MoveTensor t[6];
    int n_tensors;
    int n_layers, max_batch, n_heads, max_seq, rows;
    const int32_t* parents;
    const int32_t* starts;   // NULL: 0
    const int32_t* lengths;
};

// The slots of tensor `span` that row r takes from its parent: [lo, hi).
__device__ __forceinline__ void move_range(int span, int start, int length, uint32_t& lo, uint32_t& hi) {
    const int closed = length / kQBlock;
    if (span == kSpanAll) {
        lo = start;
        hi = length;
    } else if (span == kSpanClosed) {          // whole blocks, from the start's own block
        lo = start / kQBlock * kQBlock;
        hi = closed * kQBlock;
    } else if (span == kSpanClosedBlocks) {
        lo = start / kQBlock;
        hi = closed;
    } else {
        lo = max(start - closed * kQBlock, 0);
        hi = length - closed * kQBlock;
    }
    if (hi < lo) hi = lo;
}

template <class W>
__device__ __forceinline__ void move_columns(const MoveTensor& T, const MoveArgs& a, const int (&parent)[kRows],
                                             const uint32_t (&lo)[kRows], const uint32_t (&hi)[kRows], uint32_t first,
                                             uint32_t last) {
    // byte ranges of a plane fit 64 bits only: 2^20 slots of 256 bytes are 2^28
    const uint32_t per = kThreadsRe * (uint32_t)sizeof(W);
    const uint32_t chunks = (last - first + per - 1) / per;
    const size_t plane = (size_t)T.slots * T.slot_bytes;
    const size_t row = plane * a.n_heads;
    const uint32_t items = chunks * (uint32_t)(a.n_layers * a.n_heads);
    for (uint32_t it = blockIdx.x; it < items; it += gridDim.x) {
        const uint32_t pl = it / chunks, off = first + (it % chunks) * per + threadIdx.x * (uint32_t)sizeof(W);
        const uint32_t l = pl / a.n_heads, h = pl % a.n_heads;
        uint8_t* base = T.base + (size_t)l * a.max_batch * row + (size_t)h * plane + off;
        W v[kRows];
#pragma unroll
        for (int r = 0; r < kRows; ++r)
            if (off >= lo[r] && off < hi[r]) v[r] = *reinterpret_cast<const W*>(base + parent[r] * row);
#pragma unroll
        for (int r = 0; r < kRows; ++r)
            if (off >= lo[r] && off < hi[r]) *reinterpret_cast<W*>(base + r * row) = v[r];
    }
}

__global__ void __launch_bounds__(kThreadsRe) k_reorder(const __grid_constant__ MoveArgs a) {
    int parent[kRows], start[kRows], length[kRows];
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
        parent[r] = r;
        start[r] = length[r] = 0;
        if (r < a.rows) {
            const int p = a.parents[r];
            if (p >= 0 && p < a.rows && p != r) {
                parent[r] = p;
                length[r] = min(max(a.lengths[p], 0), a.max_seq);
                start[r] = a.starts ? min(max(a.starts[r], 0), a.max_seq) : 0;
            }
        }
    }
    for (int i = 0; i < a.n_tensors; ++i) {
        const MoveTensor T = a.t[i];
        uint32_t lo[kRows], hi[kRows], first = 0xffffffffu, last = 0;
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
            move_range(T.span, start[r], length[r], lo[r], hi[r]);
            if (parent[r] == r) hi[r] = lo[r];
            lo[r] *= T.slot_bytes;
            hi[r] *= T.slot_bytes;
            if (lo[r] < hi[r]) {
                first = min(first, lo[r]);
                last = max(last, hi[r]);
            }
        }
        if (first >= last) continue;
        if (T.slot_bytes % 16 == 0) move_columns<uint4>(T, a, parent, lo, hi, first, last);
        else move_columns<uint32_t>(T, a, parent, lo, hi, first, last);
    }
}

mk_status launch_reorder(const MoveArgs& a, void* stream) {
    k_reorder<<<kQSms * 8, kThreadsRe, 0, static_cast<cudaStream_t>(stream)>>>(a);
    return cudaGetLastError() == cudaSuccess ? MK_OK : MK_ERR_CUDA;
}

}  // namespace
}  // namespace mk

extern "C" mk_status mk_cache_reorder(const mk_config* cfg, void* k_cache, void* v_cache, int rows,
                                      const int32_t* parents, const int32_t* lengths, const int32_t* starts,
                                      void* stream) {
    if (!cfg || !k_cache || !v_cache || !parents || !lengths) return MK_ERR_INVALID_ARG;
    if (cfg->n_layers < 1 || cfg->n_layers > mk::kMaxLayers || cfg->n_kv_heads < 1 || cfg->n_kv_heads > mk::kQMaxHeads ||
        (cfg->head_dim != 64 && cfg->head_dim != 128) || cfg->max_seq < 1 || cfg->max_seq > (1 << 20) ||
        cfg->max_batch < 1 || cfg->max_batch > mk::kMaxBatch)
        return MK_ERR_UNSUPPORTED;
    if (rows < 1 || rows > cfg->max_batch) return MK_ERR_INVALID_ARG;
    if ((reinterpret_cast<uintptr_t>(k_cache) | reinterpret_cast<uintptr_t>(v_cache)) & 15) return MK_ERR_INVALID_ARG;
    mk::MoveArgs a{};
    const uint32_t sb = 2u * (uint32_t)cfg->head_dim;
    a.t[0] = {static_cast<uint8_t*>(k_cache), sb, (uint32_t)cfg->max_seq, mk::kSpanAll};
    a.t[1] = {static_cast<uint8_t*>(v_cache), sb, (uint32_t)cfg->max_seq, mk::kSpanAll};
    a.n_tensors = 2;
    a.n_layers = cfg->n_layers;
    a.max_batch = cfg->max_batch;
    a.n_heads = cfg->n_kv_heads;
    a.max_seq = cfg->max_seq;
    a.rows = rows;
    a.parents = parents;
    a.starts = starts;
    a.lengths = lengths;
    return mk::launch_reorder(a, stream);
}

extern "C" mk_status mk_qcache_reorder(const mk_qcache* c, int rows, const int32_t* parents, const int32_t* lengths,
                                       const int32_t* starts, void* stream) {
    if (!parents || !lengths) return MK_ERR_INVALID_ARG;
    if (const mk_status st = mk::qcache_check(c); st != MK_OK) return st;
    if (rows < 1 || rows > c->max_batch) return MK_ERR_INVALID_ARG;
    mk::MoveArgs a{};
    const uint32_t d = (uint32_t)c->head_dim, S = (uint32_t)c->max_seq, nb = (uint32_t)mk::qcache_blocks(c->max_seq);
    a.t[0] = {static_cast<uint8_t*>(c->k_codes), d, S, mk::kSpanClosed};
    a.t[1] = {static_cast<uint8_t*>(c->v_codes), d, S, mk::kSpanClosed};
    a.t[2] = {reinterpret_cast<uint8_t*>(c->k_scale), 4u, nb, mk::kSpanClosedBlocks};
    a.t[3] = {reinterpret_cast<uint8_t*>(c->v_scale), 4u, nb, mk::kSpanClosedBlocks};
    a.t[4] = {static_cast<uint8_t*>(c->k_tail), 2u * d, (uint32_t)mk::kQBlock, mk::kSpanOpen};
    a.t[5] = {static_cast<uint8_t*>(c->v_tail), 2u * d, (uint32_t)mk::kQBlock, mk::kSpanOpen};
    a.n_tensors = 6;
    a.n_layers = c->n_layers;
    a.max_batch = c->max_batch;
    a.n_heads = c->n_kv_heads;
    a.max_seq = c->max_seq;
    a.rows = rows;
    a.parents = parents;
    a.starts = starts;
    a.lengths = lengths;
    return mk::launch_reorder(a, stream);
}
