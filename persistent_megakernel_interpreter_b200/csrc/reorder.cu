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

// One tensor [layer][row][head][slot] of slot_bytes each; the slots that move are all
// of a row's, or the closed blocks' (codes), one entry a closed block (scales), or the
// open block's (tails).
enum Span { kSpanAll, kSpanClosed, kSpanClosedBlocks, kSpanOpen };
struct MoveTensor {
    uint8_t* base;
    uint32_t slot_bytes;
    uint32_t slots;
    int span;
};
constexpr int kTensors = 6;
struct MoveArgs {
    MoveTensor t[kTensors];
    int n_tensors;
    int n_layers, max_batch, n_heads, max_seq, rows;
    const int32_t* parents;
    const int32_t* starts;   // NULL: 0
    const int32_t* lengths;
};

// The slots of a tensor that a row takes from its parent: [lo, hi).
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

// A row that moves: bytes [lo, hi) of each (layer, head) plane at byte dst of a layer come from the
// plane at byte src.
struct alignas(8) Move {
    size_t src, dst;
    uint32_t lo, hi;
};
struct MovePlan {
    Move move[kTensors][kMaxBatch];
    uint32_t first[kTensors], chunks[kTensors];   // a plane's bytes that move for any row, in chunks
    uint32_t before[kTensors + 1];                // items of the tensors before
    int n;                                        // rows that move
};

// One item: a chunk of kThreadsRe * U words W of one (layer, head) plane, for the plan's rows (at most N).
template <class W, int N, int U>
__device__ __forceinline__ void move_chunk(const MoveTensor& T, const MoveArgs& a, const Move* moves, int n, uint32_t plane_no,
                                           uint32_t off) {
    const size_t plane = (size_t)T.slots * T.slot_bytes;
    const uint32_t l = plane_no / (uint32_t)a.n_heads, h = plane_no % (uint32_t)a.n_heads;
    uint8_t* base = T.base + ((size_t)l * a.max_batch * a.n_heads + h) * plane + off;
    constexpr uint32_t kNext = kThreadsRe * (uint32_t)sizeof(W);
    W v[N][U];
#pragma unroll
    for (int j = 0; j < N; ++j)
        if (j < n) {
            const uint8_t* src = base + moves[j].src;
            const uint32_t lo = moves[j].lo, hi = moves[j].hi;
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (off + u * kNext >= lo && off + u * kNext < hi) v[j][u] = *reinterpret_cast<const W*>(src + u * kNext);
        }
#pragma unroll
    for (int j = 0; j < N; ++j)
        if (j < n) {
            uint8_t* dst = base + moves[j].dst;
            const uint32_t lo = moves[j].lo, hi = moves[j].hi;
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (off + u * kNext >= lo && off + u * kNext < hi) *reinterpret_cast<W*>(dst + u * kNext) = v[j][u];
        }
}

// Words a thread moves of each row in one item, by the rows that move: 8 loads on the way either way.
__device__ __forceinline__ int words_each(int n) { return n <= 2 ? 4 : n <= 4 ? 2 : 1; }

// Four CTAs an SM (64 registers a thread) and several times as many CTAs as fit, which evens out the SMs: 98% of
// the measured copy rate on the 1B shape's cache (166.7 us), 96% in 8 bits (381.8 us); with 8 CTAs an SM in all
// 184 and 414 us.
__global__ void __launch_bounds__(kThreadsRe, 4) k_reorder(const __grid_constant__ MoveArgs a) {
    __shared__ MovePlan plan;
    cudaGridDependencySynchronize();     // everything enqueued before has run
    if (threadIdx.x < 32) {
        // lane r plans row r
        const int r = threadIdx.x;
        const bool row = r < a.rows;
        int parent = row ? a.parents[r] : -1;
        const int own = row ? min(max(a.lengths[r], 0), a.max_seq) : 0;
        const int start = row && a.starts ? min(max(a.starts[r], 0), a.max_seq) : 0;
        const bool moves = row && parent >= 0 && parent < a.rows && parent != r;
        const int length = __shfl_sync(0xffffffffu, own, moves ? parent : r);
        const uint32_t mask = __ballot_sync(0xffffffffu, moves);
        const int n = __popc(mask), j = __popc(mask & ((1u << r) - 1u));
        uint32_t before = 0;
        for (int i = 0; i < a.n_tensors; ++i) {
            const MoveTensor& T = a.t[i];
            uint32_t lo, hi;
            move_range(T.span, start, length, lo, hi);
            if (!moves) lo = hi;
            lo *= T.slot_bytes;
            hi *= T.slot_bytes;
            const size_t row_bytes = (size_t)T.slots * T.slot_bytes * a.n_heads;
            if (moves) plan.move[i][j] = Move{parent * row_bytes, r * row_bytes, lo, hi};
            const uint32_t first = __reduce_min_sync(0xffffffffu, lo < hi ? lo : 0xffffffffu);
            const uint32_t last = __reduce_max_sync(0xffffffffu, lo < hi ? hi : 0u);
            const uint32_t per = kThreadsRe * (T.slot_bytes % 16 ? 4u : 16u * (uint32_t)words_each(n));
            const uint32_t chunks = last > first ? (last - first + per - 1) / per : 0u;
            if (r == 0) {
                plan.first[i] = first;
                plan.chunks[i] = chunks;
                plan.before[i] = before;
            }
            before += chunks * (uint32_t)(a.n_layers * a.n_heads);
        }
        if (r == 0) {
            plan.before[a.n_tensors] = before;
            plan.n = n;
        }
    }
    __syncthreads();
    const int n = plan.n;
    const uint32_t total = plan.before[a.n_tensors], words = (uint32_t)words_each(n);
    for (uint32_t it = blockIdx.x; it < total; it += gridDim.x) {
        int i = 0;
        while (it >= plan.before[i + 1]) ++i;
        const MoveTensor& T = a.t[i];
        const uint32_t local = it - plan.before[i], chunks = plan.chunks[i], pl = local / chunks;
        const Move* m = plan.move[i];
        if (T.slot_bytes % 16 == 0) {
            const uint32_t off = plan.first[i] + ((local % chunks) * words * kThreadsRe + threadIdx.x) * 16u;
            if (n <= 2) move_chunk<uint4, 2, 4>(T, a, m, n, pl, off);
            else if (n <= 4) move_chunk<uint4, 4, 2>(T, a, m, n, pl, off);
            else move_chunk<uint4, 8, 1>(T, a, m, n, pl, off);
        } else {
            const uint32_t off = plan.first[i] + ((local % chunks) * kThreadsRe + threadIdx.x) * 4u;
            move_chunk<uint32_t, 8, 1>(T, a, m, n, pl, off);
        }
    }
}

mk_status launch_reorder(const MoveArgs& a, void* stream) {
    // as many CTAs as there can be items, at most 32 an SM
    size_t most = 0;
    for (int i = 0; i < a.n_tensors; ++i) {
        const size_t per = kThreadsRe * (a.t[i].slot_bytes % 16 ? 4u : 16u);
        most += ((size_t)a.t[i].slots * a.t[i].slot_bytes + per - 1) / per * (size_t)(a.n_layers * a.n_heads);
    }
    const size_t cap = (size_t)kQSms * 32;
    const cudaError_t e = launch_behind(k_reorder, (int)(most < cap ? most : cap), kThreadsRe, 0, static_cast<cudaStream_t>(stream), a);
    return e == cudaSuccess ? MK_OK : MK_ERR_CUDA;
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
    const uintptr_t k = reinterpret_cast<uintptr_t>(k_cache), v = reinterpret_cast<uintptr_t>(v_cache);
    if ((k | v) & 15) return MK_ERR_INVALID_ARG;
    // both are moved at once: a column may belong to one of them only
    const size_t bytes = (size_t)cfg->n_layers * cfg->max_batch * cfg->n_kv_heads * cfg->max_seq * cfg->head_dim * 2;
    if ((k < v ? v - k : k - v) < bytes) return MK_ERR_INVALID_ARG;
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
