// Beam search's choice between two decode steps: from the rows of logits of each
// sequence's beams, the n_out best continuations by running score plus log
// probability.
//
//   total(k, v) = score[k] + ((x[k][v] - m[k]) - log sum_u exp(x[k][u] - m[k])),  m[k] = max_u x[k][u]
//
// Within a row the order is the logits' own, so a row's best n_out are found on its
// raw logits while the sum is formed, in one pass over HBM (bound: 4 bytes a logit);
// only those few meet the other beams, as totals in 64 bits.
//
// One cluster per sequence. A row is cut into `splits` pieces at multiples of four
// tokens, by token number and never by address, so equal rows give equal sums
// wherever they lie. The cluster's CTAs take the pieces in turn:
//   1. each thread keeps the maximum and the running sum of its logits; the n-th
//      largest of 32 group maxima is a bound that at least n logits reach;
//   2. the logits that reach it (few: the expected number is about n) are gathered by
//      the threads whose maximum does, and ranked by counting.
// Each piece's maximum, sum and candidates go to CTA 0's shared memory (distributed
// shared memory), which ranks them all by total and writes the answer.
#include <cooperative_groups.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "qcache.h"

namespace mk {
namespace {

namespace cg = cooperative_groups;

constexpr int kBeamThreads = 512;
constexpr int kBeamWarps = kBeamThreads / 32;
constexpr int kMaxBeams = 16;
constexpr int kMaxOut = 32;
constexpr int kMaxCluster = 8;
constexpr int kMaxPieces = 16;            // pieces of a sequence's rows: beams * splits
constexpr int kList = 1024;               // gathered logits of a piece
constexpr float kLog2E = 1.4426950408889634f;
constexpr float kBig = 3.402823466e38f;

struct BeamArgs {
    const float* logits;
    long long ld;
    int batch, beams, vocab, n_out, splits, piece, eos;
    const float* scores;
    const int32_t* finished;
    int32_t* next_tokens;
    int32_t* parents;
    float* next_scores;
    int32_t* next_finished;
    int32_t* positions;
};

struct Cand {
    float x;
    int token;
};

struct BeamSmem {
    // CTA 0's: what every piece found
    Cand cand[kMaxPieces][kMaxOut];
    float m[kMaxPieces], s[kMaxPieces];
    int count[kMaxPieces];
    // each CTA's own
    Cand list[kList];
    float gmax[32], wm[kBeamWarps], ws[kBeamWarps];
    int wcount[kBeamWarps];
    int n_list, n_tail;
    float again;
    // the last step's
    double m_row[kMaxBeams], log_row[kMaxBeams];
    unsigned long long total[kMaxPieces * kMaxOut], tie[kMaxPieces * kMaxOut];
    int2 from[kMaxOut];                   // parent row, finished
};

// Whole numbers in the order of the numbers; -0 becomes 0 first, for the two are equal.
__device__ __forceinline__ uint32_t ordered(float x) {
    const uint32_t u = __float_as_uint(x + 0.0f);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ unsigned long long ordered(double x) {
    const unsigned long long u = (unsigned long long)__double_as_longlong(x + 0.0);
    return u >> 63 ? ~u : u | 0x8000000000000000ull;
}

// x with NaN as -infinity: never chosen, adds nothing to the sum.
__device__ __forceinline__ float clean(float x) { return fmaxf(x, -INFINITY); }

// Four consecutive logits of a row from token i (a multiple of 4); past the end -infinity.
template <bool ALIGNED>
__device__ __forceinline__ float4 load4(const float* row, int i, int end) {
    if (ALIGNED && i + 4 <= end) {
        const float4 v = __ldg(reinterpret_cast<const float4*>(row + i));
        return make_float4(clean(v.x), clean(v.y), clean(v.z), clean(v.w));
    }
    float4 v = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
    if (i < end) v.x = clean(__ldg(row + i));
    if (i + 1 < end) v.y = clean(__ldg(row + i + 1));
    if (i + 2 < end) v.z = clean(__ldg(row + i + 2));
    if (i + 3 < end) v.w = clean(__ldg(row + i + 3));
    return v;
}

__device__ __forceinline__ float e2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// The finite number a maximum is subtracted as: an all-masked row has none, and a row
// of the type's lowest value keeps it.
__device__ __forceinline__ float finite(float m) { return fminf(fmaxf(m, -kBig), kBig); }

__device__ __forceinline__ void join_sum(float& m, float& s, float m2, float s2) {
    const float M = fmaxf(m, m2), ref = finite(M);
    s = s * e2((m - ref) * kLog2E) + s2 * e2((m2 - ref) * kLog2E);
    m = M;
}

// The n-th largest of 32 values (one per lane), equal ones counted by lane.
__device__ __forceinline__ float nth_of_warp(float v, int n, int lane) {
    int rank = 0;
#pragma unroll
    for (int i = 0; i < 32; ++i) {
        const float o = __shfl_sync(0xffffffffu, v, i);
        rank += o > v || (o == v && i < lane);
    }
    return __shfl_sync(0xffffffffu, v, __ffs(__ballot_sync(0xffffffffu, rank == n - 1)) - 1);
}

// Piece [begin, end) of one row: its maximum and sum, and its n best logits (fewer if it is
// shorter), best first, equal logits by token. Into (out, *om, *os, *on) by all threads.
template <bool ALIGNED>
__device__ __forceinline__ void scan_piece(BeamSmem& sm, const float* row, int begin, int end, int n, Cand* out, float* om,
                                           float* os, int* on) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    n = min(n, end - begin);
    float m = -INFINITY, s = 0.f;
    constexpr int U = 4;
    for (int i = begin + 4 * tid; i < end; i += 4 * U * kBeamThreads) {
        float4 v[U];
        float bm = -INFINITY;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            v[u] = load4<ALIGNED>(row, i + 4 * u * kBeamThreads, end);
            bm = fmaxf(bm, fmaxf(fmaxf(v[u].x, v[u].y), fmaxf(v[u].z, v[u].w)));
        }
        if (bm > m) {
            s *= e2((m - finite(bm)) * kLog2E);
            m = bm;
        }
        const float ref = finite(m);
#pragma unroll
        for (int u = 0; u < U; ++u)
            s += (e2((v[u].x - ref) * kLog2E) + e2((v[u].y - ref) * kLog2E)) +
                 (e2((v[u].z - ref) * kLog2E) + e2((v[u].w - ref) * kLog2E));
    }
    // group maxima (16 threads), then the CTA's maximum and sum
    float gm = m;
#pragma unroll
    for (int k = 8; k > 0; k >>= 1) gm = fmaxf(gm, __shfl_xor_sync(0xffffffffu, gm, k));
    float cm = m, cs = s;
#pragma unroll
    for (int k = 16; k > 0; k >>= 1) {
        const float m2 = __shfl_xor_sync(0xffffffffu, cm, k), s2 = __shfl_xor_sync(0xffffffffu, cs, k);
        join_sum(cm, cs, m2, s2);
    }
    if ((lane & 15) == 0) sm.gmax[tid >> 4] = gm;
    if (lane == 0) {
        sm.wm[warp] = cm;
        sm.ws[warp] = cs;
    }
    if (tid == 0) sm.n_list = 0;
    __syncthreads();
    const float top = sm.gmax[lane];
    float bound = n > 0 ? nth_of_warp(top, n, lane) : INFINITY;
    // infinite logits share the row: the sum is their number
    const bool endless = __any_sync(0xffffffffu, top == INFINITY);
    if (endless) {
        if (tid == 0) sm.n_tail = 0;
        __syncthreads();
        if (m == INFINITY) {
            int k = 0;
            for (int i = begin + 4 * tid; i < end; i += 4 * kBeamThreads) {
                const float4 v = load4<ALIGNED>(row, i, end);
                k += (v.x == INFINITY) + (v.y == INFINITY) + (v.z == INFINITY) + (v.w == INFINITY);
            }
            atomicAdd(&sm.n_tail, k);
        }
        __syncthreads();
    }
    if (warp == 0) {
        cm = lane < kBeamWarps ? sm.wm[lane] : -INFINITY;
        cs = lane < kBeamWarps ? sm.ws[lane] : 0.f;
#pragma unroll
        for (int k = 8; k > 0; k >>= 1) {
            const float m2 = __shfl_xor_sync(0xffffffffu, cm, k), s2 = __shfl_xor_sync(0xffffffffu, cs, k);
            join_sum(cm, cs, m2, s2);
        }
        if (lane == 0) {
            *om = cm;
            *os = endless ? (float)sm.n_tail : cs;
            *on = n;
        }
    }
    if (n == 0) return;
    // gather what reaches the bound; where too much does (ties, or the best all in a few groups), only
    // what is above it; where that is still too much, raise the bound to the n-th of what was gathered
    bool above = false;
    for (;;) {
        if (m >= bound) {
            for (int i = begin + 4 * tid; i < end; i += 4 * kBeamThreads) {
                const float4 v = load4<ALIGNED>(row, i, end);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const float x = (&v.x)[k];
                    if (i + k < end && (above ? x > bound : x >= bound)) {
                        const int at = atomicAdd(&sm.n_list, 1);
                        if (at < kList) sm.list[at] = Cand{x, i + k};
                    }
                }
            }
        }
        __syncthreads();
        const int found = sm.n_list;
        if (found <= kList) break;
        if (above) {
            // the n-th largest value of the list
            for (int e = tid; e < kList; e += kBeamThreads) {
                const float x = sm.list[e].x;
                int more = 0, same = 0;
                for (int f = 0; f < kList; ++f) {
                    more += sm.list[f].x > x;
                    same += sm.list[f].x == x;
                }
                if (more < n && more + same >= n) sm.again = x;
            }
            __syncthreads();
            bound = sm.again;
        }
        above = !above;
        __syncthreads();
        if (tid == 0) sm.n_list = 0;
        __syncthreads();
    }
    int found = sm.n_list;
    if (found < n) {
        // too few above the bound: the lowest tokens that equal it fill up
        __syncthreads();
        if (tid == 0) sm.n_tail = found;
        __syncthreads();
        for (int base = begin; base < end; base += kBeamThreads) {
            const int have = sm.n_tail;
            if (have >= n) break;
            const int i = base + tid;
            const bool eq = i < end && clean(__ldg(row + i)) == bound;
            const uint32_t mask = __ballot_sync(0xffffffffu, eq);
            if (lane == 0) sm.wcount[warp] = __popc(mask);
            __syncthreads();
            int at = have, all = have;
            for (int w = 0; w < kBeamWarps; ++w) {
                if (w < warp) at += sm.wcount[w];
                all += sm.wcount[w];
            }
            at += __popc(mask & ((1u << lane) - 1u));
            if (eq && at < n) sm.list[at] = Cand{bound, i};
            __syncthreads();
            if (tid == 0) sm.n_tail = all;
            __syncthreads();
        }
        found = n;
    }
    // ranked by counting
    for (int e = tid; e < found; e += kBeamThreads) {
        const Cand c = sm.list[e];
        int rank = 0;
        for (int f = 0; f < found; ++f) {
            const Cand o = sm.list[f];
            rank += o.x > c.x || (o.x == c.x && o.token < c.token);
        }
        if (rank < n) out[rank] = c;
    }
    __syncthreads();
}

template <bool ALIGNED>
__global__ void __launch_bounds__(kBeamThreads) k_beam_select(const __grid_constant__ BeamArgs a) {
    __shared__ BeamSmem sm;
    cg::cluster_group cluster = cg::this_cluster();
    const int C = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
    const int b = blockIdx.x / C, tid = threadIdx.x;
    BeamSmem* head = cluster.map_shared_rank(&sm, 0);
    const int pieces = a.beams * a.splits;
    cluster.sync();                       // every CTA of the cluster runs: its shared memory may be written
    for (int p = rank; p < pieces; p += C) {
        const int k = p / a.splits, j = p % a.splits;
        const int begin = min(j * a.piece, a.vocab), end = min(begin + a.piece, a.vocab);
        if (a.finished && a.finished[b * a.beams + k] != 0) {
            // eos at no cost, then the lowest other tokens at -infinity; all in the row's first piece
            const int n = j == 0 ? min(a.n_out, a.vocab) : 0;
            if (tid < n) {
                const int other = tid - 1 + (tid - 1 >= a.eos);
                head->cand[p][tid] = tid == 0 ? Cand{0.f, a.eos} : Cand{-INFINITY, other};
            }
            if (tid == 0) {
                head->m[p] = j == 0 ? 0.f : -INFINITY;
                head->s[p] = j == 0 ? 1.f : 0.f;
                head->count[p] = n;
            }
            continue;
        }
        const float* row = a.logits + (size_t)(b * a.beams + k) * a.ld;
        scan_piece<ALIGNED>(sm, row, begin, end, a.n_out, head->cand[p], &head->m[p], &head->s[p], &head->count[p]);
        __syncthreads();
    }
    cluster.sync();
    if (rank != 0) return;
    // each row's maximum and log of its sum
    if (tid < a.beams) {
        float m = -INFINITY, s = 0.f;
        for (int j = 0; j < a.splits; ++j) m = fmaxf(m, sm.m[tid * a.splits + j]);
        const float ref = finite(m);
        for (int j = 0; j < a.splits; ++j) s = fmaf(sm.s[tid * a.splits + j], e2((finite(sm.m[tid * a.splits + j]) - ref) * kLog2E), s);
        sm.m_row[tid] = (double)m;
        sm.log_row[tid] = log((double)s);
    }
    __syncthreads();
    const int slots = pieces * kMaxOut;
    int total = 0;
    for (int p = 0; p < pieces; ++p) total += sm.count[p];
    // compact the candidates: slot e of piece p is number (sum of the counts before p) + e
    for (int i = tid; i < slots; i += kBeamThreads) {
        const int p = i / kMaxOut, e = i % kMaxOut;
        if (e >= sm.count[p]) continue;
        int at = e;
        for (int q = 0; q < p; ++q) at += sm.count[q];
        const Cand c = sm.cand[p][e];
        const int k = p / a.splits;
        const double m = sm.m_row[k], score = (double)a.scores[b * a.beams + k];
        // equal to the maximum (an infinite one included): no distance
        const double d = (double)c.x == m ? 0.0 : (double)c.x - m;
        double t = score + (d - sm.log_row[k]);
        if (a.finished && a.finished[b * a.beams + k] != 0) t = score + (double)c.x;
        if (c.x == -INFINITY || !(t == t)) t = -INFINITY;
        sm.total[at] = ordered(t);
        sm.tie[at] = ((unsigned long long)(kMaxBeams - 1 - k) << 56) | ((unsigned long long)ordered(c.x) << 24) |
                     (unsigned long long)((1 << 24) - 1 - c.token);
    }
    __syncthreads();
    for (int i = tid; i < total; i += kBeamThreads) {
        const unsigned long long t = sm.total[i], x = sm.tie[i];
        int r = 0;
        for (int f = 0; f < total; ++f) {
            const unsigned long long o = sm.total[f];
            r += o > t || (o == t && sm.tie[f] > x);
        }
        if (r < a.n_out) {
            const int k = kMaxBeams - 1 - (int)(x >> 56), token = (1 << 24) - 1 - (int)(x & 0xffffffu);
            const unsigned long long u = t >> 63 ? t & 0x7fffffffffffffffull : ~t;
            const int fin = a.finished ? (a.finished[b * a.beams + k] != 0 || token == a.eos) : 0;
            sm.list[r] = Cand{(float)__longlong_as_double((long long)u), token};
            sm.from[r] = make_int2(b * a.beams + k, fin);
        }
    }
    __syncthreads();                      // every read of scores and finished precedes the writes (they may be the same arrays)
    if (tid < a.n_out) {
        const size_t o = (size_t)b * a.n_out + tid;
        const int2 pf = sm.from[tid];
        a.next_tokens[o] = sm.list[tid].token;
        a.parents[o] = pf.x;
        a.next_scores[o] = sm.list[tid].x;
        if (a.next_finished) a.next_finished[o] = pf.y;
    }
    if (a.positions && tid < a.beams) a.positions[b * a.beams + tid] += 1;
}

}  // namespace
}  // namespace mk

extern "C" mk_status mk_beam_select(const float* logits, int64_t row_stride, int batch, int beams, int vocab, int n_out,
                                    const float* scores, const int32_t* finished, int32_t eos, int32_t* next_tokens,
                                    int32_t* parents, float* next_scores, int32_t* next_finished, int32_t* positions,
                                    void* stream) {
    if (!logits || !scores || !next_tokens || !parents || !next_scores) return MK_ERR_INVALID_ARG;
    if (batch < 1 || beams < 1 || vocab < 1 || n_out < 1 || row_stride < vocab) return MK_ERR_INVALID_ARG;
    if (beams > mk::kMaxBeams || n_out > mk::kMaxOut || vocab > (1 << 24) || batch > (1 << 20)) return MK_ERR_UNSUPPORTED;
    if ((int64_t)beams * vocab < n_out) return MK_ERR_INVALID_ARG;
    if (finished && (eos < 0 || eos >= vocab)) return MK_ERR_INVALID_ARG;
    if (next_finished && !finished) return MK_ERR_INVALID_ARG;
    if (reinterpret_cast<uintptr_t>(logits) & 3) return MK_ERR_INVALID_ARG;
    mk::BeamArgs a{};
    a.logits = logits;
    a.ld = row_stride;
    a.batch = batch;
    a.beams = beams;
    a.vocab = vocab;
    a.n_out = n_out;
    a.eos = finished ? eos : -1;
    a.scores = scores;
    a.finished = finished;
    a.next_tokens = next_tokens;
    a.parents = parents;
    a.next_scores = next_scores;
    a.next_finished = next_finished;
    a.positions = positions;
    int C = mk::kMaxCluster;
    while (C > 1 && (long long)batch * C > 2 * mk::kQSms) C /= 2;
    a.splits = C / beams > 1 ? C / beams : 1;
    a.piece = ((vocab + a.splits - 1) / a.splits + 3) / 4 * 4;
    if (C > beams * a.splits) C = beams * a.splits;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)(batch * C));
    cfg.blockDim = dim3(mk::kBeamThreads);
    cfg.stream = static_cast<cudaStream_t>(stream);
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeClusterDimension;
    at.val.clusterDim.x = (unsigned)C;
    at.val.clusterDim.y = at.val.clusterDim.z = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    const bool aligned = (reinterpret_cast<uintptr_t>(logits) & 15) == 0 && row_stride % 4 == 0;
    const cudaError_t e = aligned ? cudaLaunchKernelEx(&cfg, mk::k_beam_select<true>, static_cast<const mk::BeamArgs>(a))
                                  : cudaLaunchKernelEx(&cfg, mk::k_beam_select<false>, static_cast<const mk::BeamArgs>(a));
    return e == cudaSuccess && cudaGetLastError() == cudaSuccess ? MK_OK : MK_ERR_CUDA;
}
