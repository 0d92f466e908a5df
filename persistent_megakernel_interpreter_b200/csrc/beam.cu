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
// One cluster per sequence. The rows of its unfinished beams are cut into equal pieces, by token
// number and never by address, so equal rows give equal sums wherever they lie; a CTA takes a piece:
//   1. thread t reads tokens t, t + T, .. (every alignment alike: a warp reads 128 bytes in a row)
//      and keeps their maximum and running sum; from the maxima of 128 groups comes a bound that at least n
//      logits reach;
//   2. of the threads whose maximum reaches it (about n), each one's tokens are read again by its whole
//      warp at once, and what reaches the bound (about n) is gathered and ranked by counting.
// Each piece's maximum, sum and candidates go to CTA 0's shared memory (distributed
// shared memory), where one warp merges the ordered lists by total and writes the answer.
//
// Measured on one B200: 1 x 4 rows of 4096 in 6 us on the GPU, 2 x 4 rows of 128256 (3.1 MB read) in 9.7 us,
// 32 x 8 rows of 50257 (38.6 MB) in 17 us. What bounds it is the chain, not the bytes: for 2 x 4 rows about
// 1.0 us to the first load, 2.2 us of loads, 1.0 us to join the maxima, 1.2 us to gather, 0.3 us to rank, 0.8 us for the
// cluster's barrier, 1.7 us for totals and merging. (Keeping the logits in registers for the gathering
// spills: 10.2 and 20.5 us. As it is, the forms of 256 and 512 threads spill 8 bytes.)
#include <cooperative_groups.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <utility>

#include "qcache.h"

namespace mk {
namespace {

namespace cg = cooperative_groups;

constexpr int kMaxBeams = 16;
constexpr int kMaxOut = 32;
constexpr int kMaxPieces = 16;            // pieces of a sequence's rows: rows * splits
constexpr int kList = 1024;               // gathered logits of a piece
constexpr int kOwn = 8;                   // tokens a thread reads again by itself
constexpr int kLoads = 32;                // logits a thread has on the way at once
constexpr float kLog2E = 1.4426950408889634f;
constexpr float kBig = 3.402823466e38f;

struct BeamArgs {
    const float* logits;
    long long ld;
    int batch, beams, vocab, n_out, eos;
    const float* scores;
    const int32_t* finished;
    int32_t* next_tokens;
    int32_t* parents;
    float* next_scores;
    int32_t* next_finished;
    int32_t* positions;
    const int32_t* status;               // NULL, or where it is not 0 nothing is chosen
};

struct Cand {
    float x;
    int token;
};

// A candidate as two whole numbers that order it: its total, then beam, logit and token.
struct alignas(16) Key {
    unsigned long long total, tie;
};

struct BeamSmem {
    // CTA 0's: what every piece found
    Cand cand[kMaxPieces][kMaxOut];
    float m[kMaxPieces], s[kMaxPieces];
    float score[kMaxBeams], m_row[kMaxBeams];
    double log_row[kMaxBeams];
    Key key[kMaxPieces * kMaxOut];
    // each CTA's own
    Cand list[kList];
    alignas(16) float gmax[128];
    float wm[16], ws[16];
    int wcount[16];
    int n_list, n_tail;
    float again;
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

// x with NaN as -infinity: never chosen, adds nothing to the sum. (Maxima and comparisons pass NaN over
// by themselves; only sums need this, and only where there is one.)
__device__ __forceinline__ float clean(float x) { return fmaxf(x, -INFINITY); }

__device__ __forceinline__ float e2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// The finite number a maximum is subtracted as: an all-masked row has none, and a row
// of the type's lowest value keeps it.
__device__ __forceinline__ float finite(float m) { return fminf(fmaxf(m, -kBig), kBig); }

// The joint maximum and sum of N lanes: the maximum first, then each sum is rescaled once.
template <int N>
__device__ __forceinline__ void join_lanes(float& m, float& s) {
    float M = m;
#pragma unroll
    for (int k = N / 2; k > 0; k >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, k));
    s *= e2((m - finite(M)) * kLog2E);
#pragma unroll
    for (int k = N / 2; k > 0; k >>= 1) s += __shfl_xor_sync(0xffffffffu, s, k);
    m = M;
}

// A value that at least n of 128 (four per lane) reach, as large as it is cheap to find.
__device__ __forceinline__ float bound_of(float4 v, int n, int lane) {
    if (n <= 8) {
        // the n-th largest of the 32 lanes' maxima, equal ones counted by lane: about n logits of a row reach it
        const float x = fmaxf(fmaxf(v.x, v.y), fmaxf(v.z, v.w));
        int rank = 0;
#pragma unroll
        for (int i = 0; i < 32; ++i) {
            const float o = __shfl_sync(0xffffffffu, x, i);
            rank += o > x || (o == x && i < lane);
        }
        return __shfl_sync(0xffffffffu, x, __ffs(__ballot_sync(0xffffffffu, rank == n - 1)) - 1);
    }
    // more are wanted: the n-th of 32 maxima would let many times n through. The n-th largest of all 128, to
    // 16 bits (rounded down), bit by bit
    const uint32_t k[4] = {ordered(v.x), ordered(v.y), ordered(v.z), ordered(v.w)};
    uint32_t t = 0;
    for (int bit = 31; bit >= 16; --bit) {
        const uint32_t c = t | 1u << bit;
        if ((int)__reduce_add_sync(0xffffffffu, (k[0] >= c) + (k[1] >= c) + (k[2] >= c) + (k[3] >= c)) >= n) t = c;
    }
    if (t <= ordered(-INFINITY)) return -INFINITY;
    return __uint_as_float(t >> 31 ? t & 0x7fffffffu : ~t);
}

// A thread's share of tokens [begin, end): begin + t, begin + t + T, ..; its maximum and sum.
template <int T, bool CLEAN>
__device__ __forceinline__ void scan_tokens(const float* row, int begin, int end, float& m, float& s) {
    m = -INFINITY;
    s = 0.f;
    for (int i = begin + threadIdx.x; i < end; i += T * kLoads) {
        float v[kLoads], bm = -INFINITY;
#pragma unroll
        for (int u = 0; u < kLoads; ++u) v[u] = i + u * T < end ? row[i + u * T] : -INFINITY;
#pragma unroll
        for (int u = 0; u < kLoads; ++u) {
            if (CLEAN) v[u] = clean(v[u]);
            bm = fmaxf(bm, v[u]);
        }
        if (bm > m) {
            s *= e2((m - finite(bm)) * kLog2E);
            m = bm;
        }
        const float ref = finite(m);
        float part[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int u = 0; u < kLoads; ++u) part[u & 3] += e2((v[u] - ref) * kLog2E);
        s += (part[0] + part[1]) + (part[2] + part[3]);
    }
}

// Piece [begin, end) of one row: its maximum and sum, and its n best logits, best first, equal logits by
// token (padded with tokens -1 if it is shorter), into (out, *om, *os) by all threads.
template <int T>
__device__ __forceinline__ void scan_piece(BeamSmem& sm, const float* row, int begin, int end, int want, Cand* out, float* om,
                                           float* os) {
    constexpr int W = T / 32, GROUP = T / 128;   // warps; threads that share a group maximum
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int n = min(want, end - begin);
    float m, s;
    scan_tokens<T, false>(row, begin, end, m, s);
    float gm = m;
#pragma unroll
    for (int k = GROUP / 2; k > 0; k >>= 1) gm = fmaxf(gm, __shfl_xor_sync(0xffffffffu, gm, k));
    float cm = m, cs = s;
    join_lanes<32>(cm, cs);
    if ((lane & (GROUP - 1)) == 0) sm.gmax[tid / GROUP] = gm;
    if (lane == 0) {
        sm.wm[warp] = cm;
        sm.ws[warp] = cs;
    }
    if (tid == 0) sm.n_list = 0;
    const bool odd = __syncthreads_or(!(s <= kBig));
    float bound = n > 0 ? bound_of(reinterpret_cast<const float4*>(sm.gmax)[lane], n, lane) : INFINITY;
    if (odd) {
        // NaN or infinite logits: once more without the first, and infinite ones share the row, so that the sum
        // is their number
        const float reach = m;               // what the thread's numbers reach, for the gathering
        scan_tokens<T, true>(row, begin, end, m, s);
        const bool endless = __syncthreads_or(m == INFINITY);
        if (endless) {
            s = 0.f;
            for (int i = begin + tid; i < end; i += T) s += row[i] == INFINITY;
            m = INFINITY;
#pragma unroll
            for (int k = 16; k > 0; k >>= 1) s += __shfl_xor_sync(0xffffffffu, s, k);
        } else {
            join_lanes<32>(m, s);
        }
        if (lane == 0) {
            sm.wm[warp] = m;
            sm.ws[warp] = s;
        }
        m = reach;
        __syncthreads();
    }
    if (warp == W - 1) {
        cm = lane < W ? sm.wm[lane] : -INFINITY;
        cs = lane < W ? sm.ws[lane] : 0.f;
        if (__any_sync(0xffffffffu, cm == INFINITY)) {
            cm = INFINITY;
#pragma unroll
            for (int k = W / 2; k > 0; k >>= 1) cs += __shfl_xor_sync(0xffffffffu, cs, k);
        } else {
            join_lanes<W>(cm, cs);
        }
        if (lane == 0) {
            *om = cm;
            *os = cs;
        }
    }
    // gather what reaches the bound; where too much does (ties, or the best all with a few threads), only
    // what is above it; where that is still too much, raise the bound to the n-th of what was gathered
    bool above = bound == -INFINITY;
    for (;;) {
        const bool mine = n > 0 && (above ? m > bound : m >= bound);
        uint32_t hit = __ballot_sync(0xffffffffu, mine);
        if (end - begin <= kOwn * T) {
            // a short piece: each thread reads its own few again
            hit = 0;
            if (mine) {
                float x[kOwn];
#pragma unroll
                for (int u = 0; u < kOwn; ++u) x[u] = begin + tid + u * T < end ? row[begin + tid + u * T] : NAN;
#pragma unroll
                for (int u = 0; u < kOwn; ++u)
                    if (above ? x[u] > bound : x[u] >= bound) {
                        const int at = atomicAdd(&sm.n_list, 1);
                        if (at < kList) sm.list[at] = Cand{x[u], begin + tid + u * T};
                    }
            }
        }
        while (hit) {
            // two owners at once: their tokens by lanes, 128 a round each
            int owner[2];
#pragma unroll
            for (int o = 0; o < 2; ++o) {
                owner[o] = hit ? begin + warp * 32 + __ffs(hit) - 1 : end;
                hit &= hit - 1;
            }
            for (int step = lane * T; step < end - begin; step += 128 * T) {
                float x[2][4];
#pragma unroll
                for (int o = 0; o < 2; ++o)
#pragma unroll
                    for (int u = 0; u < 4; ++u) {
                        const int i = owner[o] + step + u * 32 * T;
                        x[o][u] = i < end ? row[i] : NAN;
                    }
#pragma unroll
                for (int o = 0; o < 2; ++o)
#pragma unroll
                    for (int u = 0; u < 4; ++u)
                        if (above ? x[o][u] > bound : x[o][u] >= bound) {
                            const int at = atomicAdd(&sm.n_list, 1);
                            if (at < kList) sm.list[at] = Cand{x[o][u], owner[o] + step + u * 32 * T};
                        }
            }
        }
        __syncthreads();
        const int found = sm.n_list;
        if (found <= kList) break;
        if (above) {
            // the n-th largest value of the list
            for (int e = tid; e < kList; e += T) {
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
        for (int base = begin; base < end; base += T) {
            const int have = sm.n_tail;
            if (have >= n) break;
            const int i = base + tid;
            const bool eq = i < end && clean(row[i]) == bound;
            const uint32_t mask = __ballot_sync(0xffffffffu, eq);
            if (lane == 0) sm.wcount[warp] = __popc(mask);
            __syncthreads();
            int at = have, all = have;
            for (int w = 0; w < W; ++w) {
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
    for (int e = tid; e < found; e += T) {
        const Cand c = sm.list[e];
        int rank = 0;
        for (int f = 0; f < found; ++f) {
            const Cand o = sm.list[f];
            rank += o.x > c.x || (o.x == c.x && o.token < c.token);
        }
        if (rank < n) out[rank] = c;
    }
    if (tid >= n && tid < want) out[tid] = Cand{-INFINITY, -1};
}

template <int T>
__global__ void __launch_bounds__(T, 1024 / T) k_beam_select(const __grid_constant__ BeamArgs a) {
    __shared__ BeamSmem sm;
    cg::cluster_group cluster = cg::this_cluster();
    const int C = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
    const int b = blockIdx.x / C, tid = threadIdx.x, lane = tid & 31;
    cudaGridDependencySynchronize();           // everything enqueued before has run
    if (a.status && *a.status != 0) {          // the same for every CTA: none waits for another
        const unsigned per = cluster.num_blocks(), at = blockIdx.x / per * a.n_out + threadIdx.x;
        if (blockIdx.x % per == 0 && threadIdx.x < a.n_out) a.parents[at] = -1;
        return;
    }
    auto running = cluster.barrier_arrive();   // waited for before another CTA's shared memory is written
    BeamSmem* head = cluster.map_shared_rank(&sm, 0);
    const int n = min(a.n_out, a.vocab);
    // the finished beams, as bits; the others' rows are cut into `splits` pieces each, numbered piece by
    // piece in the order of the beams, then one piece for each finished beam
    const bool mine = a.finished && lane < a.beams && a.finished[b * a.beams + (lane < a.beams ? lane : 0)] != 0;
    const uint32_t done = __ballot_sync(0xffffffffu, mine), open = ((1u << a.beams) - 1u) & ~done;
    const int rows = __popc(open);
    const int splits = rows ? max(1, min(kMaxPieces - (a.beams - rows), C) / rows) : 1;
    const int pieces = rows * splits + a.beams - rows;
    auto beam_of = [&](int p) {          // the beam of piece p
        uint32_t left = p < rows * splits ? open : done;
        for (int i = p < rows * splits ? p / splits : p - rows * splits; i > 0; --i) left &= left - 1;
        return __ffs(left) - 1;
    };
    if (rank == 0 && tid < a.beams) sm.score[tid] = a.scores[b * a.beams + tid];
    bool waited = false;
    for (int p = rank; p < pieces; p += C) {
        const int k = beam_of(p);
        if (p >= rows * splits) {
            // eos at no cost, then the lowest other tokens at -infinity
            if (!waited) cluster.barrier_wait(std::move(running));
            waited = true;
            if (tid < n) {
                const int other = tid - 1 + (tid - 1 >= a.eos);
                head->cand[p][tid] = tid == 0 ? Cand{0.f, a.eos} : Cand{-INFINITY, other};
            }
            continue;
        }
        const int size = (a.vocab + splits - 1) / splits;
        const int begin = min(p % splits * size, a.vocab), end = min(begin + size, a.vocab);
        const float* row = a.logits + (size_t)(b * a.beams + k) * a.ld;
        if (!waited) cluster.barrier_wait(std::move(running));
        waited = true;
        scan_piece<T>(sm, row, begin, end, n, head->cand[p], &head->m[p], &head->s[p]);
        __syncthreads();
    }
    if (!waited) cluster.barrier_wait(std::move(running));
    auto told = cluster.barrier_arrive();
    if (rank != 0) return;               // nothing of this CTA is read by others
    cluster.barrier_wait(std::move(told));
    // each unfinished row's maximum and the logarithm of its sum, joined from its pieces
    if (tid < rows) {
        const int k = beam_of(tid * splits), p0 = tid * splits;
        float m = -INFINITY, s = 0.f;
        for (int j = 0; j < splits; ++j) m = fmaxf(m, sm.m[p0 + j]);
        const float ref = finite(m);
        // beside an infinite maximum only the pieces that have one count: their sums are its numbers
        for (int j = 0; j < splits; ++j)
            s = fmaf(sm.s[p0 + j], m == INFINITY ? (float)(sm.m[p0 + j] == INFINITY) : e2((finite(sm.m[p0 + j]) - ref) * kLog2E), s);
        sm.m_row[k] = m;
        sm.log_row[k] = log((double)s);
    }
    __syncthreads();
    // every candidate's total
    const int total = pieces * n;
    for (int i = tid; i < total; i += T) {
        const int p = i / n, k = beam_of(p);
        const Cand c = sm.cand[p][i % n];
        const double score = (double)sm.score[k];
        double t;
        if (done >> k & 1) {
            t = score + (double)c.x;
        } else {
            // equal to the maximum (an infinite one included): no distance
            const float m = sm.m_row[k];
            const double d = c.x == m ? 0.0 : (double)c.x - (double)m;
            t = score + (d - sm.log_row[k]);
        }
        if (c.x == -INFINITY || !(t == t)) t = -INFINITY;
        Key key{0ull, 0ull};             // below every candidate
        if (c.token >= 0)
            key = Key{ordered(t), ((unsigned long long)(kMaxBeams - 1 - k) << 56) | ((unsigned long long)ordered(c.x) << 24) |
                                      (unsigned long long)((1 << 24) - 1 - c.token)};
        sm.key[i] = key;
    }
    __syncthreads();
    if (a.positions && tid < a.beams) a.positions[b * a.beams + tid] += 1;
    if (tid >= 32) return;
    // the best of the heads of the pieces' ordered lists, n_out times: lane p holds piece p's. The next one
    // that a list would offer is read while the others are compared.
    const Key none{0ull, 0ull};
    Key mine_now = lane < pieces ? sm.key[lane * n] : none, won = none;
    int used = 0;
    for (int r = 0; r < a.n_out; ++r) {
        const Key next = lane < pieces && used + 1 < n ? sm.key[lane * n + used + 1] : none;
        // the largest (total, tie), 32 bits at a time while more than one lane has it
        uint32_t left = 0xffffffffu;
#pragma unroll
        for (int part = 0; part < 4; ++part) {
            const unsigned long long word = part < 2 ? mine_now.total : mine_now.tie;
            const uint32_t v = left >> lane & 1 ? (uint32_t)(part & 1 ? word : word >> 32) : 0u;
            const uint32_t most = __reduce_max_sync(0xffffffffu, v);
            left &= __ballot_sync(0xffffffffu, v == most);
            if (!(left & (left - 1))) break;
        }
        const int winner = __ffs(left) - 1;
        const Key best{__shfl_sync(0xffffffffu, mine_now.total, winner), __shfl_sync(0xffffffffu, mine_now.tie, winner)};
        if (lane == r) won = best;
        if (lane == winner) {
            mine_now = next;
            ++used;
        }
    }
    if (lane < a.n_out) {
        const size_t o = (size_t)b * a.n_out + lane;
        const int k = kMaxBeams - 1 - (int)(won.tie >> 56), token = (1 << 24) - 1 - (int)(won.tie & 0xffffffu);
        const unsigned long long u = won.total >> 63 ? won.total & 0x7fffffffffffffffull : ~won.total;
        a.next_tokens[o] = token;
        a.parents[o] = b * a.beams + k;
        a.next_scores[o] = (float)__longlong_as_double((long long)u);
        if (a.next_finished) a.next_finished[o] = (done >> k & 1) || token == a.eos;
    }
}

template <int T>
cudaError_t launch_beam(const BeamArgs& a, int C, cudaStream_t st) {
    static std::atomic<uint64_t> seen{0};
    if (first_on_device(seen)) {
        const cudaError_t e = cudaFuncSetAttribute(k_beam_select<T>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        if (e != cudaSuccess) return e;
        seen_on_device(seen);
    }
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)(a.batch * C));
    cfg.blockDim = dim3(T);
    cfg.stream = st;
    cudaLaunchAttribute at[2]{};
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = (unsigned)C;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    // placed while the kernel before it ends; it waits for all of that before it reads or writes
    at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, k_beam_select<T>, a);
}

}  // namespace
}  // namespace mk

namespace mk {
static mk_status beam_select(const float* logits, int64_t row_stride, int batch, int beams, int vocab, int n_out,
                             const float* scores, const int32_t* finished, int32_t eos, int32_t* next_tokens,
                             int32_t* parents, float* next_scores, int32_t* next_finished, int32_t* positions,
                             const int32_t* status, void* stream) {
    if (!logits || !scores || !next_tokens || !parents || !next_scores) return MK_ERR_INVALID_ARG;
    if (batch < 1 || beams < 1 || vocab < 1 || n_out < 1 || row_stride < vocab) return MK_ERR_INVALID_ARG;
    if (beams > mk::kMaxBeams || n_out > mk::kMaxOut || vocab > (1 << 24) || batch > (1 << 20)) return MK_ERR_UNSUPPORTED;
    if ((int64_t)beams * vocab < n_out) return MK_ERR_INVALID_ARG;
    if (finished && (eos < 0 || eos >= vocab)) return MK_ERR_INVALID_ARG;
    if (next_finished && !finished) return MK_ERR_INVALID_ARG;
    // in place, a sequence's results may not lie where another's are still read
    if (batch > 1 && n_out != beams && (next_scores == scores || (finished && next_finished == finished))) return MK_ERR_INVALID_ARG;
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
    a.status = status;
    // CTAs per sequence. Few sequences with long rows or many beams take 16 (2 x 4 rows of 128256: 9.0 us against 11
    // with 8); a moderate number at least 8 (8 rows of 128256: 7.7 us, 11.4 with 16; 32 x 8 of 50257: 17,
    // 29 with 16); from there on a CTA takes a whole row (64 x 4 of 32000: 12.0 us, 20.3 with 8), of many sequences
    // with many beams two (20 x 12 of 32000: 16.3 us with 12 CTAs, 25.6 with 8; 100 x 16: 80 with 16, 69 with 8).
    const int most = batch <= 64 ? 16 : 8;
    int C = beams < most ? beams : most;
    if (batch <= 4 && (beams > 8 || (int64_t)beams * vocab >= 1 << 18)) C = 16;
    else if (batch <= 32 && C < 8) C = 8;
    // Threads by the piece's length: long pieces want loads on the way (32 x 4 rows of 128256: 20.4 us with 512,
    // 23.3 with 256), short ones several CTAs on an SM (512 x 4 rows of 4096: 16.7 us with 128, 30.5 with 256).
    const int tokens = vocab / (C > beams ? C / beams : 1);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const cudaError_t e = tokens >= 16384 ? mk::launch_beam<512>(a, C, st)
                          : tokens >= 6144 ? mk::launch_beam<256>(a, C, st)
                                           : mk::launch_beam<128>(a, C, st);
    return e == cudaSuccess ? MK_OK : MK_ERR_CUDA;
}
}  // namespace mk

extern "C" mk_status mk_beam_select(const float* logits, int64_t row_stride, int batch, int beams, int vocab, int n_out,
                                    const float* scores, const int32_t* finished, int32_t eos, int32_t* next_tokens,
                                    int32_t* parents, float* next_scores, int32_t* next_finished, int32_t* positions,
                                    void* stream) {
    return mk::beam_select(logits, row_stride, batch, beams, vocab, n_out, scores, finished, eos, next_tokens, parents,
                           next_scores, next_finished, positions, nullptr, stream);
}

extern "C" mk_status mk_beam_select_checked(const float* logits, int64_t row_stride, int batch, int beams, int vocab,
                                            int n_out, const float* scores, const int32_t* finished, int32_t eos,
                                            int32_t* next_tokens, int32_t* parents, float* next_scores,
                                            int32_t* next_finished, int32_t* positions, const int32_t* status,
                                            void* stream) {
    if (!status) return MK_ERR_INVALID_ARG;
    return mk::beam_select(logits, row_stride, batch, beams, vocab, n_out, scores, finished, eos, next_tokens, parents,
                           next_scores, next_finished, positions, status, stream);
}
