// The 8-bit KV cache: storing new keys and values, and decode attention over it.
//
// A block is kQBlock = 32 tokens of one (layer, row, head), of keys or of values:
//   scale = amax / 127 (amax the block's largest magnitude), code = rint(x * (127 / amax)), int8.
// The tokens of a row's open block (the last length % 32 of them) stay bf16 in the
// tail buffers until the block is full, so a code is rounded once, from the token's
// own bf16 value, and never again.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>

#include "qcache.h"

namespace mk {
namespace {

// ------------------------------------------------------------------ append

constexpr int kAppWarps = 4;

struct AppendArgs {
    uint8_t* codes[2];            // keys, values
    float* scale[2];
    uint16_t* tail[2];
    const uint16_t* src[2];
    long long sl, sr, sh, st;     // source strides in elements: layer, row, head, token
    int first_layer, n_layers, max_batch, n_heads, max_seq, n_blocks, rows, n_new;
    const int32_t* positions;
    const int32_t* counts;        // NULL: n_new each
};

constexpr float kRound = 12582912.0f;  // 1.5 * 2^23

__device__ __forceinline__ float bf(uint32_t bits16) { return __uint_as_float(bits16 << 16); }

// A team of HD / 64 warps per (keys or values, layer, row, head, block of the row's window). The
// window starts at the row's open block: `held` tokens already in the tail, then the new ones. A
// thread holds four pieces of 16 elements of one token each (32 registers), so codes are written in
// full 16-byte pieces. The block that stays open is written by the team of window block 0, after it
// has read the tail's old tokens.
//
// Bound by HBM (2 bytes in, 1 out). Small CTAs at 64 registers a thread: 16 layers of four prompts of
// up to 4001 tokens (688 MB) in 101 us in a graph, 104% of the measured copy rate, and 101 to 103 as calls (145 us with 8 warps a CTA, one warp a
// block and 79 registers); one token of eight rows in 1.3 us.
template <int HD>
__global__ void __launch_bounds__(32 * kAppWarps, 8) k_append(const __grid_constant__ AppendArgs a) {
    constexpr int TEAM = HD / 64, TL = 32 * TEAM, TEAMS = kAppWarps / TEAM;
    constexpr int IT = 4;                    // pieces of a thread
    constexpr int PPT = HD / 16;             // pieces of a token
    static_assert(IT * TL * 16 == kQBlock * HD, "a team covers a block");
    __shared__ float team_max[kAppWarps];
    cudaGridDependencySynchronize();         // everything enqueued before has run
    const int tl = threadIdx.x % TL, team = threadIdx.x / TL;
    const int wb = blockIdx.x * TEAMS + team;                     // window block
    const int h = blockIdx.y % a.n_heads, r = blockIdx.y / a.n_heads;
    const int which = blockIdx.z & 1, l = blockIdx.z >> 1;
    const int pos = a.positions[r];
    const int cnt = a.counts ? a.counts[r] : a.n_new;
    if (pos < 0 || cnt < 1 || cnt > a.n_new || pos > a.max_seq - cnt) return;
    const int held = pos % kQBlock, end = held + cnt;
    const int closed = end / kQBlock;        // window blocks that are full now
    if (blockIdx.x * TEAMS >= max(closed, 1)) return;
    const size_t plane = ((size_t)(a.first_layer + l) * a.max_batch + r) * a.n_heads + h;
    uint16_t* tail = a.tail[which] + plane * (kQBlock * HD);
    const uint16_t* src = a.src[which] + l * a.sl + r * a.sr + h * a.sh;
    const bool full = wb < closed;
    uint4 x[IT][2];
    float big = 0.f;                         // of magnitudes; NaN and infinity count as infinity
    if (full) {
#pragma unroll
        for (int j = 0; j < IT; ++j) {
            const int piece = j * TL + tl, tok = wb * kQBlock + piece / PPT, e = (piece % PPT) * 16;
            const uint16_t* p = tok < held ? tail + tok * HD + e : src + (tok - held) * a.st + e;
            x[j][0] = *reinterpret_cast<const uint4*>(p);
            x[j][1] = *reinterpret_cast<const uint4*>(p + 8);
        }
        // magnitudes order as their bits do: the largest of packed pairs, then of the two halves
        uint32_t top = 0;
#pragma unroll
        for (int j = 0; j < IT; ++j)
#pragma unroll
            for (int i = 0; i < 8; ++i) top = __vmaxu2(top, (&x[j][i / 4].x)[i % 4] & 0x7fff7fffu);
        top = max(top >> 16, top & 0xffffu);
        top = __reduce_max_sync(0xffffffffu, top);
        big = __uint_as_float(top << 16);
    }
    if (TEAM > 1) {
        if ((threadIdx.x & 31) == 0) team_max[threadIdx.x >> 5] = big;
        __syncthreads();
        // not fmaxf, which would pass a NaN over: the larger bits
        big = __uint_as_float(max(__float_as_uint(team_max[team * TEAM]), __float_as_uint(team_max[team * TEAM + TEAM - 1])));
    }
    if (full) {
        // a block with an infinity or a NaN gets a NaN scale: what attends to it is NaN
        const bool bad = __float_as_uint(big) >= 0x7f800000u, some = big >= kQNoBlock && !bad;
        const float inv = some ? __fdiv_rn(127.0f, big) : 0.f;
        const int blk = pos / kQBlock + wb;
        uint8_t* codes = a.codes[which] + (plane * a.max_seq + (size_t)blk * kQBlock) * HD;
#pragma unroll
        for (int j = 0; j < IT; ++j) {
            uint4 out;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                // |x| <= amax, so |x * inv| <= 127 (1 + 2^-23) and rounds to at most 127. With 1.5 * 2^23
                // added the sum's last bits are the rounded product (to nearest, ties to even, as rint)
                uint32_t c[4];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int k = q * 2 + i;
                    const uint32_t w = (&x[j][k / 4].x)[k % 4];
                    c[2 * i] = __float_as_uint(__fadd_rn(__fmul_rn(bf(w & 0xffffu), inv), kRound));
                    c[2 * i + 1] = __float_as_uint(__fadd_rn(__fmul_rn(__uint_as_float(w & 0xffff0000u), inv), kRound));
                }
                (&out.x)[q] = __byte_perm(__byte_perm(c[0], c[1], 0x0040), __byte_perm(c[2], c[3], 0x0040), 0x5410);
            }
            *reinterpret_cast<uint4*>(codes + (j * TL + tl) * 16) = bad ? make_uint4(0u, 0u, 0u, 0u) : out;
        }
        if (tl == 0)
            a.scale[which][plane * a.n_blocks + blk] = bad ? __int_as_float(0x7fffffff) : some ? __fdiv_rn(big, 127.0f) : 0.f;
    }
    if (wb == 0) {
        __syncwarp();
        // the open block's new tokens
        const int t0 = closed > 0 ? 0 : held, n = end - closed * kQBlock;
        for (int piece = t0 * PPT + tl; piece < n * PPT; piece += TL) {
            const int tok = piece / PPT, e = (piece % PPT) * 16;
            const uint16_t* p = src + (closed * kQBlock + tok - held) * a.st + e;
            const uint4 u = *reinterpret_cast<const uint4*>(p), v = *reinterpret_cast<const uint4*>(p + 8);
            *reinterpret_cast<uint4*>(tail + tok * HD + e) = u;
            *reinterpret_cast<uint4*>(tail + tok * HD + e + 8) = v;
        }
    }
}

// ------------------------------------------------------------------ attention
//
// out[h] = sum_i softmax_i(q[h] . k_i / sqrt(d)) v_i over slots i = 0 .. pos, for the
// group's query heads h of one (row, KV head).
//
// The codes are int8, so both products run on the tensor cores' integer path
// (mma.sync m16n8k32, exact 32-bit sums) without a conversion of any code: the other
// operand is cut into four 8-bit digits, which fill the 16 rows of A for 4 heads. Head
// h has its digits 3 and 2 in rows h and h + 8, digits 1 and 0 in rows h + 4 and
// h + 12, so lanes of groups g < 4 and g >= 4 hold two digits each of head g % 4.
//   scores:  q as 30-bit whole numbers (its head's largest magnitude sets the step)
//   outputs: weights as 32-bit whole numbers, 2^31 m 2^(s + e - M), where 2^e m is the
//            block's value scale (1 <= m < 2) and M the running maximum of s + e, rounded up
// The softmax's sum l is that of 2^(s - M + 39): of the scores alone, for the weight of a block whose values
// are far smaller than another's rounds to nothing while its keys still count. With -67 <= e <= 121 (blocks
// below 2^-60 are zeros, and a block of zeros counts as e = -67, so that it never sets the size that
// others' weights are held relative to) a term is at most 2^106, 2^20 of them stay finite, and one that is flushed
// to zero is below 2^-44 of the largest. M is a whole number, so every change of unit is by an exact
// power of two; one exponential serves a key's weight and its term of the sum.
// Accumulators start at the bits of 1.5 * 2^23, so that read as a float they are that
// plus the sum (below 2^22 in magnitude: 128 * 127 * 128 in a score, 255 * 127 * 64 in
// an output), and one FMA turns each into its share of the fp32 result.
//
// A score is rounded once to fp32 and is the same number in the maximum and in its weight, whatever its size.
// Keys behind a cut inside a closed block get a score of -infinity.
//
// A warp works alone on a batch of 8 KB (64 keys and values of 64 dims, 32 of 128), with
// a running (M, l, O) of its own, fed by a private ring of asynchronous copies; the warps
// join at the end.
//
// Bound by HBM: 2 * dim bytes a key and KV head. Measured on one B200, in a graph (as calls in a stream): 4 rows of
// up to 60001 keys of 128 dims (307 MB) in 50.8 us (52 to 54), 6.05 TB/s, 92% of the measured copy rate; 8 rows of up to
// 16384 keys of 64 dims (105 MB) in 21.7 us (22.1), 74%; 129 keys in 3.2 us (3.4); one row of 16384 keys and 8 heads
// in 7.9 us of 64 dims, 11.4 of 128. Around the stream of bytes there are about 5 us: 1.5 to launch, 0.7
// for the plan, 1 until the first batch is here, 0.6 to join a CTA's warps, 1.5 for the joining kernel. As fp16
// products (codes converted, the other operand in two parts) the two long ones took 32 and 114 us at first and 30
// and 72 with the rings: twice the instructions for half the products.

constexpr int kAttWarps = 4;
// Batches in a warp's ring, and CTAs an SM holds: two of the 64-dim split's CTAs (253 registers a thread), with a batch
// more on the way each; three at 128 dims (168 registers, 8 bytes of spills). 8 x 16384 keys of 64 dims: 21.7 us, 21.8 with
// (2, 3); 4 x 60001 of 128 dims: 50.8 us, 53.1 with (3, 2).
__host__ __device__ constexpr int attn_stages(int hd) { return hd == 64 ? 3 : 2; }
__host__ __device__ constexpr int attn_per_sm(int hd) { return hd == 64 ? 2 : 3; }
constexpr int kHalf = 4096;            // bytes of a batch's keys, and of its values
__host__ __device__ constexpr int batch_blocks(int hd) { return hd == 64 ? 2 : 1; }
constexpr float kLowest = -3.402823466e38f;   // maxima are finite: a difference of two is a number or an infinity
constexpr float kLog2e = 1.4426950408889634f;

struct AttnArgs {
    const uint8_t* codes[2];
    const float* scale[2];
    const uint16_t* tail[2];
    int layer, max_batch, n_heads, group, max_seq, n_blocks, rows, max_ctx;
    const float* q;               // [rows][n_heads * group][HD]
    const int32_t* positions;
    const int32_t* lengths;       // tokens that each row holds; NULL: positions[row] + 1
    float* out;
    float* part_ml;               // [slots][group][2]
    float* part_o;                // [slots][group][HD]
    int n_cta;                    // CTAs of the split over blocks (0: one CTA per (row, head), no partials)
};

__device__ __forceinline__ uint32_t smem32(const void* p) { return static_cast<uint32_t>(__cvta_generic_to_shared(p)); }
__device__ __forceinline__ void copy16(void* dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void copy4(void* dst, const void* src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
constexpr int kLeastScale = -67;       // of a value block: 2^-60 / 127 = 1.008 * 2^-67
constexpr int kSumBits = 39;           // sums are in units of 2^(M - 39)
constexpr float kSumUnit = 0x1p39f;
// Powers of two for whole numbers d <= 0, from d's place in the bits of kMagic + d: 2^d itself (no less than 2^-126)
// and l 2^d for a sum l (positive, or a NaN that stays one), to which d may do more than one number holds.
constexpr uint32_t kMagicBits = 0x4b400000u;
constexpr float kMagic = 12582912.0f;  // 1.5 * 2^23
__device__ __forceinline__ float pow2(float d) { return __uint_as_float(__float_as_uint(fmaxf(d, -126.0f) + (kMagic + 127.0f)) << 23); }
__device__ __forceinline__ float scaled(float l, float d) {
    const int by = (int)(__float_as_uint(fmaxf(d, -252.0f) + kMagic) << 23);
    return fmaf(l, 0.0f, __int_as_float(max(__float_as_int(l) + by, 0)));
}

// C += A B, C read and written as 32-bit whole numbers; A's bytes signed (queries) or not (weights).
__device__ __forceinline__ void mma_s8(uint32_t (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+r"(c[0]), "+r"(c[1]), "+r"(c[2]), "+r"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_u8(uint32_t (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k32.row.col.s32.u8.s8.s32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+r"(c[0]), "+r"(c[1]), "+r"(c[2]), "+r"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// (the sum in accumulator c) * mul, exact for a power of two
__device__ __forceinline__ float sum_of(uint32_t c, float mul) { return fmaf(__uint_as_float(c), mul, -kMagic * mul); }

// A CTA's running result of one (row, KV head): per warp (and the open block) a maximum, a
// sum and an output per head, joined at the end; and each warp's ring of batches.
template <int HD>
struct AttnSmem {
    static constexpr int kStages = attn_stages(HD);
    alignas(16) uint8_t ring[kAttWarps][kStages][2][kHalf];
    float scale[kAttWarps][kStages][2][2];   // keys' and values', of the batch's blocks
    alignas(16) float tail_o[kMaxGroupHeads][HD];
    float m[kAttWarps + 1][kMaxGroupHeads];
    float l[kAttWarps + 1][kMaxGroupHeads];
    // The queries, in quarters of a head (what one lane of a fragment reads) 16 bytes apart, so that the
    // lanes' 16-byte reads meet every bank once.
    static constexpr int kQuarter = HD / 4 + 4;
    alignas(16) float q[kMaxGroupHeads][4][kQuarter];
    __device__ __forceinline__ float& query(int h, int d) { return q[h][d / (HD / 4)][d % (HD / 4)]; }
    // Part p's output of head h, dim d: a warp's lie in its own ring once the ring is drained, an eighth of a
    // head (what one lane writes) and the heads 16 bytes apart, for the same reason.
    static constexpr int kEighth = HD / 8 + 4, kHead = 8 * kEighth + 4;
    __device__ __forceinline__ float* warp_o(int p, int h) { return reinterpret_cast<float*>(ring[p]) + h * kHead; }
    __device__ __forceinline__ float o(int p, int h, int d) {
        return p == kAttWarps ? tail_o[h][d] : warp_o(p, h)[d / (HD / 8) * kEighth + d % (HD / 8)];
    }
};
static_assert(kMaxGroupHeads * AttnSmem<128>::kHead * sizeof(float) <= 2 * kHalf, "a warp's outputs lie in its ring");

// The 16-byte piece c of row r sits at piece swizzled(r, c) of its row, so that the
// fragment reads below meet every bank once: of eight lanes that read a piece of keys in
// one cycle, two rows come with the even or the odd pieces each; of the lanes that read
// values, four rows two apart with two pieces each.
template <int HD>
__device__ __forceinline__ int swizzled(int r, int c) {
    return HD == 64 ? c ^ (r >> 1 & 3) : c ^ (r & 7);
}

// A batch's keys and values, of which `blocks` blocks are there, and their scales.
template <int HD>
__device__ __forceinline__ void fetch_batch(AttnSmem<HD>& sm, int warp, int lane, int stage, const uint8_t* k, const uint8_t* v,
                                            const float* ks, const float* vs, int blocks) {
    constexpr int CPR = HD / 16, PER = kQBlock * HD / 512;   // pieces of a row; of a block, per lane
#pragma unroll
    for (int b = 0; b < batch_blocks(HD); ++b)
        if (b < blocks) {
#pragma unroll
            for (int j = b * PER; j < (b + 1) * PER; ++j) {
                const int i = j * 32 + lane, r = i / CPR, c = i % CPR;
                const int at = r * HD + 16 * swizzled<HD>(r, c);
                copy16(&sm.ring[warp][stage][0][at], k + i * 16);
                copy16(&sm.ring[warp][stage][1][at], v + i * 16);
            }
        }
    if (lane < 2 * blocks) copy4(&sm.scale[warp][stage][lane & 1][lane >> 1], (lane & 1 ? vs : ks) + (lane >> 1));
}

// The closed blocks [b0, b1) of one (row, KV head), of whose slots those below `keys` are attended to: where they
// lie, and a warp's fetches of them. Warp w takes the batches at b0 + (w + 4 i) batch_blocks.
template <int HD>
struct AttnSource {
    const uint8_t *k, *v;
    const float *ks, *vs;
    int b0, b1, keys;
    __device__ __forceinline__ AttnSource(const AttnArgs& a, size_t plane, int first, int last, int n)
        : b0(first), b1(last), keys(min(n, last * kQBlock)) {
        k = a.codes[0] + plane * a.max_seq * HD;
        v = a.codes[1] + plane * a.max_seq * HD;
        ks = a.scale[0] + plane * a.n_blocks;
        vs = a.scale[1] + plane * a.n_blocks;
    }
    __device__ __forceinline__ int first(int warp) const { return b0 + warp * batch_blocks(HD); }
    static constexpr int kStep = kAttWarps * batch_blocks(HD);
    __device__ __forceinline__ void fetch(AttnSmem<HD>& sm, int warp, int lane, int blk, int stage) const {
        if (blk < b1)
            fetch_batch<HD>(sm, warp, lane, stage, k + (size_t)blk * (kQBlock * HD), v + (size_t)blk * (kQBlock * HD), ks + blk,
                            vs + blk, min(batch_blocks(HD), b1 - blk));
        copy_commit();
    }
    // The first batches, before anything else is done for these blocks.
    __device__ __forceinline__ void start(AttnSmem<HD>& sm, int warp, int lane) const {
#pragma unroll
        for (int i = 0; i < attn_stages(HD) - 1; ++i) fetch(sm, warp, lane, first(warp) + i * kStep, i);
    }
};

// The blocks of src by the CTA's warps, into part `warp` of sm. src.start() has run.
template <int HD>
__device__ __forceinline__ void attn_blocks(const AttnArgs& a, AttnSmem<HD>& sm, const AttnSource<HD>& src, int warp,
                                            int lane) {
    constexpr int BB = batch_blocks(HD), kStages = attn_stages(HD);
    constexpr int KEYS = BB * kQBlock, NT = KEYS / 8;   // keys of a batch, 8-key tiles
    constexpr int C = HD / 64;               // 16-byte pieces of a key per lane: C t, C t + 1, ..
    constexpr int VD = HD / 8;               // dims of a value per lane: VD g, VD g + 1, ..
    const int g = lane >> 2, t = lane & 3, head = g & 3;
    const bool up = g >= 4;
    // A of the scores: digits of q. K step j of a tile covers the lane's dims 16 (j / 2) + 8 (j % 2)
    // + 0 .. 7 behind (HD / 4) t.
    uint32_t qa[2 * C][4];
    float kmul;
    const uint32_t sel_q = up ? 0x5140u : 0x7362u;   // (lower, lower, upper, upper) digits of two elements
    {
        float big = 0.f, q[HD / 4];
        bool bad = false;
#pragma unroll
        for (int e = 0; e < HD / 4; e += 4) {
            const float4 v = *reinterpret_cast<const float4*>(&sm.q[head < a.group ? head : 0][t][e]);
            q[e] = v.x; q[e + 1] = v.y; q[e + 2] = v.z; q[e + 3] = v.w;
        }
#pragma unroll
        for (int e = 0; e < HD / 4; ++e) {
            big = fmaxf(big, fabsf(q[e]));
            bad |= !(fabsf(q[e]) < INFINITY);
        }
        big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 1));
        big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 2));
        bad |= __shfl_xor_sync(0xffffffffu, bad, 1);
        bad |= __shfl_xor_sync(0xffffffffu, bad, 2);
        // |q| < 2^(ex + 1) becomes a whole number below 2^30, its digits within -128 .. 127
        int ex = big > 0.f && !bad ? ilogbf(big) : 0;
        ex = max(ex, -90);
        const float step = exp2f((float)(29 - ex));
        kmul = bad ? __int_as_float(0x7fffffff) : exp2f((float)(ex - 29)) * (HD == 64 ? 0.125f : 0.08838834764831845f) * kLog2e;
#pragma unroll
        for (int j = 0; j < 2 * C; ++j)
#pragma unroll
            for (int w = 0; w < 2; ++w) {
                // x = sum of d_i 256^i with d_i in -128 .. 127: the bytes of x + 0x808080 are d_i + 128 but
                // for the top one, and d_i itself once the added bits are flipped
                uint32_t x[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int v = head < a.group ? __float2int_rn(q[16 * (j / 2) + 8 * (j % 2) + 4 * w + e] * step) : 0;
                    x[e] = ((uint32_t)v + 0x808080u) ^ 0x808080u;
                }
                const uint32_t p = __byte_perm(x[0], x[1], sel_q), r = __byte_perm(x[2], x[3], sel_q);
                qa[j][2 * w] = __byte_perm(p, r, 0x7632);
                qa[j][2 * w + 1] = __byte_perm(p, r, 0x5410);
            }
    }
    const float sm0 = up ? 256.0f : 16777216.0f, sm1 = up ? 1.0f : 65536.0f;       // a score's digits
    const float vm0 = sm0 * 0x1p-31f, vm1 = sm1 * 0x1p-31f;                       // an output's
    // a pair of weights (own, other half's) as bytes (lower digit, lower, upper, upper) in the keys' order
    const uint32_t sel_w = up ? 0x1504u : 0x7362u;
    // lanes of odd t read the two keys of a pair in the other order at 64 dims (other banks)
    const bool odd = HD == 64 && (t & 1);
    const uint32_t sel_lo = odd ? 0x1504u : 0x5140u, sel_hi = odd ? 0x3726u : 0x7362u;
    float M = kLowest, l = 0.f, o[VD][2];
#pragma unroll
    for (int i = 0; i < VD; ++i) o[i][0] = o[i][1] = 0.f;
    const int b1 = src.b1;
    int stage = 0;
    for (int blk = src.first(warp); blk < b1; blk += src.kStep) {
        copy_wait<kStages - 2>();
        __syncwarp();                        // this batch is here for every lane, and all are done with the last
        src.fetch(sm, warp, lane, blk + (kStages - 1) * src.kStep, stage == 0 ? kStages - 1 : stage - 1);
        const uint8_t* kp = sm.ring[warp][stage][0];
        const uint8_t* vp = sm.ring[warp][stage][1];
        float ks[BB];
        uint32_t vs[BB];                     // the bits of 2^e m
        int ev[BB], left[BB];
#pragma unroll
        for (int b = 0; b < BB; ++b) {
            // the block's keys that count, from the lane's first on (of the 32 that are its own and its pair's)
            left[b] = src.keys - (blk + b) * kQBlock - 2 * t - up;
            ks[b] = sm.scale[warp][stage][0][b] * kmul;
            vs[b] = __float_as_uint(sm.scale[warp][stage][1][b]);
            ev[b] = max((int)(vs[b] >> 23) - 127, kLeastScale);
        }
        stage = stage == kStages - 1 ? 0 : stage + 1;
        // lane (g, t) ends with the score of head g % 4 and key 8 n + 2 t, + 1 for g >= 4
        float s[NT], most[BB];               // most: the lane's largest score of a block, rounded up
#pragma unroll
        for (int b = 0; b < BB; ++b) most[b] = -INFINITY;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            uint32_t acc[4] = {kMagicBits, kMagicBits, kMagicBits, kMagicBits};
#pragma unroll
            for (int c = 0; c < C; ++c) {
                const uint4 w = *reinterpret_cast<const uint4*>(kp + (8 * n + g) * HD + 16 * swizzled<HD>(8 * n + g, C * t + c));
                mma_s8(acc, qa[2 * c], w.x, w.y);
                mma_s8(acc, qa[2 * c + 1], w.z, w.w);
            }
            const float f0 = sum_of(acc[0], sm0) + sum_of(acc[2], sm1), f1 = sum_of(acc[1], sm0) + sum_of(acc[3], sm1);
            s[n] = (up ? f1 : f0) + __shfl_xor_sync(0xffffffffu, up ? f0 : f1, 16);
            const int b = n / (kQBlock / 8);
            // rounded here, like a sum of its products, and so the same number in the maximum and in the weight
            s[n] = 8 * (n % (kQBlock / 8)) < left[b] ? s[n] * ks[b] : -INFINITY;
            most[b] = fmaxf(most[b], s[n]);
        }
        float top = -INFINITY;
#pragma unroll
        for (int b = 0; b < BB; ++b) {
            most[b] = fmaxf(ceilf(most[b]), kLowest);
            top = fmaxf(top, most[b] + (float)ev[b]);
        }
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 16));
        const float Mn = fmaxf(M, top);
        const float f = pow2(M - Mn);
        l = scaled(l, M - Mn);
        M = Mn;
        uint32_t wp[NT];                     // the pair's digits
#pragma unroll
        for (int b = 0; b < BB; ++b) {
            // what the lane's exponentials, 2^(s - most), still lack: as a weight 2^31 m 2^(most + e - M), as a term
            // of the sum 2^(most - M + 39)
            const int k = __float_as_int(fmaxf(most[b] + (float)ev[b] - M, -400.0f) + kMagic) - (int)kMagicBits;
            const float vm = __uint_as_float((vs[b] & 0x7fffffu) | (uint32_t)max(k + 127 + 31, 0) << 23);
            const float unit = __uint_as_float((uint32_t)max(k - ev[b] + 127 + kSumBits, 0) << 23);
            float sum = 0.f;
#pragma unroll
            for (int n = b * (kQBlock / 8); n < (b + 1) * (kQBlock / 8); ++n) {
                const float w = ex2(s[n] - most[b]);
                sum += w;
                const uint32_t W = __float2uint_rn(w * vm);
                wp[n] = __byte_perm(W, __shfl_xor_sync(0xffffffffu, W, 16), sel_w);
            }
            // a NaN scale's bits are those of a NaN
            l = fmaf(sum, vs[b] > 0x7f800000u && (b == 0 || blk + b < b1) ? __uint_as_float(0x7fffffffu) : unit, l);
        }
        uint32_t pa[NT / 4][4];
#pragma unroll
        for (int k = 0; k < NT / 4; ++k)
#pragma unroll
            for (int w = 0; w < 2; ++w) {
                pa[k][2 * w] = __byte_perm(wp[4 * k + 2 * w], wp[4 * k + 2 * w + 1], 0x7632);
                pa[k][2 * w + 1] = __byte_perm(wp[4 * k + 2 * w], wp[4 * k + 2 * w + 1], 0x5410);
            }
#pragma unroll
        for (int j = 0; j < VD / 8; ++j) {
            // dims 8 j .. 8 j + 7 of the lane's, in two words of each key
            uint32_t acc[8][4];
#pragma unroll
            for (int i = 0; i < 8; ++i) acc[i][0] = acc[i][1] = acc[i][2] = acc[i][3] = kMagicBits;
#pragma unroll
            for (int k = 0; k < NT / 4; ++k) {
                uint32_t bw[2][8];           // [half of the K step][dim]: that dim of four keys
#pragma unroll
                for (int w = 0; w < 2; ++w) {
                    uint2 x[4];              // keys 8 n + 2 t, + 1 of tiles n = 4 k + 2 w, + 1
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int r = 8 * (4 * k + 2 * w + i / 2) + 2 * t + (HD == 64 ? (i & 1) ^ (t & 1) : i & 1);
                        const int c = HD == 64 ? g >> 1 : g;
                        x[i] = *reinterpret_cast<const uint2*>(vp + r * HD + 16 * swizzled<HD>(r, c) + (HD == 64 ? 8 * (g & 1) : 8 * j));
                    }
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const uint32_t x0 = h ? x[0].y : x[0].x, x1 = h ? x[1].y : x[1].x;
                        const uint32_t x2 = h ? x[2].y : x[2].x, x3 = h ? x[3].y : x[3].x;
                        const uint32_t p = __byte_perm(x0, x1, sel_lo), q = __byte_perm(x2, x3, sel_lo);
                        const uint32_t r = __byte_perm(x0, x1, sel_hi), u = __byte_perm(x2, x3, sel_hi);
                        bw[w][4 * h] = __byte_perm(p, q, 0x5410);
                        bw[w][4 * h + 1] = __byte_perm(p, q, 0x7632);
                        bw[w][4 * h + 2] = __byte_perm(r, u, 0x5410);
                        bw[w][4 * h + 3] = __byte_perm(r, u, 0x7632);
                    }
                }
#pragma unroll
                for (int i = 0; i < 8; ++i) mma_u8(acc[i], pa[k], bw[0][i], bw[1][i]);
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                o[8 * j + i][0] = fmaf(o[8 * j + i][0], f, sum_of(acc[i][0], vm0) + sum_of(acc[i][2], vm1));
                o[8 * j + i][1] = fmaf(o[8 * j + i][1], f, sum_of(acc[i][1], vm0) + sum_of(acc[i][3], vm1));
            }
        }
    }
    copy_wait<0>();
    __syncwarp();
    // the halves of the digits, and the lanes' shares of the sum (keys 2 t of tile n, or 2 t + 1)
    l += __shfl_xor_sync(0xffffffffu, l, 1);
    l += __shfl_xor_sync(0xffffffffu, l, 2);
    l += __shfl_xor_sync(0xffffffffu, l, 16);
    if (g < a.group && t == 0) {
        sm.m[warp][g] = M;
        sm.l[warp][g] = l;
    }
#pragma unroll
    for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int i = 0; i < VD; i += 4) {
            float4 x;
#pragma unroll
            for (int k = 0; k < 4; ++k) (&x.x)[k] = o[i + k][e] + __shfl_xor_sync(0xffffffffu, o[i + k][e], 16);
            if (g < a.group) *reinterpret_cast<float4*>(sm.warp_o(warp, g) + (2 * t + e) * sm.kEighth + i) = x;
        }
}

// The open block's n < 32 bf16 tokens, fp32 on the CUDA cores: warp h takes head h,
// lane i scores token i, then each lane sums HD / 32 dims. At 64 dims its loads go out with the first
// batches', ahead of the wait for the queries (129 keys 3.8 -> 3.5 us); at 128 that many more registers
// spill (53.7 -> 55.2 us at 4 x 60001 keys). Half the values' follow behind the scores.
template <int HD>
struct AttnTail {
    static constexpr int D = HD / 32, H = kQBlock / 2;
    uint4 kr[HD / 8];
    uint32_t vr[H][D / 2];
    const uint16_t* vt;
    __device__ __forceinline__ void load_values(int first, int n) {
#pragma unroll
        for (int i = 0; i < H; ++i)
#pragma unroll
            for (int d = 0; d < D / 2; ++d) vr[i][d] = *reinterpret_cast<const uint32_t*>(vt + min(first + i, n - 1) * HD + 2 * d);
    }
    __device__ __forceinline__ void load(const AttnArgs& a, size_t plane, int n, int lane) {
        const uint16_t* kt = a.tail[0] + plane * (kQBlock * HD) + (size_t)min(lane, n - 1) * HD;
        vt = a.tail[1] + plane * (kQBlock * HD) + lane * D;
#pragma unroll
        for (int e = 0; e < HD / 8; ++e) kr[e] = *reinterpret_cast<const uint4*>(kt + 8 * e);
        load_values(0, n);
    }
    __device__ __forceinline__ void attend(AttnSmem<HD>& sm, int n, int warp, int lane);
};

template <int HD>
__device__ __forceinline__ void AttnTail<HD>::attend(AttnSmem<HD>& sm, int n, int warp, int lane) {
    float s = 0.f;
#pragma unroll
    for (int e = 0; e < HD / 8; ++e)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t w = (&kr[e].x)[i];
            s = fmaf(__uint_as_float(w << 16), sm.query(warp, 8 * e + 2 * i), s);
            s = fmaf(__uint_as_float(w & 0xffff0000u), sm.query(warp, 8 * e + 2 * i + 1), s);
        }
    s = lane < n ? s * (kLog2e * (HD == 64 ? 0.125f : 0.08838834764831845f)) : -INFINITY;
    float m = s;
#pragma unroll
    for (int k = 16; k > 0; k >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, k));
    m = fmaxf(ceilf(m), kLowest);             // e = 0
    const float w = lane < n ? exp2f(s - m) : 0.f;
    float l = w;
#pragma unroll
    for (int k = 16; k > 0; k >>= 1) l += __shfl_xor_sync(0xffffffffu, l, k);
    float o[D];
#pragma unroll
    for (int d = 0; d < D; ++d) o[d] = 0.f;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
        if (half * H >= n) break;
        if (half == 1) load_values(H, n);
        // tokens behind the last (the last one's values) weigh nothing
#pragma unroll
        for (int i = 0; i < H; ++i) {
            const float wi = __shfl_sync(0xffffffffu, w, half * H + i);
#pragma unroll
            for (int d = 0; d < D / 2; ++d) {
                o[2 * d] = fmaf(wi, __uint_as_float(vr[i][d] << 16), o[2 * d]);
                o[2 * d + 1] = fmaf(wi, __uint_as_float(vr[i][d] & 0xffff0000u), o[2 * d + 1]);
            }
        }
    }
    if (lane == 0) {
        sm.m[kAttWarps][warp] = m;
        sm.l[kAttWarps][warp] = l * kSumUnit;
    }
#pragma unroll
    for (int d = 0; d < D; ++d) sm.tail_o[warp][lane * D + d] = o[d];
}

// Two or four consecutive floats. The loads stay in their order, ahead of the shuffles that follow.
__device__ __forceinline__ void load(const float* p, float (&x)[2]) {
    asm volatile("ld.global.v2.f32 {%0, %1}, [%2];" : "=f"(x[0]), "=f"(x[1]) : "l"(p));
}
__device__ __forceinline__ void load(const float* p, float (&x)[4]) {
    asm volatile("ld.global.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(x[0]), "=f"(x[1]), "=f"(x[2]), "=f"(x[3]) : "l"(p));
}
__device__ __forceinline__ void store(float* p, const float (&x)[2]) { *reinterpret_cast<float2*>(p) = make_float2(x[0], x[1]); }
__device__ __forceinline__ void store(float* p, const float (&x)[4]) { *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]); }

// The largest and the sum of eight lanes.
__device__ __forceinline__ float max_of_8(float x) {
#pragma unroll
    for (int k = 4; k > 0; k >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, k));
    return x;
}
__device__ __forceinline__ float sum_of_8(float x) {
#pragma unroll
    for (int k = 4; k > 0; k >>= 1) x += __shfl_xor_sync(0xffffffffu, x, k);
    return x;
}

// Joins the parts in sm whose mask bit is set. FINAL: the output row; else a partial. Warp h has head h, so
// that a thread forms each part's factor once.
template <int HD, bool FINAL>
__device__ __forceinline__ void attn_join(const AttnArgs& a, AttnSmem<HD>& sm, uint32_t parts, float* o, float* ml) {
    __syncthreads();
    static_assert(kMaxGroupHeads <= kAttWarps, "a warp for every head");
    constexpr int D = HD / 32;
    const int h = threadIdx.x >> 5, d = (threadIdx.x & 31) * D;
    if (h < a.group) {
        float m[kAttWarps + 1], x[kAttWarps + 1][D], ls[kAttWarps + 1], M = -INFINITY;
#pragma unroll
        for (int p = 0; p <= kAttWarps; ++p) {
            const bool there = parts >> p & 1;
            m[p] = there ? sm.m[p][h] : -INFINITY;
            ls[p] = there ? sm.l[p][h] : 0.f;
#pragma unroll
            for (int i = 0; i < D; ++i) x[p][i] = there ? sm.o(p, h, d + i) : 0.f;
            M = fmaxf(M, m[p]);
        }
        float l = 0.f, y[D];
#pragma unroll
        for (int i = 0; i < D; ++i) y[i] = 0.f;
#pragma unroll
        for (int p = 0; p <= kAttWarps; ++p) {
            const float w = pow2(m[p] - M);
            l += scaled(ls[p], m[p] - M);
#pragma unroll
            for (int i = 0; i < D; ++i) y[i] = fmaf(w, x[p][i], y[i]);
        }
        if (FINAL) {
            l *= 1.0f / kSumUnit;
#pragma unroll
            for (int i = 0; i < D; ++i) o[h * HD + d + i] = y[i] / l;
        } else {
            store(o + h * HD + d, y);
            if (d == 0) *reinterpret_cast<float2*>(ml + 2 * h) = make_float2(M, l);
        }
    }
    __syncthreads();
}

template <int HD>
__device__ __forceinline__ AttnSmem<HD>& attn_smem() {
    extern __shared__ __align__(16) uint8_t attn_raw[];
    return *reinterpret_cast<AttnSmem<HD>*>(attn_raw);
}

// The slots that row b attends to, and whether the last of them lie in its open block. A row's length says which of
// its blocks are closed: a cut inside a closed block is read from the codes.
struct RowKeys {
    int n;
    bool open;
    __device__ __forceinline__ RowKeys(const AttnArgs& a, int b) {
        // from L2, for the joining kernel reads them before it waits
        const int pos = __ldcg(a.positions + b), length = a.lengths ? min(__ldcg(a.lengths + b), a.max_seq) : min(pos, a.max_seq - 1) + 1;
        n = max(min(min(pos, a.max_ctx - 1) + 1, length), 0);
        open = n > length / kQBlock * kQBlock;
    }
    __device__ __forceinline__ RowKeys(int keys, bool in_open) : n(keys), open(in_open) {}
};

// The order in which the split deals out blocks: row by row, head by head, each (row, KV head) with its
// blocks (the open one included) behind kPad units without work, which stand for what starting and
// joining one more piece costs the CTA that has them. 4 / 8 / 12 / 16 / 24 units: 52.3 / 52.0 / 51.9 /
// 51.6 / 50.8 us at 4 x 60001 keys of 128 dims, 22.2 / 21.8 / 21.9 / 21.6 / 21.7 at 8 x 16384 of 64.
constexpr int kPad = 24;
__device__ __forceinline__ int attn_units(int keys) { return (keys + kQBlock - 1) / kQBlock; }
__device__ __forceinline__ int attn_share(int keys) { return keys ? attn_units(keys) + kPad : 0; }

// `units` over `n` CTAs, in order: the first `more` CTAs take each + 1 of them, the others `each`.
template <int HD>
struct SplitPlan {
    int keys[kMaxBatch];                 // of each row
    uint32_t open;                       // the rows whose open block is attended to
    int n, each, more;
    __device__ __forceinline__ explicit SplitPlan(const AttnArgs& a) {
        int units = 0;
        // lane b reads row b's
        const int lane = threadIdx.x & 31;
        const RowKeys own = lane < a.rows ? RowKeys(a, lane) : RowKeys(0, false);
#pragma unroll
        for (int b = 0; b < kMaxBatch; ++b) keys[b] = __shfl_sync(0xffffffffu, own.n, b);
        open = __ballot_sync(0xffffffffu, own.open);
#pragma unroll
        for (int b = 0; b < kMaxBatch; ++b) units += attn_share(keys[b]) * a.n_heads;
        constexpr int least = kAttWarps * batch_blocks(HD);   // a batch for each warp
        n = min(a.n_cta, (units + least - 1) / least);
        each = n ? units / n : 0;
        more = units - n * each;
    }
    __device__ __forceinline__ int start(int c) const { return c * each + min(c, more); }
    __device__ __forceinline__ int owner(int u) const {
        const int big = more * (each + 1);
        return u < big ? u / (each + 1) : more + (u - big) / each;
    }
    // The row of unit u, its keys and its first unit.
    __device__ __forceinline__ void row_of(int u, int n_heads, int& row, int& row_keys, int& first) const {
        int at = 0;
        row = row_keys = first = 0;
#pragma unroll
        for (int b = 0; b < kMaxBatch; ++b) {
            const int next = at + attn_share(keys[b]) * n_heads;
            if (u >= at && u < next) {
                row = b;
                row_keys = keys[b];
                first = at;
            }
            at = next;
        }
    }
};

// Blocks [u, stop) of one (row, KV head) that attends to `keys`, the open one included, into the
// parts of sm: which, as bits.
template <int HD>
__device__ __forceinline__ uint32_t attn_range(const AttnArgs& a, AttnSmem<HD>& sm, int b, int h, int u, int stop, RowKeys keys) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const size_t plane = ((size_t)a.layer * a.max_batch + b) * a.n_heads + h;
    const int nb = keys.open ? keys.n / kQBlock : attn_units(keys.n);
    const AttnSource<HD> src(a, plane, u, min(stop, nb), keys.n);
    // the queries' loads go out ahead of the many of the first batches
    constexpr int QE = kMaxGroupHeads * HD / (32 * kAttWarps);
    const float* q = a.q + ((size_t)b * a.n_heads + h) * a.group * HD;
    float qv[QE];
#pragma unroll
    for (int i = 0; i < QE; ++i) {
        const int e = i * 32 * kAttWarps + (int)threadIdx.x;
        qv[i] = e < a.group * HD ? q[e] : 0.f;
    }
    src.start(sm, warp, lane);
    // the open block, by the warps of the group's heads
    const int nt = stop > nb && warp < a.group ? keys.n - nb * kQBlock : 0;
    AttnTail<HD> tail;
    if (HD == 64 && nt) tail.load(a, plane, nt, lane);
#pragma unroll
    for (int i = 0; i < QE; ++i) {
        const int e = i * 32 * kAttWarps + (int)threadIdx.x;
        sm.query(e / HD, e % HD) = qv[i];
    }
    __syncthreads();
    uint32_t parts = 0;
    if (nt) {
        if (HD != 64) tail.load(a, plane, nt, lane);
        tail.attend(sm, nt, warp, lane);
    }
    if (stop > nb) parts = 1u << kAttWarps;
    if (src.b0 < src.b1) {
        attn_blocks<HD>(a, sm, src, warp, lane);
        parts |= (1u << kAttWarps) - 1;
    }
    return parts;
}

// One CTA per (row, KV head): all its blocks.
template <int HD>
__global__ void __launch_bounds__(32 * kAttWarps, attn_per_sm(HD)) k_attn_whole(const __grid_constant__ AttnArgs a) {
    AttnSmem<HD>& sm = attn_smem<HD>();
    const int h = blockIdx.x % a.n_heads, b = blockIdx.x / a.n_heads;
    cudaGridDependencySynchronize();     // everything enqueued before has run
    const RowKeys keys(a, b);
    float* out = a.out + ((size_t)b * a.n_heads + h) * a.group * HD;
    if (keys.n == 0) {
        for (int e = threadIdx.x; e < a.group * HD; e += 32 * kAttWarps) out[e] = 0.f;
        return;
    }
    const uint32_t parts = attn_range<HD>(a, sm, b, h, 0, attn_units(keys.n), keys);
    attn_join<HD, true>(a, sm, parts, out, nullptr);
}

// The split: CTA c takes its range of the order, which may cover several (row, KV head)
// pairs; each piece becomes partial slot c + pair (distinct: both only grow along the
// order).
template <int HD>
__global__ void __launch_bounds__(32 * kAttWarps, attn_per_sm(HD)) k_attn_split(const __grid_constant__ AttnArgs a) {
    AttnSmem<HD>& sm = attn_smem<HD>();
    cudaGridDependencySynchronize();     // everything enqueued before has run
    // once every CTA runs, the joining kernel may be placed where CTAs end; what it reads before it waits for
    // them (the positions) has been written by then
    cudaTriggerProgrammaticLaunchCompletion();
    const SplitPlan<HD> P(a);
    const int c = blockIdx.x;
    if (c >= P.n) return;
    const int u1 = P.start(c + 1);
    for (int u = P.start(c); u < u1;) {
        int b, keys, first;
        P.row_of(u, a.n_heads, b, keys, first);
        const int share = attn_share(keys), h = (u - first) / share, base = first + h * share;
        const int end = min(u1, base + share);
        // without the padding; a piece of nothing but padding is no piece
        const int from = max(u - base - kPad, 0), stop = end - base - kPad;
        if (stop > from) {
            const uint32_t parts = attn_range<HD>(a, sm, b, h, from, stop, RowKeys(keys, P.open >> b & 1));
            const size_t slot = (size_t)c + b * a.n_heads + h;
            attn_join<HD, false>(a, sm, parts, a.part_o + slot * a.group * HD, a.part_ml + slot * a.group * 2);
        }
        u = end;
    }
}

// Joins the partials of one (row, query head): warps take kJoinEach slots in turn, lanes the dims. (8, 8)
// against (8, 4) warps and slots: 15.8 and 17.2 us for one row of 65536 keys and 8 heads of 64 dims, 8.7 and 10.7
// with one head; 16 warps are no faster there and 1 us slower at 8 x 8 pairs.
constexpr int kJoinWarps = 8, kJoinEach = 8;
template <int HD>
__global__ void __launch_bounds__(32 * kJoinWarps) k_attn_merge_q(const __grid_constant__ AttnArgs a) {
    constexpr int D = HD / 32;
    __shared__ float so[kJoinWarps][HD], sm[kJoinWarps], sl[kJoinWarps];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int heads = a.n_heads * a.group, b = blockIdx.x / heads, hq = blockIdx.x % heads;
    const int h = hq / a.group, hg = hq % a.group, pair = b * a.n_heads + h;
    const SplitPlan<HD> P(a);
    int first = 0, keys = 0;
#pragma unroll
    for (int i = 0; i < kMaxBatch; ++i) {
        if (i < b) first += attn_share(P.keys[i]) * a.n_heads;
        if (i == b) keys = P.keys[i];
    }
    const int share = attn_share(keys);
    first += h * share;
    const int c0 = share ? P.owner(first + kPad) : 0, total = share ? P.owner(first + share - 1) - c0 + 1 : 0;
    cudaGridDependencySynchronize();
    // kJoinEach partials of a warp at once, every load issued before the first is used. At 128 dims lane k of every
    // eight forms the factor of the k-th partial and shuffles pass it (one row of 1024 keys and 8 heads: 5.6 us, 6.0 where
    // every lane forms all eight), at 64 dims every lane forms them (2 rows of 16384 keys: 9.1 us, 9.8 with shuffles).
    float M = -INFINITY, l = 0.f, o[D];
#pragma unroll
    for (int d = 0; d < D; ++d) o[d] = 0.f;
    const size_t slot = (size_t)c0 + pair;
    for (int i = warp * kJoinEach; i < total; i += kJoinWarps * kJoinEach) {
        float p[kJoinEach][D];
        auto at = [&](int k) { return (slot + min(i + k, total - 1)) * a.group + hg; };
        if constexpr (D == 4) {
            static_assert(kJoinEach == 8, "a lane for each");
            float ml[2];
            load(a.part_ml + at(lane & 7) * 2, ml);
#pragma unroll
            for (int k = 0; k < kJoinEach; ++k) load(a.part_o + at(k) * HD + lane * D, p[k]);
            const bool there = i + (lane & 7) < total;
            const float Mn = fmaxf(M, max_of_8(ml[0])), f = pow2(M - Mn), own = there ? pow2(ml[0] - Mn) : 0.f;
            l = scaled(l, M - Mn) + sum_of_8(there ? scaled(ml[1], ml[0] - Mn) : 0.f);
            M = Mn;
#pragma unroll
            for (int d = 0; d < D; ++d) o[d] *= f;
#pragma unroll
            for (int k = 0; k < kJoinEach; ++k) {
                const float w = __shfl_sync(0xffffffffu, own, k);
#pragma unroll
                for (int d = 0; d < D; ++d) o[d] = fmaf(p[k][d], w, o[d]);
            }
        } else {
            float2 ml[kJoinEach];
#pragma unroll
            for (int k = 0; k < kJoinEach; ++k) {
                ml[k] = *reinterpret_cast<const float2*>(a.part_ml + at(k) * 2);
                const float2 x = *reinterpret_cast<const float2*>(a.part_o + at(k) * HD + lane * D);
                p[k][0] = x.x;
                p[k][1] = x.y;
                if (i + k >= total) ml[k] = make_float2(-INFINITY, 0.f);   // a partial's maximum is a number
            }
            float Mn = M;
#pragma unroll
            for (int k = 0; k < kJoinEach; ++k) Mn = fmaxf(Mn, ml[k].x);
            const float f = pow2(M - Mn);
            l = scaled(l, M - Mn);
            M = Mn;
#pragma unroll
            for (int d = 0; d < D; ++d) o[d] *= f;
#pragma unroll
            for (int k = 0; k < kJoinEach; ++k) {
                const float w = pow2(ml[k].x - M);
                l += scaled(ml[k].y, ml[k].x - M);
#pragma unroll
                for (int d = 0; d < D; ++d) o[d] = fmaf(p[k][d], w, o[d]);
            }
        }
    }
#pragma unroll
    for (int d = 0; d < D; ++d) so[warp][lane * D + d] = o[d];
    if (lane == 0) {
        sm[warp] = M;
        sl[warp] = l;
    }
    __syncthreads();
    const int e = threadIdx.x;
    if (e >= HD) return;
    float* out = a.out + ((size_t)b * heads + hq) * HD;
    if (total == 0) {
        out[e] = 0.f;
        return;
    }
    const int used = min((total + kJoinEach - 1) / kJoinEach, kJoinWarps);
    float top = -INFINITY, L = 0.f, x = 0.f;
    for (int i = 0; i < used; ++i) top = fmaxf(top, sm[i]);
    for (int i = 0; i < used; ++i) {
        L += scaled(sl[i], sm[i] - top);
        x = fmaf(pow2(sm[i] - top), so[i][e], x);
    }
    out[e] = x / (L * (1.0f / kSumUnit));
}

// ------------------------------------------------------------------ launches

// One CTA per (row, KV head) up to these contexts, in one kernel; beyond, the split and its joining kernel.
// With 8 pairs the two take 4.7 and 4.6 us at 1024 keys of 64 dims, 7.4 and 4.8 at 2048; 5.3 and 5.4 at 512 keys of
// 128, 8.1 and 5.4 at 1024. With 64 pairs 7.4 and 8.0 us at 2048 keys of 64 dims, 12.8 and 9.8 at 4096;
// 8.2 and 9.1 at 1024 of 128, 13.7 and 10.8 at 2048.
bool attn_is_split(int hd, int pairs, int max_ctx) { return max_ctx > (pairs >= 32 ? 131072 : 65536) / hd; }
// Floats of the partials' maxima and sums; the outputs behind them are read 16 bytes at a time.
size_t attn_ml_floats(size_t slots) { return (2 * slots + 3) / 4 * 4; }
int attn_ctas(int hd) { return kQSms * attn_per_sm(hd); }
size_t attn_slots(int hd, int rows, int n_heads) { return (size_t)attn_ctas(hd) + (size_t)rows * n_heads; }

template <int HD>
cudaError_t attn_launch(const AttnArgs& a, cudaStream_t st) {
    const int smem = (int)sizeof(AttnSmem<HD>);
    const bool whole = a.n_cta == 0;
    static std::atomic<uint64_t> seen{0};
    cudaError_t e = cudaSuccess;
    if (first_on_device(seen)) {
        e = cudaFuncSetAttribute(k_attn_whole<HD>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e == cudaSuccess) e = cudaFuncSetAttribute(k_attn_split<HD>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) return e;
        seen_on_device(seen);
    }
    if (whole) return launch_behind(k_attn_whole<HD>, a.rows * a.n_heads, 32 * kAttWarps, smem, st, a);
    e = launch_behind(k_attn_split<HD>, a.n_cta, 32 * kAttWarps, smem, st, a);
    if (e != cudaSuccess) return e;
    return launch_behind(k_attn_merge_q<HD>, a.rows * a.n_heads * a.group, 32 * kJoinWarps, 0, st, a);
}

}  // namespace
}  // namespace mk

extern "C" mk_status mk_qcache_append(const mk_qcache* c, int first_layer, int n_layers, int rows, int n_new,
                                      const void* k_new, const void* v_new, const int64_t* strides,
                                      const int32_t* positions, const int32_t* counts, void* stream) {
    if (!k_new || !v_new || !strides || !positions) return MK_ERR_INVALID_ARG;
    if (const mk_status st = mk::qcache_check(c); st != MK_OK) return st;
    if (first_layer < 0 || n_layers < 1 || first_layer > c->n_layers - n_layers || rows < 1 || rows > c->max_batch ||
        n_new < 1 || n_new > c->max_seq)
        return MK_ERR_INVALID_ARG;
    if ((reinterpret_cast<uintptr_t>(k_new) | reinterpret_cast<uintptr_t>(v_new)) & 15) return MK_ERR_INVALID_ARG;
    for (int i = 0; i < 4; ++i)
        if (strides[i] & 7) return MK_ERR_INVALID_ARG;
    mk::AppendArgs a{};
    a.codes[0] = static_cast<uint8_t*>(c->k_codes);
    a.codes[1] = static_cast<uint8_t*>(c->v_codes);
    a.scale[0] = c->k_scale;
    a.scale[1] = c->v_scale;
    a.tail[0] = static_cast<uint16_t*>(c->k_tail);
    a.tail[1] = static_cast<uint16_t*>(c->v_tail);
    a.src[0] = static_cast<const uint16_t*>(k_new);
    a.src[1] = static_cast<const uint16_t*>(v_new);
    a.sl = strides[0];
    a.sr = strides[1];
    a.sh = strides[2];
    a.st = strides[3];
    a.first_layer = first_layer;
    a.n_layers = n_layers;
    a.max_batch = c->max_batch;
    a.n_heads = c->n_kv_heads;
    a.max_seq = c->max_seq;
    a.n_blocks = mk::qcache_blocks(c->max_seq);
    a.rows = rows;
    a.n_new = n_new;
    a.positions = positions;
    a.counts = counts;
    const int window = (mk::kQBlock - 1 + n_new) / mk::kQBlock;   // full blocks of a window at most
    const int per = mk::kAppWarps / (c->head_dim / 64);           // of them, a CTA's
    const dim3 grid((unsigned)(((window < 1 ? 1 : window) + per - 1) / per), (unsigned)(rows * c->n_kv_heads),
                    (unsigned)(2 * n_layers));
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const cudaError_t e = c->head_dim == 64 ? mk::launch_behind(mk::k_append<64>, grid, 32 * mk::kAppWarps, 0, st, a)
                                            : mk::launch_behind(mk::k_append<128>, grid, 32 * mk::kAppWarps, 0, st, a);
    return e == cudaSuccess ? MK_OK : MK_ERR_CUDA;
}

extern "C" size_t mk_qcache_attention_workspace(const mk_qcache* c, int rows, int n_heads, int max_ctx) {
    if (mk::qcache_check(c) != MK_OK || rows < 1 || rows > c->max_batch || n_heads < c->n_kv_heads ||
        n_heads % c->n_kv_heads != 0 || n_heads / c->n_kv_heads > mk::kMaxGroupHeads || max_ctx < 1 ||
        max_ctx > c->max_seq || !mk::attn_is_split(c->head_dim, rows * c->n_kv_heads, max_ctx))
        return 0;
    const size_t slots = mk::attn_slots(c->head_dim, rows, c->n_kv_heads) * (size_t)(n_heads / c->n_kv_heads);
    return (mk::attn_ml_floats(slots) + slots * (size_t)c->head_dim) * sizeof(float);
}

namespace mk {
// lengths: NULL for rows that hold positions[r] + 1 tokens.
static mk_status attention(const mk_qcache* c, int layer, int rows, int n_heads, int max_ctx, const float* q,
                           const int32_t* positions, const int32_t* lengths, float* out, void* workspace,
                           size_t workspace_bytes, void* stream) {
    if (!q || !positions || !out) return MK_ERR_INVALID_ARG;
    if (const mk_status st = mk::qcache_check(c); st != MK_OK) return st;
    if (n_heads < c->n_kv_heads || n_heads % c->n_kv_heads != 0 || n_heads / c->n_kv_heads > mk::kMaxGroupHeads)
        return MK_ERR_UNSUPPORTED;
    if (layer < 0 || layer >= c->n_layers || rows < 1 || rows > c->max_batch || max_ctx < 1 || max_ctx > c->max_seq)
        return MK_ERR_INVALID_ARG;
    const size_t need = mk_qcache_attention_workspace(c, rows, n_heads, max_ctx);
    if (need && (!workspace || workspace_bytes < need || (reinterpret_cast<uintptr_t>(workspace) & 15)))
        return MK_ERR_INVALID_ARG;
    mk::AttnArgs a{};
    a.codes[0] = static_cast<const uint8_t*>(c->k_codes);
    a.codes[1] = static_cast<const uint8_t*>(c->v_codes);
    a.scale[0] = c->k_scale;
    a.scale[1] = c->v_scale;
    a.tail[0] = static_cast<const uint16_t*>(c->k_tail);
    a.tail[1] = static_cast<const uint16_t*>(c->v_tail);
    a.layer = layer;
    a.max_batch = c->max_batch;
    a.n_heads = c->n_kv_heads;
    a.group = n_heads / c->n_kv_heads;
    a.max_seq = c->max_seq;
    a.n_blocks = mk::qcache_blocks(c->max_seq);
    a.rows = rows;
    a.max_ctx = max_ctx;
    a.q = q;
    a.positions = positions;
    a.lengths = lengths;
    a.out = out;
    if (need) {
        a.n_cta = mk::attn_ctas(c->head_dim);
        a.part_ml = static_cast<float*>(workspace);
        a.part_o = a.part_ml + mk::attn_ml_floats(mk::attn_slots(c->head_dim, rows, c->n_kv_heads) * (size_t)a.group);
    }
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const cudaError_t e = c->head_dim == 64 ? mk::attn_launch<64>(a, st) : mk::attn_launch<128>(a, st);
    return e == cudaSuccess ? MK_OK : MK_ERR_CUDA;
}
}  // namespace mk

extern "C" mk_status mk_qcache_attention(const mk_qcache* c, int layer, int rows, int n_heads, int max_ctx,
                                         const float* q, const int32_t* positions, float* out, void* workspace,
                                         size_t workspace_bytes, void* stream) {
    return mk::attention(c, layer, rows, n_heads, max_ctx, q, positions, nullptr, out, workspace, workspace_bytes, stream);
}

extern "C" mk_status mk_qcache_attention_prefix(const mk_qcache* c, int layer, int rows, int n_heads, int max_ctx,
                                                const float* q, const int32_t* positions, const int32_t* lengths,
                                                float* out, void* workspace, size_t workspace_bytes, void* stream) {
    if (!lengths) return MK_ERR_INVALID_ARG;
    return mk::attention(c, layer, rows, n_heads, max_ctx, q, positions, lengths, out, workspace, workspace_bytes, stream);
}
