// The 8-bit KV cache: storing new keys and values, and decode attention over it.
//
// A block is kQBlock = 32 tokens of one (layer, row, head), of keys or of values:
//   scale = amax / 127 (amax the block's largest magnitude), code = rint(x * (127 / amax)), int8.
// The tokens of a row's open block (the last length % 32 of them) stay bf16 in the
// tail buffers until the block is full, so a code is rounded once, from the token's
// own bf16 value, and never again.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math.h>

#include "qcache.h"

namespace mk {
namespace {

// ------------------------------------------------------------------ append

constexpr int kAppWarps = 8;

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

__device__ __forceinline__ float bf(uint32_t bits16) { return __uint_as_float(bits16 << 16); }

// One warp per (keys or values, layer, row, head, block of the row's window). The
// window starts at the row's open block: `held` tokens already in the tail, then the
// new ones. Lane i of iteration j holds 16 consecutive elements of one token, so a
// block of codes is written in full 16-byte pieces. The block that stays open is
// written by the warp of window block 0, after it has read the tail's old tokens.
template <int HD>
__global__ void __launch_bounds__(32 * kAppWarps) k_append(const __grid_constant__ AppendArgs a) {
    constexpr int IT = kQBlock * HD / 512;   // 16-element pieces per lane
    constexpr int PPT = HD / 16;             // pieces per token
    const int lane = threadIdx.x & 31;
    const int wb = blockIdx.x * kAppWarps + (threadIdx.x >> 5);   // window block
    const int h = blockIdx.y % a.n_heads, r = blockIdx.y / a.n_heads;
    const int which = blockIdx.z & 1, l = blockIdx.z >> 1;
    const int pos = a.positions[r];
    const int cnt = a.counts ? a.counts[r] : a.n_new;
    if (pos < 0 || cnt < 1 || cnt > a.n_new || pos > a.max_seq - cnt) return;
    const int held = pos % kQBlock, end = held + cnt;
    const int closed = end / kQBlock;        // window blocks that are full now
    if (wb >= max(closed, 1)) return;
    const size_t plane = ((size_t)(a.first_layer + l) * a.max_batch + r) * a.n_heads + h;
    uint16_t* tail = a.tail[which] + plane * (kQBlock * HD);
    const uint16_t* src = a.src[which] + l * a.sl + r * a.sr + h * a.sh;
    if (wb < closed) {
        uint4 x[IT][2];
        float big = 0.f;
        bool bad = false;
#pragma unroll
        for (int j = 0; j < IT; ++j) {
            const int piece = j * 32 + lane, tok = wb * kQBlock + piece / PPT, e = (piece % PPT) * 16;
            const uint16_t* p = tok < held ? tail + tok * HD + e : src + (size_t)(tok - held) * a.st + e;
            x[j][0] = *reinterpret_cast<const uint4*>(p);
            x[j][1] = *reinterpret_cast<const uint4*>(p + 8);
        }
#pragma unroll
        for (int j = 0; j < IT; ++j)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const uint32_t w = (&x[j][i / 4].x)[i % 4];
                const float u = fabsf(bf(w & 0xffffu)), v = fabsf(__uint_as_float(w & 0xffff0000u));
                big = fmaxf(big, fmaxf(u, v));
                bad |= !(u <= 3.4e38f) | !(v <= 3.4e38f);
            }
#pragma unroll
        for (int m = 16; m > 0; m >>= 1) big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, m));
        // a block with an infinity or a NaN gets a NaN scale: what attends to it is NaN
        bad = __any_sync(0xffffffffu, bad);
        const bool some = big >= kQNoBlock && !bad;
        const float inv = some ? __fdiv_rn(127.0f, big) : 0.f;
        const int blk = pos / kQBlock + wb;
        uint8_t* codes = a.codes[which] + (plane * a.max_seq + (size_t)blk * kQBlock) * HD;
#pragma unroll
        for (int j = 0; j < IT; ++j) {
            uint4 out;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                uint32_t word = 0;
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int k = q * 2 + i;
                    const uint32_t w = (&x[j][k / 4].x)[k % 4];
                    // |x| <= amax, so |x * inv| <= 127 (1 + 2^-23) and rounds to at most 127
                    const int c0 = __float2int_rn(__fmul_rn(bf(w & 0xffffu), inv));
                    const int c1 = __float2int_rn(__fmul_rn(__uint_as_float(w & 0xffff0000u), inv));
                    word |= ((uint32_t)(c0 & 0xff) | (uint32_t)(c1 & 0xff) << 8) << (16 * i);
                }
                (&out.x)[q] = word;
            }
            *reinterpret_cast<uint4*>(codes + (j * 32 + lane) * 16) = out;
        }
        if (lane == 0)
            a.scale[which][plane * a.n_blocks + blk] = bad ? __int_as_float(0x7fffffff) : some ? __fdiv_rn(big, 127.0f) : 0.f;
    }
    if (wb == 0) {
        __syncwarp();
        // the open block's new tokens
        const int t0 = closed > 0 ? 0 : held, n = end - closed * kQBlock;
        for (int piece = t0 * PPT + lane; piece < n * PPT; piece += 32) {
            const int tok = piece / PPT, e = (piece % PPT) * 16;
            const uint16_t* p = src + (size_t)(closed * kQBlock + tok - held) * a.st + e;
            const uint4 u = *reinterpret_cast<const uint4*>(p), v = *reinterpret_cast<const uint4*>(p + 8);
            *reinterpret_cast<uint4*>(tail + tok * HD + e) = u;
            *reinterpret_cast<uint4*>(tail + tok * HD + e + 8) = v;
        }
    }
}

// ------------------------------------------------------------------ attention
//
// out[h] = sum_i softmax_i(q[h] . k_i / sqrt(d)) v_i over slots i = 0 .. pos, for the
// group's query heads h of one (row, KV head). Codes are whole numbers of at most 127
// and so exact in fp16; the products run on the tensor cores (mma.sync m16n8k16,
// fp32 accumulation) with the other operand split into two fp16 parts, 22 bits in
// all: rows 0-7 of A hold the heads' high parts, rows 8-15 the low parts, and the two
// rows of the accumulator are added.
//   scores:  S[head][key]  = (sum_d q[head][d] code[key][d]) * k_scale
//   outputs: O[head][d]   += sum_key w[head][key] code[key][d]
// The value scale goes into the exponent: w = 2^(s + log2 v_scale - M), with M the
// running maximum of that sum, and l += w / v_scale, so that O / l is the softmax's
// output. The accumulator layout of S is the A layout of w, so the weights stay in
// their lane.

constexpr int kAttWarps = 4;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kWeightBits = 15.0f;   // weights are scaled by 2^15: at most 32768, fp16's normal range down to 2^-29

struct AttnArgs {
    const uint8_t* codes[2];
    const float* scale[2];
    const uint16_t* tail[2];
    int layer, max_batch, n_heads, group, max_seq, n_blocks, rows, max_ctx;
    const float* q;               // [rows][n_heads * group][HD]
    const int32_t* positions;
    float* out;
    float* part_ml;               // [slots][group][2]
    float* part_o;                // [slots][group][HD]
    int n_cta;                    // CTAs of the split over blocks (0: one CTA per (row, head), no partials)
};

__device__ __forceinline__ uint4 ld_code16(const uint8_t* p) {
    uint4 r;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "l"(p));
    return r;
}
__device__ __forceinline__ uint2 ld_code8(const uint8_t* p) {
    uint2 r;
    asm volatile("ld.global.nc.v2.u32 {%0,%1}, [%2];" : "=r"(r.x), "=r"(r.y) : "l"(p));
    return r;
}

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Bytes 0 and 2 of w (int8) as a pair of fp16: 0x6400 | (code + 128) is 1024 + code + 128.
__device__ __forceinline__ uint32_t codes_even(uint32_t w) {
    uint32_t r;
    asm("lop3.b32 %0, %1, 0x00ff00ff, 0x64806480, 0x6a;" : "=r"(r) : "r"(w));
    const __half2 h = __hsub2(*reinterpret_cast<__half2*>(&r), __half2(__ushort_as_half(0x6480), __ushort_as_half(0x6480)));
    return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t codes_odd(uint32_t w) { return codes_even(w >> 8); }

__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// x, y as fp16 pairs: the high parts and what they leave.
__device__ __forceinline__ void split2(float x, float y, uint32_t& hi, uint32_t& lo) {
    const __half2 h = __floats2half2_rn(x, y);
    const float2 f = __half22float2(h);
    const __half2 r = __floats2half2_rn(x - f.x, y - f.y);
    hi = *reinterpret_cast<const uint32_t*>(&h);
    lo = *reinterpret_cast<const uint32_t*>(&r);
}

// A CTA's running result of one (row, KV head): per warp (and the tail) a maximum, a
// sum and an output per head, joined at the end.
template <int HD>
struct AttnSmem {
    float o[kAttWarps + 1][kMaxGroupHeads][HD];
    float m[kAttWarps + 1][kMaxGroupHeads];
    float l[kAttWarps + 1][kMaxGroupHeads];
    float q[kMaxGroupHeads][HD];
};

// Blocks [b0, b1) of one (row, KV head) by the CTA's warps, into sm.o/m/l[warp].
template <int HD>
__device__ __forceinline__ void attn_blocks(const AttnArgs& a, AttnSmem<HD>& sm, size_t plane, int b0, int b1, int warp,
                                            int lane) {
    constexpr int KS = 2048 / HD;            // keys of a step: 2 KB of keys, 2 KB of values
    constexpr int NT = KS / 8;               // 8-key tiles
    constexpr int C = HD / 64;               // 16-byte pieces of a key per lane
    constexpr int VD = HD / 8;               // dims of a value per lane
    const int g = lane >> 2, t = lane & 3;
    // A fragments of q: head g's dims 64 c + 16 t + 4 i + {0, 2, 1, 3} in k-step 4 c + i. Each head
    // is scaled by a power of two to magnitudes below 512, so both parts stay normal.
    uint32_t qa[4 * C][4];
    float kmul;
    {
        float v[C][16], big = 0.f;
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                v[c][e] = g < a.group ? sm.q[g < kMaxGroupHeads ? g : 0][64 * c + 16 * t + e] : 0.f;
                big = fmaxf(big, fabsf(v[c][e]));
            }
        big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 1));
        big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 2));
        int ex = big > 0.f ? ilogbf(big) : 0;
        ex = ex > 120 ? 120 : ex < -110 ? -110 : ex;
        const float up = exp2f((float)(8 - ex));
        kmul = exp2f((float)(ex - 8)) * kLog2e * rsqrtf((float)HD);
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float* w = &v[c][4 * i];
                split2(w[0] * up, w[2] * up, qa[4 * c + i][0], qa[4 * c + i][1]);
                split2(w[1] * up, w[3] * up, qa[4 * c + i][2], qa[4 * c + i][3]);
            }
    }
    float M = -1e30f, l = 0.f, o[VD][4];
    float lv_ref = 0.f;
#pragma unroll
    for (int i = 0; i < VD; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
    const uint8_t* kc = a.codes[0] + plane * a.max_seq * HD;
    const uint8_t* vc = a.codes[1] + plane * a.max_seq * HD;
    const float* ksc = a.scale[0] + plane * a.n_blocks;
    const float* vsc = a.scale[1] + plane * a.n_blocks;
    constexpr int SPB = kQBlock / KS;        // steps per block
    const int s1 = b1 * SPB;
    for (int s = b0 * SPB + warp; s < s1; s += kAttWarps) {
        const uint8_t* kp = kc + (size_t)s * 2048 + g * HD + 16 * t;
        const uint8_t* vp = vc + (size_t)s * 2048 + (2 * t) * HD + g * VD;
        uint4 kr[NT][C];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int c = 0; c < C; ++c) kr[n][c] = ld_code16(kp + n * 8 * HD + 64 * c);
        uint32_t vr[NT][2][VD / 4];          // keys 8 n + 2 t, + 1
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const uint8_t* p = vp + (n * 8 + e) * HD;
                if constexpr (VD == 8) {
                    const uint2 u = ld_code8(p);
                    vr[n][e][0] = u.x; vr[n][e][1] = u.y;
                } else {
                    const uint4 u = ld_code16(p);
                    vr[n][e][0] = u.x; vr[n][e][1] = u.y; vr[n][e][2] = u.z; vr[n][e][3] = u.w;
                }
            }
        const float ks = __ldg(ksc + s / SPB) * kmul;
        const float vs = __ldg(vsc + s / SPB);
        // a block of zeros (scale 0): any reference serves, its codes add nothing to O
        const float lv = vs == 0.f ? lv_ref : log2f(vs);
        lv_ref = lv;
        const float ivs = vs == 0.f ? exp2f(-lv) : __fdividef(1.0f, vs);
        float w[NT][2], top = -INFINITY;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            float acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int c = 0; c < C; ++c)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint32_t word = (&kr[n][c].x)[i];
                    mma16816(acc, qa[4 * c + i], codes_even(word), codes_odd(word));
                }
            w[n][0] = fmaf(acc[0] + acc[2], ks, lv);
            w[n][1] = fmaf(acc[1] + acc[3], ks, lv);
            top = fmaxf(top, fmaxf(w[n][0], w[n][1]));
        }
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
        if (__any_sync(0xffffffffu, top > M)) {
            const float Mn = fmaxf(M, top), f = ex2(M - Mn);
            M = Mn;
            l *= f;
#pragma unroll
            for (int i = 0; i < VD; ++i)
#pragma unroll
                for (int k = 0; k < 4; ++k) o[i][k] *= f;
        }
        const float off = kWeightBits - M;
        uint32_t pa[NT / 2][4];
        float sum = 0.f;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const float w0 = ex2(w[n][0] + off), w1 = ex2(w[n][1] + off);
            sum += w0 + w1;
            split2(w0, w1, pa[n / 2][(n & 1) * 2], pa[n / 2][(n & 1) * 2 + 1]);
        }
        l = fmaf(sum, ivs, l);
#pragma unroll
        for (int k = 0; k < NT / 2; ++k)
#pragma unroll
            for (int j = 0; j < VD / 4; ++j) {
                // dims 4 j .. 4 j + 3 of the lane's: keys (2 t, 2 t + 1) and (2 t + 8, 2 t + 9) as pairs
                const uint32_t x0 = vr[2 * k][0][j], y0 = vr[2 * k][1][j], x1 = vr[2 * k + 1][0][j], y1 = vr[2 * k + 1][1][j];
                const uint32_t p0 = __byte_perm(x0, y0, 0x5410), r0 = __byte_perm(x0, y0, 0x7632);
                const uint32_t p1 = __byte_perm(x1, y1, 0x5410), r1 = __byte_perm(x1, y1, 0x7632);
                mma16816(o[4 * j], pa[k], codes_even(p0), codes_even(p1));
                mma16816(o[4 * j + 1], pa[k], codes_odd(p0), codes_odd(p1));
                mma16816(o[4 * j + 2], pa[k], codes_even(r0), codes_even(r1));
                mma16816(o[4 * j + 3], pa[k], codes_odd(r0), codes_odd(r1));
            }
    }
    l += __shfl_xor_sync(0xffffffffu, l, 1);
    l += __shfl_xor_sync(0xffffffffu, l, 2);
    if (g < a.group && g < kMaxGroupHeads) {
        if (t == 0) {
            sm.m[warp][g] = M;
            sm.l[warp][g] = l;
        }
#pragma unroll
        for (int i = 0; i < VD; ++i) {
            sm.o[warp][g][(2 * t) * VD + i] = o[i][0] + o[i][2];
            sm.o[warp][g][(2 * t + 1) * VD + i] = o[i][1] + o[i][3];
        }
    }
}

// The open block's n < 32 bf16 tokens, fp32 on the CUDA cores: warp h takes head h,
// lane i scores token i, then each lane sums HD / 32 dims.
template <int HD>
__device__ __forceinline__ void attn_tail(const AttnArgs& a, AttnSmem<HD>& sm, size_t plane, int n, int warp, int lane) {
    if (warp >= a.group) return;
    const uint16_t* kt = a.tail[0] + plane * (kQBlock * HD) + (size_t)min(lane, n - 1) * HD;
    const uint16_t* vt = a.tail[1] + plane * (kQBlock * HD);
    float s = 0.f;
#pragma unroll
    for (int e = 0; e < HD; e += 8) {
        const uint4 u = *reinterpret_cast<const uint4*>(kt + e);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t w = (&u.x)[i];
            s = fmaf(__uint_as_float(w << 16), sm.q[warp][e + 2 * i], s);
            s = fmaf(__uint_as_float(w & 0xffff0000u), sm.q[warp][e + 2 * i + 1], s);
        }
    }
    s = lane < n ? s * (kLog2e * rsqrtf((float)HD)) : -INFINITY;
    float m = s;
#pragma unroll
    for (int k = 16; k > 0; k >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, k));
    m = fmaxf(m, -1e30f);
    const float w = lane < n ? exp2f(s - m + kWeightBits) : 0.f;
    float l = w;
#pragma unroll
    for (int k = 16; k > 0; k >>= 1) l += __shfl_xor_sync(0xffffffffu, l, k);
    constexpr int D = HD / 32;
    float o[D];
#pragma unroll
    for (int d = 0; d < D; ++d) o[d] = 0.f;
    for (int i = 0; i < n; ++i) {
        const float wi = __shfl_sync(0xffffffffu, w, i);
#pragma unroll
        for (int d = 0; d < D; d += 2) {
            const uint32_t u = *reinterpret_cast<const uint32_t*>(vt + i * HD + lane * D + d);
            o[d] = fmaf(wi, __uint_as_float(u << 16), o[d]);
            o[d + 1] = fmaf(wi, __uint_as_float(u & 0xffff0000u), o[d + 1]);
        }
    }
    if (lane == 0) {
        sm.m[kAttWarps][warp] = m;
        sm.l[kAttWarps][warp] = l;
    }
#pragma unroll
    for (int d = 0; d < D; ++d) sm.o[kAttWarps][warp][lane * D + d] = o[d];
}

// Joins the parts in sm whose mask bit is set. FINAL: the output row; else a partial.
template <int HD, bool FINAL>
__device__ __forceinline__ void attn_join(const AttnArgs& a, AttnSmem<HD>& sm, uint32_t parts, float* o, float* ml) {
    __syncthreads();
    for (int e = threadIdx.x; e < a.group * HD; e += 32 * kAttWarps) {
        const int h = e / HD, d = e % HD;
        float M = -INFINITY;
#pragma unroll
        for (int p = 0; p <= kAttWarps; ++p)
            if (parts >> p & 1) M = fmaxf(M, sm.m[p][h]);
        float l = 0.f, x = 0.f;
#pragma unroll
        for (int p = 0; p <= kAttWarps; ++p)
            if (parts >> p & 1) {
                const float f = exp2f(sm.m[p][h] - M);
                l = fmaf(f, sm.l[p][h], l);
                x = fmaf(f, sm.o[p][h][d], x);
            }
        if (FINAL) {
            o[e] = x / l;
        } else {
            o[e] = x;
            if (d == 0) {
                ml[2 * h] = M;
                ml[2 * h + 1] = l;
            }
        }
    }
    __syncthreads();
}

template <int HD>
__device__ __forceinline__ void attn_load_q(const AttnArgs& a, AttnSmem<HD>& sm, int b, int h) {
    const float* q = a.q + ((size_t)b * a.n_heads + h) * a.group * HD;
    for (int e = threadIdx.x; e < a.group * HD; e += 32 * kAttWarps) (&sm.q[0][0])[e] = q[e];
    __syncthreads();
}

__device__ __forceinline__ int attn_keys(const AttnArgs& a, int b) {
    const int pos = a.positions[b];
    return pos >= a.max_ctx ? a.max_ctx : max(pos, -1) + 1;
}

// How the blocks of all rows and KV heads, in that order, are cut over the CTAs of the
// split: `units` blocks over `n` CTAs, CTA c taking [c units / n, (c + 1) units / n).
struct SplitPlan {
    int units, n;
    __device__ __forceinline__ int start(int c) const { return (int)((long long)c * units / n); }
    __device__ __forceinline__ int owner(int u) const { return (int)(((long long)(u + 1) * n - 1) / units); }
};
constexpr int kMinUnits = kAttWarps;     // blocks per CTA at least
__device__ __forceinline__ SplitPlan split_plan(const AttnArgs& a) {
    SplitPlan p{0, 0};
    for (int b = 0; b < a.rows; ++b) p.units += attn_keys(a, b) / kQBlock * a.n_heads;
    p.n = min(a.n_cta, (p.units + kMinUnits - 1) / kMinUnits);
    return p;
}

// One CTA per (row, KV head): all its blocks and its open block.
template <int HD>
__global__ void __launch_bounds__(32 * kAttWarps) k_attn_whole(const __grid_constant__ AttnArgs a) {
    __shared__ AttnSmem<HD> sm;
    const int h = blockIdx.x % a.n_heads, b = blockIdx.x / a.n_heads;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int keys = attn_keys(a, b);
    float* out = a.out + ((size_t)b * a.n_heads + h) * a.group * HD;
    if (keys == 0) {
        for (int e = threadIdx.x; e < a.group * HD; e += 32 * kAttWarps) out[e] = 0.f;
        return;
    }
    const size_t plane = ((size_t)a.layer * a.max_batch + b) * a.n_heads + h;
    attn_load_q(a, sm, b, h);
    const int nb = keys / kQBlock, nt = keys % kQBlock;
    uint32_t parts = 0;
    if (nb) {
        attn_blocks<HD>(a, sm, plane, 0, nb, warp, lane);
        parts = (1u << kAttWarps) - 1;
    }
    if (nt) {
        attn_tail<HD>(a, sm, plane, nt, warp, lane);
        parts |= 1u << kAttWarps;
    }
    attn_join<HD, true>(a, sm, parts, out, nullptr);
}

// The split: CTA c takes its range of blocks, which may cover several (row, KV head)
// pairs; each piece becomes partial slot c + pair (distinct: both only grow along the
// order of the blocks). The last rows * n_heads CTAs take the open blocks, slot
// n_cta + pairs + pair.
template <int HD>
__global__ void __launch_bounds__(32 * kAttWarps) k_attn_split(const __grid_constant__ AttnArgs a) {
    __shared__ AttnSmem<HD> sm;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int pairs = a.rows * a.n_heads;
    if ((int)blockIdx.x < pairs) {
        const int pair = blockIdx.x, b = pair / a.n_heads, h = pair % a.n_heads;
        const int nt = attn_keys(a, b) % kQBlock;
        if (nt) {
            attn_load_q(a, sm, b, h);
            attn_tail<HD>(a, sm, ((size_t)a.layer * a.max_batch + b) * a.n_heads + h, nt, warp, lane);
            const size_t slot = (size_t)a.n_cta + pairs + pair;
            attn_join<HD, false>(a, sm, 1u << kAttWarps, a.part_o + slot * a.group * HD, a.part_ml + slot * a.group * 2);
        }
    } else {
        const int c = blockIdx.x - pairs;
        const SplitPlan P = split_plan(a);
        if (c < P.n) {
            const int u0 = P.start(c), u1 = P.start(c + 1);
            int first = 0;   // first unit of row b
            for (int b = 0; b < a.rows && first < u1; ++b) {
                const int nb = attn_keys(a, b) / kQBlock;
                const int last = first + nb * a.n_heads;
                for (int u = max(u0, first); u < min(u1, last);) {
                    const int h = (u - first) / nb, base = first + h * nb;
                    const int stop = min(u1, base + nb);
                    attn_load_q(a, sm, b, h);
                    attn_blocks<HD>(a, sm, ((size_t)a.layer * a.max_batch + b) * a.n_heads + h, u - base, stop - base, warp, lane);
                    const size_t slot = (size_t)c + b * a.n_heads + h;
                    attn_join<HD, false>(a, sm, (1u << kAttWarps) - 1, a.part_o + slot * a.group * HD,
                                         a.part_ml + slot * a.group * 2);
                    u = stop;
                }
                first = last;
            }
        }
    }
    cudaTriggerProgrammaticLaunchCompletion();
}

// Joins the partials of one (row, query head): warps take slots in turn, lanes the dims.
constexpr int kJoinWarps = 8;
template <int HD>
__global__ void __launch_bounds__(32 * kJoinWarps) k_attn_merge_q(const __grid_constant__ AttnArgs a) {
    constexpr int D = HD / 32;
    __shared__ float so[kJoinWarps][HD], sm[kJoinWarps], sl[kJoinWarps];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int heads = a.n_heads * a.group, b = blockIdx.x / heads, hq = blockIdx.x % heads;
    const int h = hq / a.group, hg = hq % a.group, pairs = a.rows * a.n_heads, pair = b * a.n_heads + h;
    const int keys = attn_keys(a, b), nb = keys / kQBlock, nt = keys % kQBlock;
    const SplitPlan P = split_plan(a);
    int first = 0;
    for (int i = 0; i < b; ++i) first += attn_keys(a, i) / kQBlock * a.n_heads;
    first += h * nb;
    const int c0 = nb ? P.owner(first) : 0, n = nb ? P.owner(first + nb - 1) - c0 + 1 : 0;
    const int total = n + (nt ? 1 : 0);
    cudaGridDependencySynchronize();
    float M = -INFINITY, l = 0.f, o[D];
#pragma unroll
    for (int d = 0; d < D; ++d) o[d] = 0.f;
    for (int i = warp; i < total; i += kJoinWarps) {
        const size_t slot = i < n ? (size_t)c0 + i + pair : (size_t)a.n_cta + pairs + pair;
        const float2 ml = *reinterpret_cast<const float2*>(a.part_ml + (slot * a.group + hg) * 2);
        const float* p = a.part_o + (slot * a.group + hg) * HD + lane * D;
        const float Mn = fmaxf(M, ml.x), f = exp2f(M - Mn), w = exp2f(ml.x - Mn);
        M = Mn;
        l = fmaf(l, f, ml.y * w);
#pragma unroll
        for (int d = 0; d < D; ++d) o[d] = fmaf(o[d], f, p[d] * w);
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
    const int used = min(total, kJoinWarps);
    float top = -INFINITY, L = 0.f, x = 0.f;
    for (int i = 0; i < used; ++i) top = fmaxf(top, sm[i]);
    for (int i = 0; i < used; ++i) {
        const float f = exp2f(sm[i] - top);
        L = fmaf(f, sl[i], L);
        x = fmaf(f, so[i][e], x);
    }
    out[e] = x / L;
}

// ------------------------------------------------------------------ launches

constexpr int kSplitCtas = kQSms * 3;
constexpr int kWholeCtx = 512;    // contexts up to here run one CTA per (row, head)

bool attn_is_split(int max_ctx) { return max_ctx > kWholeCtx; }
size_t attn_slots(int rows, int n_heads) { return (size_t)kSplitCtas + 2 * (size_t)rows * n_heads; }

template <int HD>
cudaError_t attn_launch(AttnArgs& a, cudaStream_t st) {
    if (a.n_cta == 0) {
        k_attn_whole<HD><<<a.rows * a.n_heads, 32 * kAttWarps, 0, st>>>(a);
        return cudaGetLastError();
    }
    k_attn_split<HD><<<a.n_cta + a.rows * a.n_heads, 32 * kAttWarps, 0, st>>>(a);
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)(a.rows * a.n_heads * a.group));
    cfg.blockDim = dim3(32 * kJoinWarps);
    cfg.stream = st;
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, k_attn_merge_q<HD>, static_cast<const AttnArgs>(a));
    return e != cudaSuccess ? e : cudaGetLastError();
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
    const int wb = window < 1 ? 1 : window;
    const dim3 grid((unsigned)((wb + mk::kAppWarps - 1) / mk::kAppWarps), (unsigned)(rows * c->n_kv_heads),
                    (unsigned)(2 * n_layers));
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (c->head_dim == 64) mk::k_append<64><<<grid, 32 * mk::kAppWarps, 0, st>>>(a);
    else mk::k_append<128><<<grid, 32 * mk::kAppWarps, 0, st>>>(a);
    return cudaGetLastError() == cudaSuccess ? MK_OK : MK_ERR_CUDA;
}

extern "C" size_t mk_qcache_attention_workspace(const mk_qcache* c, int rows, int n_heads, int max_ctx) {
    if (mk::qcache_check(c) != MK_OK || rows < 1 || rows > c->max_batch || n_heads < c->n_kv_heads ||
        n_heads % c->n_kv_heads != 0 || n_heads / c->n_kv_heads > mk::kMaxGroupHeads || max_ctx < 1 ||
        max_ctx > c->max_seq || !mk::attn_is_split(max_ctx))
        return 0;
    const size_t slots = mk::attn_slots(rows, c->n_kv_heads) * (size_t)(n_heads / c->n_kv_heads);
    return slots * (size_t)(c->head_dim + 2) * sizeof(float);
}

extern "C" mk_status mk_qcache_attention(const mk_qcache* c, int layer, int rows, int n_heads, int max_ctx,
                                         const float* q, const int32_t* positions, float* out, void* workspace,
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
    a.out = out;
    if (need) {
        a.n_cta = mk::kSplitCtas;
        a.part_ml = static_cast<float*>(workspace);
        a.part_o = a.part_ml + mk::attn_slots(rows, c->n_kv_heads) * (size_t)a.group * 2;
    }
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const cudaError_t e = c->head_dim == 64 ? mk::attn_launch<64>(a, st) : mk::attn_launch<128>(a, st);
    return e == cudaSuccess ? MK_OK : MK_ERR_CUDA;
}
