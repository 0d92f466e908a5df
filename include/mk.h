/*
 * mk.h -- C ABI of the persistent decode megakernel library (libmk.so).
 *
 * One decode step of a Llama-style decoder (batch 1 or a few sequences) runs as
 * ONE persistent sm_100a kernel: one CTA per SM, each working through a
 * host-built list of instructions, with dependencies between instructions
 * resolved inside the kernel rather than by kernel boundaries. This is the design
 * of the "Look Ma, No Bubbles" Llama-3.2-1B megakernel (summaries: sections
 * "Fusing Operations with an On-GPU Interpreter" and "Custom Synchronization
 * Mechanism") and of the Cohere decode megakernel (section "Megakernel 是什么": a
 * resident block per SM reading a host-written task list of tile-sized work
 * items). Those designs wait on atomic-increment counters; here the activations
 * that cross SMs carry their own validity (64-bit words tagged with the step,
 * layer and producer), the consumer polls the words themselves, and counters
 * remain as completion counts (see mk_read_counters).
 *
 * Conventions for every entry point:
 *   - Pointers documented as "device" must be CUDA device memory of the handle's
 *     device; "host" pointers are ordinary host memory.
 *   - bf16 tensors are arrays of uint16 bit patterns (IEEE bfloat16), row-major.
 *   - `stream` is a cudaStream_t passed as void* (NULL = legacy default stream).
 *   - No entry point throws; each returns an mk_status. Host-checkable errors are
 *     returned before anything is enqueued. Errors found by the GPU during a step
 *     are recorded on the device and reported by mk_get_status().
 *   - A handle is not thread-safe; distinct handles are independent.
 *   - Calls that enqueue GPU work for a handle (the decode steps) run on the calling
 *     thread's current device and are refused with MK_ERR_INVALID_ARG when that is
 *     not the handle's device. The synchronous calls (create, schedule, status,
 *     readers, destroy) switch to the handle's device themselves and give the
 *     caller's current device back before they return.
 */
#ifndef MK_H
#define MK_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum mk_status {
    MK_OK = 0,
    MK_ERR_INVALID_ARG = 1,   /* null pointer, bad size, batch > schedule batch ... */
    MK_ERR_CUDA = 2,          /* a CUDA runtime call failed (message via mk_get_status) */
    MK_ERR_UNSUPPORTED = 3,   /* shape this build has no kernel for, or the device cannot
                                 keep one CTA resident on every SM */
    MK_ERR_NO_SCHEDULE = 4,   /* mk_decode_step before mk_build_schedule */
    MK_ERR_TIMEOUT = 5,       /* device: a counter or barrier wait ran past its budget */
    MK_ERR_BAD_TOKEN = 6,     /* device: token outside [0, vocab) */
    MK_ERR_BAD_POSITION = 7,  /* device: position outside [0, min(max_seq, max_ctx)) */
    MK_ERR_OUT_OF_MEMORY = 8
} mk_status;

/* Model shape. The decoder is Llama-style: RMSNorm (eps inside the root),
 * rotate-half RoPE with inv_freq_i = rope_theta^(-2i/head_dim), grouped-query
 * attention (query head h reads KV head h / (n_heads / n_kv_heads)), SiLU-gated
 * MLP, tied embeddings (the embedding table is also the LM head). */
typedef struct mk_config {
    int32_t n_layers, hidden, n_heads, n_kv_heads, head_dim, ffn, vocab;
    float rms_eps;
    double rope_theta;
    int32_t max_batch;   /* batch dimension of the KV cache and largest schedulable batch */
    int32_t max_seq;     /* slot dimension of the KV cache */
} mk_config;
/* Accepted ranges (else MK_ERR_UNSUPPORTED from mk_create, 0 from mk_packed_bytes):
 * 1..64 layers; hidden a multiple of 256 up to 65536; head_dim 64 or 128; at most 32
 * query heads and 4 per KV head; n_heads*head_dim a multiple of 256; ffn a multiple
 * of 1024 up to 262144; vocab a multiple of 4 up to 2^24; max_batch 1..8; max_seq
 * 1..2^20. mk_create further needs a shape the kernels are instantiated for. */

/* Weight pointers for mk_create. Matrices are bf16 row-major [out][in]:
 *   wq [n_heads*head_dim][hidden], wk/wv [n_kv_heads*head_dim][hidden],
 *   wo [hidden][n_heads*head_dim], wgate/wup [ffn][hidden], wdown [hidden][ffn],
 *   embed [vocab][hidden]; norm vectors bf16 [hidden].
 * Per-layer fields are HOST arrays of n_layers pointers. With mk_create the
 * pointed-to tensors are device memory; with mk_pack_weights_host they are host
 * memory. The library copies what it needs: the caller may free them after the
 * call returns. */
typedef struct mk_weights {
    const void* embed;
    const void* const* attn_norm;
    const void* const* wq;
    const void* const* wk;
    const void* const* wv;
    const void* const* wo;
    const void* const* mlp_norm;
    const void* const* wgate;
    const void* const* wup;
    const void* const* wdown;
    const void* final_norm;
} mk_weights;

typedef struct mk_handle mk_handle;

/* Create a handle on `device`: validates the shape, packs the weights into one
 * library-owned device buffer (layout: see mk_pack_weights_host), builds the RoPE
 * table (angles in double, cos/sin stored as float) and allocates the scratch
 * (activations, attention partials, counters). Synchronous. On error *out is NULL.
 * Defining passage: the Cohere decode megakernel page ("Cohere 开源 Megakernel 推理
 * 系统"), section "Megakernel 是什么": one resident thread block per SM for the
 * whole decode step, working from host-prepared tile-sized tasks; the handle
 * holds what those tasks read, laid out once before any step (weights as
 * contiguous tiles, the RoPE table, the counters and scratch in global memory). */
mk_status mk_create(const mk_config* cfg, const mk_weights* w, int device, mk_handle** out);

/* Options for mk_build_schedule; pass NULL for defaults. Zero fields mean "auto". */
typedef struct mk_schedule_opts {
    int32_t n_sm;            /* SMs to use (<= device SMs); 0 = all */
    int32_t part_keys;       /* keys per attention partition (a multiple of 8 up to the
                                ring's keys-per-stage, else a multiple of it); 0 = one
                                partition per (sequence, KV group) up to 320 keys, beyond
                                that as many as leave one item per SM (each of at most
                                512 keys and what the ring holds) */
    int32_t rowblocks_down;  /* 4-row blocks per down-projection instruction at most
                                (1..16); 0 = 16 */
    uint32_t seed;           /* 0 = plain greedy placement; else ties are broken by a
                                seeded shuffle (for robustness tests) */
    int32_t wait_timeout_ms; /* budget of every device wait; 0 = 2000 ms */
    int32_t test_drop_item;  /* failure-detection test hook: 1-based index, in the list
                                order, of one instruction that computes but never publishes
                                its outputs or its completion (its consumers then end the
                                step with MK_ERR_TIMEOUT); 0 = none */
    int32_t trace;           /* nonzero: every step records per-job timestamps (see
                                mk_read_trace) */
    int32_t proj;            /* the projections' arithmetic at batch > 1: MK_PROJ_AUTO
                                (the tensor cores), MK_PROJ_CUDA_CORES or
                                MK_PROJ_TENSOR_CORES (batch 1 always runs on the CUDA
                                cores) */
} mk_schedule_opts;

/* mk_schedule_opts.proj. Tensor cores: each instruction's weight rows stream as
 * 64-column TMA boxes (128-byte swizzle) and one thread issues tcgen05.mma
 * (M = 128 weight rows, N = 16: the batch's fp32 inputs split into bf16 high and
 * low parts, K = 16 per instruction) into an fp32 accumulator in Tensor Memory,
 * read back by the compute warps for the same fused epilogues; four warps issue
 * the MMAs, one per K step of each box. CUDA cores: each 4-row tile's batched fp32
 * dot product, as at batch 1. AUTO picks the tensor cores: measured on the
 * 3B-style shape at batch 8 and 2048 positions (one B200) the step takes 6.30 ms
 * against 6.63 ms. The two differ only in the order and form of the fp32
 * accumulation. The tensor-core path needs a vocabulary that is a multiple of 8
 * (else the CUDA cores run). */
#define MK_PROJ_AUTO 0
#define MK_PROJ_CUDA_CORES 1
#define MK_PROJ_TENSOR_CORES 2

/* Build the per-SM instruction lists for `batch` sequences (1 <= batch <= max_batch)
 * whose steps use at most `max_ctx` keys (position + 1 <= max_ctx <= max_seq), and
 * upload them. Replaces any earlier schedule. Synchronous.
 * Defining passages: the "Look Ma, No Bubbles" summary, section "Fusing Operations
 * with an On-GPU Interpreter" (each SM executes a sequence of instructions such as
 * fused RMSNorm + QKV + RoPE, attention, ...), and the Stanford write-up
 * ("斯坦福团队新作：Llama-1B实现毫秒级推理获Andrej Karpathy盛赞"), section
 * "Megakernel：从零设计的融合思路" (an execution plan per SM, dependencies between
 * instructions arranged statically before the run); the Cohere page, section
 * "Megakernel 是什么" (the host writes the task list into global memory).
 * The attention of a (sequence, KV group) is split into at most 32 key partitions,
 * each holding at most what the SM's weight ring holds at once (and 512 keys), so
 * max_ctx has a ceiling that depends on the shape and batch: 16384 keys for the
 * Llama-3.2-1B shape; for head_dim 128 with 24 query and 8 KV heads, 12288 at
 * batch 1 and 7168 at batch 2-8 (on the CUDA-core path 12288 at batch 2 and 6144 at
 * 3-8). A larger max_ctx
 * (or a part_keys that needs more than 32 partitions) returns MK_ERR_INVALID_ARG. */
mk_status mk_build_schedule(mk_handle* h, int batch, int max_ctx, const mk_schedule_opts* opts);

/* One decode step of the persistent megakernel, asynchronous on `stream`.
 * Defining passage: the "Look Ma, No Bubbles" summary, section "Megakernel: The
 * Core Solution" (the whole Llama-1B forward pass as one kernel, so loads and
 * compute continue across what would be kernel boundaries), with section "Custom
 * Synchronization Mechanism" (dependencies inside the kernel; the MLP's
 * intermediate state in four chunks so the down-projection starts early).
 *   tokens, positions : device int32 [batch]
 *   k_cache, v_cache  : device bf16 [n_layers][max_batch][n_kv_heads][max_seq][head_dim],
 *                       caller-owned; sequence b reads slots 0..positions[b] and writes
 *                       slot positions[b] (its RoPE'd key and its value)
 *   logits            : device fp32 [batch][vocab]
 * Enqueues exactly one cooperative kernel launch; no host synchronisation, no
 * allocation. A step with a bad token or position writes no KV slot and leaves the
 * logits unspecified; the error is reported by mk_get_status. Returns
 * MK_ERR_INVALID_ARG (nothing enqueued) for a NULL pointer, a KV cache that is not
 * 16-byte aligned, or a calling thread whose current device is not the handle's;
 * MK_ERR_NO_SCHEDULE before mk_build_schedule. */
mk_status mk_decode_step(mk_handle* h, const int32_t* tokens, const int32_t* positions,
                         void* k_cache, void* v_cache, float* logits, void* stream);

/* n_steps greedy decode steps back to back, asynchronous on `stream`, with no host
 * work between them: each is mk_decode_step with the greedy choice fused into its
 * LM head. Each LM-head instruction reduces its rows to the best (largest logit,
 * lowest index among equal ones, NaN never chosen; an all-NaN row gives 0) per
 * sequence; the SM that completes the step's LM head picks each sequence's next
 * token from those and writes it over tokens[b], writes positions[b] + 1 over
 * positions[b], and, when `generated` (device int32 [n_steps][batch]) is given,
 * stores it at generated[step][b]. The next launch then decodes it. The tokens
 * equal mk_greedy_select's on the same logits, bit for bit; `logits` holds the
 * last step's. Arguments as for mk_decode_step (tokens and positions are read and
 * written); n_steps >= 1 launches are enqueued. The caller keeps the positions
 * below max_ctx: a step past it is skipped and reported (MK_ERR_BAD_POSITION), as
 * are the steps after it. Defining passage: the "Look Ma, No Bubbles" summary,
 * section "Megakernel: The Core Solution" (no kernel boundaries inside a forward
 * pass): here the token choice, too, stays inside the step's kernel. */
mk_status mk_decode_steps_greedy(mk_handle* h, int32_t* tokens, int32_t* positions, void* k_cache,
                                 void* v_cache, float* logits, int32_t* generated, int n_steps, void* stream);

/* The same step as a sequence of ordinary kernels (one per op and layer), the
 * multi-kernel "bubble" baseline; identical arguments, identical arithmetic, so
 * its results equal mk_decode_step's bit for bit. Capturable in a CUDA graph. */
mk_status mk_baseline_decode_step(mk_handle* h, const int32_t* tokens, const int32_t* positions,
                                  void* k_cache, void* v_cache, float* logits, void* stream);

/* End-to-end step from HOST buffers: copies tokens and positions (host int32
 * [batch], preferably pinned) to the device, runs mk_decode_step, copies the
 * logits back to `logits_host` (fp32 [batch][vocab]) and synchronises `stream`.
 * Uses handle-owned device staging (no allocation per call). Returns the
 * host-side status; device-detected errors are reported by mk_get_status. */
mk_status mk_decode_step_host(mk_handle* h, const int32_t* tokens_host,
                              const int32_t* positions_host, void* k_cache, void* v_cache,
                              float* logits_host, void* stream);

/* Synchronises the device, then reports and clears the device-side error state.
 * *device_status receives the first error recorded since the last call (MK_OK if
 * none); msg (may be NULL) receives a one-line description. After an error every
 * step is skipped until this call clears it. Returns MK_ERR_CUDA if the sync fails. */
mk_status mk_get_status(mk_handle* h, mk_status* device_status, char* msg, size_t msg_len);

/* The device int32 that holds what mk_get_status would report, for kernels that go by it; valid until the
 * handle's next mk_build_schedule or mk_destroy. NULL for a NULL handle and before mk_build_schedule. */
const int32_t* mk_device_status(mk_handle* h);

/* Frees everything the handle owns. NULL is allowed. */
void mk_destroy(mk_handle* h);

const char* mk_status_str(mk_status s);

/* Greedy selection between decode steps: next_tokens[b] = the index v in [0, vocab)
 * of the largest logits[b][v], the lowest such index where several are equal (the
 * greedy decoding rule of the decoder's generation loop). NaN entries are never
 * selected; a row of NaNs gives 0.
 *   logits       device fp32 [batch][vocab], rows contiguous (mk_decode_step's output)
 *   batch, vocab >= 1
 *   next_tokens  device int32 [batch]; may be the tokens buffer of the next
 *                mk_decode_step, so a decode loop needs no host round trip
 *   positions    device int32 [batch] or NULL: when given, each positions[b] is
 *                incremented by one in the same launch
 *   stream       the CUDA stream the selection is enqueued on
 * Enqueues one kernel launch (one CTA per sequence) on the calling thread's current
 * device, which must own the buffers and the stream; no synchronisation, no
 * allocation, capturable in a CUDA graph. Returns MK_ERR_INVALID_ARG for a NULL
 * logits or next_tokens pointer or a size below 1, MK_ERR_CUDA if the launch fails. */
mk_status mk_greedy_select(const float* logits, int batch, int vocab, int32_t* next_tokens,
                           int32_t* positions, void* stream);

/* ------------------------------------------------------------------ beams
 *
 * Beam search over decode steps: mk_beam_select picks the continuations, mk_cache_reorder
 * (or mk_qcache_reorder) lets the rows of the cache follow them. A sequence's beams are
 * `beams` consecutive rows of the step's batch. */

/* The n_out best continuations of each of `batch` sequences with `beams` rows of logits
 * each: by total(k, v) = scores[k] + log_softmax(logits[k])[v], larger first; equal
 * totals in the order of the beams, within a beam by the larger logit, equal logits by
 * the lower token. Totals are formed and compared in 64 bits, from a row maximum and a
 * 32-bit sum; scores are rounded to fp32 on the way out.
 *   logits        device fp32 [batch * beams][vocab], rows row_stride elements apart
 *                 (row_stride >= vocab; any 4-byte alignment, all alike)
 *   beams         1..16; n_out 1..32 and at most beams * vocab; vocab 1..2^24
 *   scores        device fp32 [batch][beams], running log probabilities; a beam that
 *                 is not in use has -infinity
 *   finished      device int32 [batch][beams] or NULL. A nonzero beam's logits are not
 *                 read: its one continuation is `eos` at its own score
 *   eos           a token in [0, vocab) when `finished` is given; else unused
 *   next_tokens   device int32 [batch][n_out], best first
 *   parents       device int32 [batch][n_out]: the ROW (sequence * beams + beam) it continues
 *   next_scores   device fp32 [batch][n_out]
 *   next_finished device int32 [batch][n_out] or NULL (needs `finished`): 1 where the parent
 *                 was finished or the token is eos, else 0
 *   positions     device int32 [batch * beams] or NULL: each is incremented by one
 * A masked logit (-infinity) and a NaN are chosen only where nothing else is left, with score
 * -infinity; they add nothing to the row's sum. Infinite logits share their row's probability.
 * next_scores may be scores, and next_finished may be finished: of several sequences only with n_out ==
 * beams (else MK_ERR_INVALID_ARG). Any other overlap of inputs and outputs is an error that is not detected.
 * Enqueues one kernel launch (one cluster of CTAs per sequence) on the calling thread's current
 * device, which must own the buffers and the stream; no synchronisation, no allocation, no
 * workspace, capturable in a CUDA graph. MK_ERR_INVALID_ARG for a NULL required pointer, a size
 * out of range or an eos outside [0, vocab); MK_ERR_UNSUPPORTED above the limits on beams,
 * n_out, vocab and batch (2^20). */
mk_status mk_beam_select(const float* logits, int64_t row_stride, int batch, int beams, int vocab, int n_out,
                         const float* scores, const int32_t* finished, int32_t eos, int32_t* next_tokens,
                         int32_t* parents, float* next_scores, int32_t* next_finished, int32_t* positions,
                         void* stream);

/* The same behind a step that may have failed: where *status (device int32, read when the call runs) is not
 * MK_OK, nothing is chosen; every parent is -1, which mk_cache_reorder and mk_qcache_reorder leave alone, and
 * the other outputs and the positions stay as they are. status: a step's status_out, or mk_device_status(). */
mk_status mk_beam_select_checked(const float* logits, int64_t row_stride, int batch, int beams, int vocab, int n_out,
                                 const float* scores, const int32_t* finished, int32_t eos, int32_t* next_tokens,
                                 int32_t* parents, float* next_scores, int32_t* next_finished, int32_t* positions,
                                 const int32_t* status, void* stream);

/* Rows of a KV cache take over other rows' slots, all at once and in place: for each row r < rows,
 * layer and head, slots starts[r] <= s < lengths[parents[r]] of row r become those of row parents[r]
 * as they were before the call. Reorders beams (parents from mk_beam_select, lengths = the advanced
 * positions), forks a sequence into free rows, and compacts live rows over finished ones.
 *   cfg              reads n_layers, n_kv_heads, head_dim, max_batch and max_seq only
 *   k_cache, v_cache device bf16 [n_layers][max_batch][n_kv_heads][max_seq][head_dim], 16-byte aligned
 *   rows             1..max_batch
 *   parents          device int32 [rows]: a row below `rows`; the row itself or any other value
 *                    leaves row r as it is
 *   lengths          device int32 [rows]: the slots in use of each row BEFORE the call (clamped to
 *                    [0, max_seq])
 *   starts           device int32 [rows] or NULL (0): slots below starts[r] are the same in row r and
 *                    its parent (a shared prompt) and are not moved
 * Slots outside those ranges and rows >= rows are not touched. Enqueues one kernel launch on the
 * calling thread's current device; no synchronisation, no allocation, capturable. MK_ERR_INVALID_ARG
 * for a NULL pointer, an unaligned cache, caches that overlap or a bad row count, MK_ERR_UNSUPPORTED for a geometry
 * outside mk_create's ranges. */
mk_status mk_cache_reorder(const mk_config* cfg, void* k_cache, void* v_cache, int rows, const int32_t* parents,
                           const int32_t* lengths, const int32_t* starts, void* stream);

/* ------------------------------------------------------------------ the 8-bit cache
 *
 * A KV cache in 8 bits with one scale per block of MK_QCACHE_BLOCK tokens of one head, for keys and
 * for values: code = rint(x * (127 / amax)), scale = amax / 127, value = code * scale, amax the
 * block's largest magnitude. It takes half the bytes of the bf16 cache, so half of what a decode step
 * at a long context reads. The tokens of a row's open block (the last length % MK_QCACHE_BLOCK) stay
 * bf16 in the tail buffers until the block is full, and are rounded once, from their own values.
 * A row's length only grows, or goes back to a multiple of MK_QCACHE_BLOCK (its open block is then
 * empty), or to a length inside the block that is open now.
 * A block whose amax is below 2^-60 is held as zeros (scale 0). A block that holds an infinity or a
 * NaN gets a NaN scale: whatever attends to it is NaN. */
#define MK_QCACHE_BLOCK 32

/* Caller-owned device buffers; nothing in them needs to be initialised, and only the calls below
 * write them. The codes and tails are 16-byte aligned. n_blocks = ceil(max_seq / MK_QCACHE_BLOCK). Accepted: 1..64 layers, max_batch 1..8,
 * 1..32 KV heads, max_seq 1..2^20, head_dim 64 or 128. */
typedef struct mk_qcache {
    int32_t n_layers, max_batch, n_kv_heads, max_seq, head_dim, reserved0;
    void* k_codes;   /* int8 [n_layers][max_batch][n_kv_heads][max_seq][head_dim] */
    void* v_codes;
    float* k_scale;  /* [n_layers][max_batch][n_kv_heads][n_blocks] */
    float* v_scale;
    void* k_tail;    /* bf16 [n_layers][max_batch][n_kv_heads][MK_QCACHE_BLOCK][head_dim] */
    void* v_tail;
} mk_qcache;

/* Stores new keys and values: a decoded token, a prompt, or a bf16 cache that is taken over.
 * Row r gets counts[r] tokens at slots positions[r] .. positions[r] + counts[r] - 1, in each of the
 * layers first_layer .. first_layer + n_layers - 1; blocks that become full are quantised.
 *   k_new, v_new  device bf16, 16-byte aligned; element (layer, row, head, token, dim) sits at
 *                 layer * strides[0] + row * strides[1] + head * strides[2] + token * strides[3] + dim
 *                 (layer counted from first_layer; strides in elements, multiples of 8, host array)
 *   rows          1..max_batch; n_new >= 1: the tokens k_new and v_new hold per row
 *   positions     device int32 [rows]: the row's length so far
 *   counts        device int32 [rows] or NULL (n_new each)
 * A row whose count is outside 1..n_new, or whose tokens would not fit [0, max_seq), is left as it is.
 * k_new and v_new may not overlap the cache's buffers. One kernel launch; no allocation, capturable. */
mk_status mk_qcache_append(const mk_qcache* c, int first_layer, int n_layers, int rows, int n_new, const void* k_new,
                           const void* v_new, const int64_t* strides, const int32_t* positions, const int32_t* counts,
                           void* stream);

/* mk_cache_reorder on the 8-bit cache: closed blocks from the one that holds starts[r] move whole, the
 * open block's tokens from starts[r] on. Row r's open block must have been that of its parent up to
 * starts[r] (as it is where the slots below starts[r] are the same in both). */
mk_status mk_qcache_reorder(const mk_qcache* c, int rows, const int32_t* parents, const int32_t* lengths,
                            const int32_t* starts, void* stream);

/* Decode attention of one layer over the 8-bit cache, one query token per row: for each row r and query
 * head h, out = sum_s softmax_s(q . k_s / sqrt(head_dim)) v_s over the slots s = 0 .. positions[r] of
 * KV head h / (n_heads / n_kv_heads).
 *   positions     device int32 [rows]: the row's last token, or another one of its open block; it says which
 *                 of the row's blocks are closed and so held as codes. For an earlier slot of a row that holds more,
 *                 call mk_qcache_attention_prefix, unless it is the last slot of a closed block
 *   n_heads       a multiple of n_kv_heads, at most 4 query heads per KV head (else MK_ERR_UNSUPPORTED)
 *   max_ctx       1..max_seq: at most the first max_ctx slots of a row are read (a larger position is still
 *                 where the row ends); a negative position (an empty row) gives zeros
 *   q, out        device fp32 [rows][n_heads][head_dim]
 *   workspace     device, 16-byte aligned, mk_qcache_attention_workspace() bytes; need not be
 *                 initialised, belongs to the call until it has run (calls that overlap on the GPU
 *                 need one each); may be NULL where that is 0
 * Both products are exact sums of whole numbers (a head's queries in 30 bits of its largest, the softmax's
 * weights times their block's value scale in 31 bits of the largest so far), scaled and added in fp32; the
 * softmax's sum is fp32 and takes every key at its weight, whatever the sizes of the values. The open block is fp32. A query
 * head with an infinity or a NaN gives NaN, as does a q . k beyond fp32's range. One or two kernel launches; no allocation,
 * capturable; the same inputs give the same bits. */
mk_status mk_qcache_attention(const mk_qcache* c, int layer, int rows, int n_heads, int max_ctx, const float* q,
                              const int32_t* positions, float* out, void* workspace, size_t workspace_bytes,
                              void* stream);

/* The same for any slots of a row: attends to s = 0 .. positions[r] of a row that holds lengths[r] tokens (device
 * int32 [rows]; positions and max_ctx beyond it stop at it). */
mk_status mk_qcache_attention_prefix(const mk_qcache* c, int layer, int rows, int n_heads, int max_ctx, const float* q,
                                     const int32_t* positions, const int32_t* lengths, float* out, void* workspace,
                                     size_t workspace_bytes, void* stream);

/* Bytes of workspace either attention call with these arguments needs (0 also for arguments it
 * refuses). */
size_t mk_qcache_attention_workspace(const mk_qcache* c, int rows, int n_heads, int max_ctx);

/* One decode step on the 8-bit cache, as a sequence of ordinary kernels (one per op and layer,
 * asynchronous on `stream`): mk_baseline_decode_step with the new key and value stored by
 * mk_qcache_append and attention by mk_qcache_attention. For contexts beyond what
 * mk_build_schedule takes, or a cache of half the bytes; it needs no schedule.
 *   c                the cache; n_layers, n_kv_heads and head_dim as the handle's model
 *   batch, max_ctx   1 <= batch <= c->max_batch; positions[b] + 1 <= max_ctx <= min(c->max_seq, the
 *                    model's max_seq)
 *   tokens, positions, logits  as for mk_decode_step; sequence b attends to slots 0..positions[b]
 *   workspace        device, 256-byte aligned, mk_decode_step_qcache_workspace() bytes; need not be
 *                    initialised, belongs to the call until it has run
 *   status_out       device int32 or NULL: the step's device status (MK_OK, MK_ERR_BAD_TOKEN,
 *                    MK_ERR_BAD_POSITION); it is not reported by mk_get_status
 * A step with a bad token or position leaves the cache as it is and the logits unspecified. Runs on
 * the calling thread's current device, which must be the handle's. No allocation, capturable. */
mk_status mk_decode_step_qcache(mk_handle* h, const mk_qcache* c, int batch, int max_ctx, const int32_t* tokens,
                                const int32_t* positions, float* logits, void* workspace, size_t workspace_bytes,
                                int32_t* status_out, void* stream);

/* Bytes of workspace a mk_decode_step_qcache call with these arguments needs (0 for arguments it
 * refuses). */
size_t mk_decode_step_qcache_workspace(mk_handle* h, const mk_qcache* c, int batch, int max_ctx);

/* ------------------------------------------------------------------ inspection */

/* One instruction of the per-SM lists (48 bytes). An SM's CTA runs its list in
 * order; each instruction is one "job" for all of the CTA's compute warps (a
 * down-projection is four jobs, one per MLP chunk; up to eight consecutive
 * attention items form one job, one item per warp). The kinds: */
enum {
    MK_OP_QKV = 1,     /* RMSNorm + QKV matvec + RoPE; writes q and the KV slot */
    MK_OP_ATTN = 2,    /* GQA attention over one key partition of a (sequence, KV group)
                          pair; the pair's last partition to finish merges the pair */
    MK_OP_OPROJ = 3,   /* O-projection + residual */
    MK_OP_GATEUP = 4,  /* RMSNorm + gate/up matvec + SiLU-gated product */
    MK_OP_DOWN = 5,    /* down-projection over the 4 MLP chunks + residual */
    MK_OP_LMHEAD = 6   /* final RMSNorm + LM head */
};
#define MK_NO_COUNTER 0xffffffffu

typedef struct mk_instr {
    uint16_t op, layer;
    uint16_t batch;      /* sequence (MK_OP_ATTN), else 0 */
    uint16_t group;      /* KV group (QKV, ATTN), else 0 */
    uint32_t first;      /* first 4-row tile / row block (DOWN) / first key (ATTN);
                            GATEUP: first tile of the SM's slice of each MLP chunk */
    uint32_t count;      /* tiles / row blocks / keys */
    uint32_t seq;        /* index of its first ring stage fill in this SM's stream */
    uint32_t nfill;      /* ring stage fills it consumes */
    uint32_t wait_ctr;   /* counter waited on (MK_NO_COUNTER: none); DOWN waits on the
                            4 consecutive chunk counters wait_ctr .. wait_ctr+3 */
    uint32_t wait_n;     /* increments that counter receives per step (DOWN: chunk 0) */
    uint32_t signal_ctr; /* counter incremented by one when the instruction is done;
                            ATTN: the layer's attention counter, incremented once per
                            query head when that head's output is final */
    uint32_t job_items;  /* 1: every instruction (an attention item included) is one
                            job of the SM's compute warps (DOWN: four, one per chunk) */
    uint32_t aux0, aux1; /* DOWN: per-step increments of chunk counters 1, 2 (low and
                            high 16 bits of aux0) and 3 (aux1). ATTN: aux0 = the pair's
                            arrival counter (heads whose partial is stored). LMHEAD:
                            aux0 = its ordinal among the step's LM-head instructions. GATEUP:
                            aux0 = tiles per chunk; the instruction's tile i is tile
                            (i / aux0) * (ffn / 8) + first + i % aux0 (chunk-major). QKV and
                            GATEUP: aux1 = how many consecutive counters from signal_ctr
                            the instruction increments by one each (the KV groups / MLP
                            chunks its tiles touch; 0 reads as 1). Else 0 */
} mk_instr;

typedef struct mk_schedule_info {
    int32_t n_sm, batch, max_ctx, part_keys, n_parts, keys_per_stage;
    int32_t stage_bytes, n_stages, n_counters, n_instr;
    uint64_t bytes_per_step;    /* weight + KV bytes one step streams */
    uint64_t max_sm_bytes;      /* largest per-SM share of those bytes */
    uint64_t min_sm_bytes;
    int32_t proj;               /* the projections' path: MK_PROJ_CUDA_CORES or _TENSOR_CORES */
    int32_t reserved0;
} mk_schedule_info;

/* Plans a schedule on the host only (no device, no handle): writes up to
 * `cap` instructions to instr_out (may be NULL to query), n_sm+1 list offsets to
 * sm_offsets (may be NULL) and the summary to info. `stage_bytes` is the ring
 * stage size the kernel would use (0 = the library's choice for this shape).
 * Returns MK_ERR_INVALID_ARG if cap is too small (info->n_instr says how many). */
mk_status mk_plan_schedule_host(const mk_config* cfg, int batch, int max_ctx, int n_sm,
                                const mk_schedule_opts* opts, mk_instr* instr_out, size_t cap,
                                int32_t* sm_offsets, mk_schedule_info* info);

/* One tensor map of the tensor-core path (mk_schedule_opts.proj): a view of the
 * packed weights (mk_pack_weights_host's layout) as bf16 elements. Element
 * (c_0, ..., c_{rank-1}) sits at byte base_offset + 2 * c_0 + sum_{i >= 1} c_i *
 * strides[i - 1] of the packed buffer; box is the block one TMA copy reads (one
 * fill: 64 columns x rows x boxes of 64 columns). index is the map's place in the
 * kernel's table. */
typedef struct mk_tmap_spec {
    int32_t index, rank;
    uint64_t base_offset;
    uint64_t dims[5];
    uint64_t strides[4];
    uint32_t box[5];
} mk_tmap_spec;

/* The tensor maps a schedule with ring stages of `stage_bytes` uses (host only, for
 * inspection and tests): writes up to `cap` specs to out (may be NULL to query)
 * and their count to *n. MK_ERR_UNSUPPORTED for a shape the kernels do not take. */
mk_status mk_tensor_map_specs_host(const mk_config* cfg, uint32_t stage_bytes, mk_tmap_spec* out, size_t cap,
                                   size_t* n);

/* Summary of the handle's current schedule. */
mk_status mk_get_schedule_info(mk_handle* h, mk_schedule_info* info);

/* Copies the handle's step counters (uint32 each) to host memory: the
 * dependency counters, then epoch, then the end-of-step arrival count.
 * *n_total receives how many exist; at most n are copied. Synchronous. */
mk_status mk_read_counters(mk_handle* h, uint32_t* host, size_t n, size_t* n_total);

/* Per-job timestamps of the last traced step (schedule built with opts.trace):
 * uint64 [n_sm][jobs][16] globaltimer nanoseconds -- 0 activation warp starts
 * waiting for a free input slot, 1 slot free, 2 the activation warp starts its
 * part of the job, 3 its part is ready (the slot is handed to the compute
 * warps), 4 compute warp 0 starts (it then builds the job's input from the
 * producers' tagged words), 5 the job's last compute warp finished, 6 op |
 * layer << 8 | chunk << 24, 7 compute warp 0 has its first ring fill of the job
 * (0 if it had none), 8..15 finer op-specific points of compute warp 0 (15: the
 * job's input built; 0 where unused).
 * *jobs receives the per-SM job capacity; at most `bytes` are copied.
 * Synchronous. */
mk_status mk_read_trace(mk_handle* h, uint64_t* host, size_t bytes, int32_t* jobs);

/* Bytes of the packed weight buffer for `cfg`. */
size_t mk_packed_bytes(const mk_config* cfg);

/* Packs host weights into `dst` (host, mk_packed_bytes(cfg) bytes) with the same
 * layout mk_create builds on the device, 256-byte aligned regions in this order:
 *   embed      [vocab][hidden] unchanged (it is also the LM head);
 *   per layer:
 *     QKV      4-row tiles of [4][hidden]; KV group g holds, in order, its
 *              n_heads/n_kv_heads query heads, key head g, value head g; a query or
 *              key head's tile j holds rows {2j, 2j+d/2, 2j+1, 2j+1+d/2} (the two
 *              RoPE pairs), a value head's tile j rows {4j..4j+3};
 *     O        wo unchanged [hidden][n_heads*head_dim];
 *     gate/up  tile j = rows {gate 2j, up 2j, gate 2j+1, up 2j+1} of [4][hidden];
 *     down     for row block r (rows 4r..4r+3), chunk c (columns c*ffn/4 ..): a
 *              [4][ffn/4] tile, ordered [r][c];
 *   norms      attn_norm[l], mlp_norm[l] for each layer, then final_norm.
 * Bit copy only. */
mk_status mk_pack_weights_host(const mk_config* cfg, const mk_weights* w, void* dst,
                               size_t dst_bytes);

/* The multi-kernel decode step (as mk_baseline_decode_step) for callers that
 * cannot allocate device memory -- an engine whose device memory is all handed
 * out by its own arena, or code running where cudaMalloc is not allowed. It
 * needs no handle and allocates nothing (no cudaMalloc, no cudaFree, no
 * allocating library call); the web pages describe no such entry point, it has
 * no counterpart there. The caller owns every input and output:
 *   cfg               the model (as for mk_create)
 *   packed            device, mk_packed_bytes(cfg) bytes in the mk_pack_weights_host
 *                     layout (e.g. packed on the host and copied by the caller)
 *   tokens, positions device int32 [batch]
 *   k_cache, v_cache  device bf16 [n_layers][max_batch][n_kv_heads][max_seq][head_dim]
 *                     (as for mk_decode_step: reads slots 0..positions[b], writes
 *                     slot positions[b])
 *   logits            device fp32 [batch][vocab]
 *   batch, max_ctx    1 <= batch <= cfg->max_batch; positions[b] + 1 <= max_ctx <=
 *                     cfg->max_seq
 *   status_out        device int32 or NULL: receives the step's device status
 *                     (MK_OK, MK_ERR_BAD_TOKEN, MK_ERR_BAD_POSITION)
 *   stream            the CUDA stream the step is enqueued on
 * Scratch (activations, attention partials, the RoPE table, the error word) lives
 * in one 4 MiB device array of the library, per device, held until the process
 * exits. Its layout does not depend on max_ctx: the RoPE table holds a fixed
 * number of positions per head_dim (8192 at 64, 4096 at 128) in a 2 MiB region,
 * the activations follow at a fixed offset. The first call on a device (with that
 * device current) looks up the array's device address, and a call whose
 * rope_theta or head_dim differs from the table in the array uploads a new table
 * from the stack: make those calls before any stream capture (during a capture
 * such a call returns MK_ERR_INVALID_ARG), and do not replay a graph captured
 * before a change of rope_theta or head_dim. Every call shares the array and
 * leaves its contents for the next; the error word is cleared by each call. Calls
 * that overlap on the GPU (on different streams, or from different host threads)
 * race on it.
 * Returns MK_ERR_INVALID_ARG for bad arguments, for max_ctx beyond the RoPE
 * table's positions, and for a step whose activations and attention partials
 * exceed the array's other 2 MiB (more than 32 attention partitions of 320 keys
 * are refused too). */
mk_status mk_baseline_decode_step_noalloc(const mk_config* cfg, const void* packed, const int32_t* tokens,
                                          const int32_t* positions, void* k_cache, void* v_cache, float* logits,
                                          int batch, int max_ctx, int32_t* status_out, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* MK_H */
