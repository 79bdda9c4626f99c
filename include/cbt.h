/*
 * cbt.h -- C ABI of the continuous-batching decode engine (libcbt.so).
 *
 * One GB300, one process.  The library runs a pre-norm decoder transformer
 * (RMSNorm, grouped-query attention with RoPE, SwiGLU FFN) over many live
 * sequences at once:
 *
 *   - cbt_decode_step_batch(seq_ids, last_tokens) -> logits[B]: one token per
 *     live sequence.  Every projection (QKV, O, gate/up, down, lm_head) runs
 *     once over all B rows, so each weight is read from HBM once per step; the
 *     amortisation law on the gnosis page ("The throughput law": sharedCost =
 *     w + L*a against naiveCost = L*(w + a)).  Attention is per sequence: row
 *     s reads its own KV slab over positions [0, t_s], applies RoPE at t_s,
 *     appends its new K/V at t_s and t_s is bumped (gnosis page,
 *     "decode_step_batch -- paint-by-numbers", Delta 1..3).
 *   - cbt_prefill_segmented(seq_ids, seg_lens, tokens): K prompts packed in one
 *     pass; the projections run once over all sum(seg_lens) tokens and
 *     attention is block-diagonal causal, token g of a segment starting at
 *     seg_start attending to [seg_start, g] only (gnosis page, "REVISED: the
 *     hard kernel already exists -- forward_batch_segmented").  Returns the
 *     logits of each segment's last token only (mlx-bun batching design,
 *     section 4.2: slice the last position before the head).
 *   - slabs: one KV slab per live sequence, allocated from a caller-provided
 *     device arena and freed on retire (gnosis page, "1. Native station:
 *     per-sequence KV + a batched decode step": an N-slot KV arena keyed by a
 *     sequence id, prefillSeq / freeSeq).
 *   - greedy sampling: argmax over each row's logits, the lowest vocabulary id
 *     winning ties (mlx-bun batching design, section 4.4 "Vectorized
 *     homogeneous sampling", and its campaign note on tied candidate scores).
 *
 * Conventions for every call:
 *   - Return value: CBT_OK (0) or a negative cbt_status; cbt_status_str()
 *     names it.  Errors the host can see (bad or duplicate slab id, batch
 *     above max_batch, capacity overflow, pool exhausted, null pointers,
 *     sizes out of range) are reported BEFORE any work is queued and leave
 *     the engine unchanged.
 *   - Work is queued asynchronously on the engine's CUDA stream.  Errors only
 *     the device can see (a token id >= vocab) set a device error word that
 *     cbt_last_device_error() reads; the offending row's outputs are then
 *     unspecified, other rows are unaffected, and nothing traps.
 *   - Ownership: the caller owns and frees the weights, the KV arena, token
 *     and logits buffers; the engine borrows them for its lifetime and never
 *     frees them.  The engine owns its scratch memory, which it allocates in
 *     cbt_engine_create and frees in cbt_engine_destroy.
 *   - An engine is not thread safe: one host thread at a time.
 */
#ifndef CBT_H
#define CBT_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef int32_t cbt_status;
#define CBT_OK 0
#define CBT_ERR_INVALID -1        /* a size or config field out of range */
#define CBT_ERR_NULL -2           /* a required pointer is NULL */
#define CBT_ERR_BAD_SLAB -3       /* slab id unknown or already freed */
#define CBT_ERR_DUP_SLAB -4       /* the same slab id twice in one call */
#define CBT_ERR_BATCH -5          /* B > max_batch or K > max_batch */
#define CBT_ERR_CAPACITY -6       /* a slab would grow past its capacity */
#define CBT_ERR_POOL_EXHAUSTED -7 /* no free extent large enough in the KV arena */
#define CBT_ERR_TOKENS -8         /* sum of seg_lens above max_prefill_tokens */
#define CBT_ERR_CUDA -9           /* a CUDA runtime call failed */
#define CBT_ERR_DEVICE -10        /* the device error word was set (see below) */
#define CBT_ERR_UNSUPPORTED -11   /* shape not supported by the kernels */
#define CBT_ERR_LIMIT -12         /* size above the fixed scratch of cbt_greedy_head_noalloc */

/* device error word codes, as returned by cbt_last_device_error in *code */
#define CBT_DEV_OK 0
#define CBT_DEV_TOKEN_RANGE 1 /* a token id outside [0, vocab) */
#define CBT_DEV_TIMEOUT 2     /* a kernel's bounded wait ran out; it stopped early (info: role) */
#define CBT_DEV_WORK_ITEM 3   /* an attention work item its kernel cannot take (info: item) */
#define CBT_DEV_PAGE_ID 4     /* a page id outside the pool (info: the row or token) */
#define CBT_DEV_PAGES 5       /* too few free pages, or a free count out of range (info: missing) */
#define CBT_DEV_LENGTH 6      /* a row's lengths are outside what the call allows (info: the row) */
#define CBT_DEV_TOKENS 7      /* more new tokens than max_tokens (info: max_tokens) */

#define CBT_WEIGHTS_BF16 0    /* bf16, row-major [out][in] */
#define CBT_WEIGHTS_AFFINE4 1 /* 4-bit affine, see cbt_linear */

typedef struct {
  int32_t n_layers;
  int32_t d_model;
  int32_t n_heads;    /* query heads */
  int32_t n_kv_heads; /* key/value heads; q head j reads kv head j / (n_heads / n_kv_heads) */
  int32_t head_dim;   /* must be 64 or 128 */
  int32_t d_ff;       /* SwiGLU hidden size */
  int32_t vocab;
  float rms_eps;
  double rope_theta; /* RoPE rotate-half form, pair (i, i + head_dim/2) turned by
                        pos * rope_theta^(-2i/head_dim) */
  int32_t weight_format; /* CBT_WEIGHTS_BF16 or CBT_WEIGHTS_AFFINE4 */
  int32_t group_size;    /* CBT_WEIGHTS_AFFINE4 only: must be 64 */
} cbt_model_config;

/* One projection W [out][in] (y = x W^T), device pointers.
 * BF16:    w = bf16 [out][in] row-major; scales = biases = NULL.
 * AFFINE4: w = uint32 [out][in/8], element 8j+k of a row in bits 4k..4k+3 of word j;
 *          scales, biases = bf16 [out][in/group]; the weight is scale*q + bias of its
 *          group (MLX-style affine quantisation; cbt_quantize_affine4 produces it). */
typedef struct {
  const void* w;
  const void* scales;
  const void* biases;
} cbt_linear;

typedef struct {
  cbt_linear wqkv;       /* [(n_heads + 2 n_kv_heads) * head_dim][d_model]: q rows, k rows, v rows */
  cbt_linear wo;         /* [d_model][n_heads * head_dim] */
  cbt_linear wgu;        /* [2 d_ff][d_model]: gate rows [0, d_ff), up rows [d_ff, 2 d_ff) */
  cbt_linear wd;         /* [d_model][d_ff] */
  const void* attn_norm; /* bf16 [d_model] RMSNorm gain before attention */
  const void* ffn_norm;  /* bf16 [d_model] RMSNorm gain before the FFN */
} cbt_layer_weights;

typedef struct {
  const void* embed;                /* bf16 [vocab][d_model] (never quantised) */
  cbt_linear lm_head;               /* [vocab][d_model] */
  const void* final_norm;           /* bf16 [d_model] */
  const cbt_layer_weights* layers;  /* host array [n_layers]; copied by cbt_engine_create */
} cbt_weights;

typedef struct {
  void* kv_arena;            /* device memory for all KV slabs, 256-byte aligned, borrowed */
  size_t kv_arena_bytes;
  int32_t max_batch;         /* most rows per decode step and most segments per prefill */
  int32_t max_prefill_tokens;/* most tokens (sum of seg_lens) per prefill call */
  void* stream;              /* cudaStream_t all work is queued on; NULL = legacy default */
  int32_t kv_page_tokens;    /* 0: each slab is one extent of the arena, reserved at
                              * cbt_kv_slab_alloc for its whole capacity.  > 0 (a multiple of
                              * 128): paged KV -- a slab takes pages of this many positions
                              * from the arena as its positions are first written (prefill,
                              * decode, import, copy_prefix), so a slab's capacity is only a
                              * limit and no capacity is held unused; a call that needs a page
                              * the arena cannot give fails with CBT_ERR_POOL_EXHAUSTED before
                              * queuing anything (pages it took are returned).  Page p of a
                              * slab holds positions [p * kv_page_tokens, (p + 1) *
                              * kv_page_tokens) in the layout described at cbt_slab_bytes.
                              * Pages may be shared between slabs (cbt_kv_slab_share_prefix);
                              * a call that writes a position in a shared page first queues a
                              * copy of that page into a new page of the writing slab (copy on
                              * write), and that page counts towards the same pool check. */
  int32_t kv_bits;           /* 0 or 16: bf16 KV.  8 or 4: affine KV of that many bits (the
                              * mlx-bun batching design's quantised KV, "--kv-quant 4|8"): per
                              * position and (layer, K|V, kv head), head_dim codes plus a bf16
                              * scale and bias per 64 dims; a value reads back as scale * code +
                              * bias, with L = 2^kv_bits - 1, scale = bf16((max - min) / L),
                              * bias = bf16(min), code = clamp(rint((x - bias) / scale), 0, L)
                              * over its group of 64 (cbt_quantize_kv).  A segment that starts a
                              * sequence (its slab at position 0) is prefilled in bf16 and then
                              * converted (the design's conversion point), so its prefill logits
                              * equal the bf16 engine's; every later call -- a decode step, or a
                              * prefill segment continuing the slab (a chunked prompt) --
                              * quantises each position it appends before attention reads all
                              * positions through their codes.  Slabs (and pages) take
                              * cbt_slab_bytes_kvq bytes; the engine also holds max_batch *
                              * cbt_slab_bytes(cfg, 128) bytes of the arena for the decode rows'
                              * bf16 staging (CBT_ERR_POOL_EXHAUSTED from cbt_engine_create if it
                              * does not fit).  Needs n_heads / n_kv_heads in {1, 2, 4, 8} and
                              * the tensor-core path (cbt_engine_create returns
                              * CBT_ERR_UNSUPPORTED otherwise); works with paged KV.
                              * cbt_kv_slab_import quantises what it imports; cbt_kv_slab_export
                              * gives each value as bf16(fp32(scale * code + bias)), the product
                              * and sum taken in double; cbt_kv_slab_copy_prefix copies codes,
                              * scales and biases; cbt_kv_slab_share_prefix shares pages.  During
                              * a call, intermediate bf16 slabs of the prompts' (or the import's)
                              * size are taken from the arena and returned. */
} cbt_engine_params;

typedef struct {
  int32_t live_slabs;
  int32_t max_batch;
  int64_t slab_bytes_in_use;  /* bytes of the arena held by live slabs */
  int64_t arena_bytes;
  int64_t largest_free_bytes; /* largest single free extent */
  int64_t scratch_bytes;      /* device scratch the engine allocated */
  int64_t decode_steps;       /* decode steps queued so far */
  int64_t prefill_tokens;     /* prefill tokens queued so far */
} cbt_stats;

typedef struct cbt_engine cbt_engine;

/* Bytes of a quantised KV slab (or page) of capacity cap at kv_bits = bits (8 or 4): per
 * (layer, K|V, kv head) block codes [round64(cap)][head_dim * bits / 8] uint8 (at 4 bits element
 * 2i in the low nibble of byte i, 2i + 1 in its high nibble), then bf16 scales and bf16 biases
 * [round64(cap)][head_dim / 64]; the total rounded up to 4 KiB.  0 if head_dim is not a multiple
 * of 64, cap <= 0 or bits is not 8 or 4.  cbt_slab_bytes_kv8(c, cap) = cbt_slab_bytes_kvq(c,
 * cap, 8). */
size_t cbt_slab_bytes_kvq(const cbt_model_config* c, int32_t cap, int32_t bits);
size_t cbt_slab_bytes_kv8(const cbt_model_config* c, int32_t cap);

/* Affine quantisation of bf16 rows, groups of 64 along each row (the kv_bits = bits format).
 *   x       device bf16 [rows][cols], 4-byte aligned; cols a multiple of 64.
 *   bits    8 or 4.
 *   codes   device uint8 [rows][cols * bits / 8] (2-byte aligned at 8 bits); scales, biases
 *           device bf16 [rows][cols / 64].
 *   stream  cudaStream_t (NULL: legacy default stream); queued, not synchronised.
 * CBT_ERR_NULL, CBT_ERR_INVALID (bits, shape or alignment), CBT_ERR_CUDA.
 * cbt_quantize_kv8 is cbt_quantize_kv with bits = 8. */
cbt_status cbt_quantize_kv(const void* x, int32_t rows, int32_t cols, int32_t bits, void* codes,
                           void* scales, void* biases, void* stream);
cbt_status cbt_quantize_kv8(const void* x, int32_t rows, int32_t cols, void* codes, void* scales,
                            void* biases, void* stream);

const char* cbt_status_str(cbt_status s);

/* Create an engine over the caller's weights and KV arena.  Copies the config, the weight
 * pointer tables and the params; allocates device scratch sized for max_batch rows and
 * max_prefill_tokens tokens.  On failure *out is NULL and nothing is allocated. */
cbt_status cbt_engine_create(const cbt_model_config* cfg, const cbt_weights* weights,
                             const cbt_engine_params* params, cbt_engine** out);

/* Synchronise the engine's stream and free everything the engine allocated. */
cbt_status cbt_engine_destroy(cbt_engine* e);

/* Bytes one slab of `capacity_tokens` positions takes in the arena: the capacity rounded up
 * to a multiple of 64 (C), times n_layers * 2 (K, V) * n_kv_heads * head_dim * 2 bytes,
 * rounded up to 4 KiB.  Slab layout (bf16): [layer][K|V][kv head] blocks of C * head_dim
 * elements; a K block is [position][head_dim]; a V block is [position / 64][head_dim][64]
 * (each group of 64 positions transposed), so both attention contractions read K-major
 * tiles.  Import and export use the plain layout described at cbt_kv_slab_import. */
size_t cbt_slab_bytes(const cbt_model_config* cfg, int32_t capacity_tokens);

/* Reserve a slab for one sequence (host-side first-fit allocator over the arena, no
 * device work).  The slab starts empty (position 0).  The slab id is the sequence id
 * every later call uses. */
cbt_status cbt_kv_slab_alloc(cbt_engine* e, int32_t capacity_tokens, int32_t* slab_id);

/* Return a slab to the arena (host-side bookkeeping only).  Work already queued on the
 * engine stream that uses the slab still runs before any later work on that stream can
 * reuse its extent, so a slab may be freed right after the step that last used it. */
cbt_status cbt_kv_slab_free(cbt_engine* e, int32_t slab_id);

/* retire: free the slabs of finished sequences (EOS or length limit), n ids. */
cbt_status cbt_retire(cbt_engine* e, const int32_t* slab_ids, int32_t n);

/* Current position (tokens held) of a slab. */
cbt_status cbt_kv_slab_position(cbt_engine* e, int32_t slab_id, int32_t* pos);

/* Save/restore a sequence's state.  import copies n_tokens positions of K and V into the
 * slab (positions [0, n_tokens)) and sets its position to n_tokens; export copies
 * positions [0, n_tokens) out.  k and v are bf16 [n_layers][n_kv_heads][n_tokens][head_dim],
 * on the host (on_host != 0) or on the device.  Queued on the engine stream. */
cbt_status cbt_kv_slab_import(cbt_engine* e, int32_t slab_id, const void* k, const void* v,
                              int32_t n_tokens, int32_t on_host);
cbt_status cbt_kv_slab_export(cbt_engine* e, int32_t slab_id, void* k, void* v,
                              int32_t n_tokens, int32_t on_host);

/* Prefix reuse: copy positions [0, n_tokens) of slab src_id's K and V into slab dst_id and set
 * dst's position to n_tokens, so a prefill of dst continues after a prefix that was computed
 * once (the mlx-bun batching design, sections 1 and 4.2: sub-agents share long system
 * prompts; a joiner's prefill starts from the longest cached prefix, so N agents sharing a
 * prompt reuse one prefill).  Here the reuse is a device-to-device copy of the prefix's bytes
 * (n_tokens x 2 x n_layers x n_kv_heads x head_dim bf16), queued on the engine stream; the
 * slabs stay independent afterwards.
 *   src_id, dst_id  distinct live slabs; n_tokens <= src's position and <= dst's capacity.
 * Errors (nothing queued, nothing changed): CBT_ERR_BAD_SLAB, CBT_ERR_INVALID (same slab or
 * n_tokens < 0), CBT_ERR_CAPACITY, CBT_ERR_CUDA. */
cbt_status cbt_kv_slab_copy_prefix(cbt_engine* e, int32_t src_id, int32_t dst_id,
                                   int32_t n_tokens);

/* Prefix sharing (the same pages, the mlx-bun batching design, sections 1 and 4.2): slab dst_id
 * takes positions [0, n_tokens) of slab src_id without a copy and its position becomes n_tokens.
 * On a paged engine dst holds src's first ceil(n_tokens / kv_page_tokens) pages by reference
 * (no device work, no arena bytes); the first later write into a shared page by either slab
 * (prefill, decode, import, copy_prefix into it) copies that one page first, so neither slab
 * ever sees the other's later positions, and a page returns to the arena when its last holder
 * frees it.  On a contiguous engine there are no pages to share and the call is
 * cbt_kv_slab_copy_prefix.
 *   src_id, dst_id  distinct live slabs; dst at position 0 (pages it holds are released);
 *                   n_tokens <= src's position and <= dst's capacity.
 * Errors (nothing queued, nothing changed): CBT_ERR_BAD_SLAB, CBT_ERR_INVALID (same slab,
 * n_tokens < 0 or dst's position not 0), CBT_ERR_CAPACITY, and on a contiguous engine those of
 * cbt_kv_slab_copy_prefix. */
cbt_status cbt_kv_slab_share_prefix(cbt_engine* e, int32_t src_id, int32_t dst_id,
                                    int32_t n_tokens);

/* Segmented prefill of K prompts (forward_batch_segmented).
 *   slab_ids  host int32 [K], distinct live slabs.  Segment s's tokens go to positions
 *             [p_s, p_s + seg_lens[s]) of its slab, p_s being the slab's current position
 *             (0 for a fresh slab: positions are segment-local from 0); each token attends
 *             to positions [0, its own] of its own slab only.
 *   seg_lens  host int32 [K], each >= 1, sum <= max_prefill_tokens, p_s + seg_lens[s] <=
 *             capacity.
 *   tokens    device int32 [sum seg_lens], the segments back to back.
 *   logits    device float [K][vocab]: logits of each segment's last token; NULL allowed.
 *   next_tokens device int32 [K]: greedy argmax of those logits; NULL allowed.
 * Afterwards each slab's position is p_s + seg_lens[s]. */
cbt_status cbt_prefill_segmented(cbt_engine* e, const int32_t* slab_ids, const int32_t* seg_lens,
                                 int32_t K, const int32_t* tokens, float* logits,
                                 int32_t* next_tokens);

/* One continuous-batching decode step (decode_step_batch).
 *   slab_ids    host int32 [B], distinct live slabs; row b is the sequence of slab_ids[b].
 *   last_tokens device int32 [B]: the token each row feeds (may be the previous step's
 *               next_tokens buffer, so greedy decode needs no host round trip).
 *   logits      device float [B][vocab] or NULL.
 *   next_tokens device int32 [B] or NULL: greedy argmax of each row, lowest id on ties.
 * Row b's token is placed at position t_b (the slab's current position, which must be
 * below its capacity), attends to [0, t_b] of its own slab, and t_b becomes t_b + 1.
 * B == 0 is a no-op. */
cbt_status cbt_decode_step_batch(cbt_engine* e, const int32_t* slab_ids, int32_t B,
                                 const int32_t* last_tokens, float* logits, int32_t* next_tokens);

/* Synchronise the engine's stream, then read and clear the device error word.
 * *code = CBT_DEV_OK or a CBT_DEV_* code, *info = the offending row or token index.
 * Returns CBT_OK, or CBT_ERR_CUDA if the stream reported an error. */
cbt_status cbt_last_device_error(cbt_engine* e, int32_t* code, int32_t* info);

cbt_status cbt_engine_stats(cbt_engine* e, cbt_stats* out);

/* Number of kernel launches the library queued so far, all engines together (for launch
 * accounting; e may be NULL). */
int64_t cbt_kernel_launches(cbt_engine* e);

/* Measurement.  Kernel classes: */
#define CBT_KCLASS_PROJ 0  /* projections QKV, O, gate/up (+SwiGLU), down, lm_head: weight streaming */
#define CBT_KCLASS_ATTN 1  /* RoPE + KV append and attention over the slabs */
#define CBT_KCLASS_OTHER 2 /* embedding, norms, RoPE tables, argmax, gathers */
#define CBT_NUM_KCLASSES 3

/* Bracket every launch group of the classes in class_mask (bit k = class k) with CUDA
 * events on the engine stream, from now on; 0 turns it off.  Clears earlier records.
 * Events only mark the stream between kernels; they change no result. */
cbt_status cbt_engine_set_timing(cbt_engine* e, int32_t class_mask);

/* Synchronise the stream and sum the records of one class since cbt_engine_set_timing:
 * total device milliseconds, number of bracketed intervals, and the algorithmic bytes those
 * intervals moved (each weight once, activations in and out, each live KV position once). */
cbt_status cbt_engine_timing(cbt_engine* e, int32_t kclass, double* total_ms, int64_t* intervals,
                             double* algorithmic_bytes);

/* Failure-detection test of the bounded device waits.  Every wait in the library's kernels
 * (on an mbarrier, a cluster peer or a flag) gives up after a bounded number of polls, records
 * CBT_DEV_TIMEOUT in the device error word (info: the role that gave up) and lets its kernel
 * end; nothing traps or hangs.  This call arms the next cbt_decode_step_batch of the engine so
 * that its lm_head projection requests none of its weight tiles and every wait of that launch
 * runs out after spin_limit polls.  That step then reports CBT_DEV_TIMEOUT through
 * cbt_last_device_error; its logits and next tokens are unspecified, everything else it does
 * (the K/V it appends, the positions it bumps) is as in a normal step, and later steps are
 * unaffected.  Bf16 weights on the tensor-core path only (else CBT_ERR_UNSUPPORTED);
 * spin_limit > 0 (else CBT_ERR_INVALID). */
cbt_status cbt_engine_test_stall(cbt_engine* e, int32_t spin_limit);

/* In-step stamps (measurement).  With enable != 0, every later decode step -- replayed steps
 * included -- records for each of its projection and attention launches (CBT_KCLASS_PROJ,
 * CBT_KCLASS_ATTN) the earliest time one of the launch's CTAs could start work that depends on
 * the previous kernel and the latest time one of them ended, in globaltimer nanoseconds.  The
 * stamps change no result.  cbt_engine_stamps synchronises the stream and copies the records of
 * the last decode step: *n = their number; for i < min(cap, *n) classes[i] = the launch's class,
 * times[2i] = begin, times[2i + 1] = end.  (A step's launches overlap through programmatic
 * dependent launch; the union of a class's intervals is its share of the step.) */
cbt_status cbt_engine_set_stamps(cbt_engine* e, int32_t enable);
cbt_status cbt_engine_stamps(cbt_engine* e, int32_t cap, int32_t* n, int32_t* classes,
                             uint64_t* times);

/* MLX-style 4-bit affine quantisation of a bf16 matrix on the device, groups of `group`
 * (64) along each row: scale = bf16((max - min) / 15), bias = bf16(min),
 * q = clamp(rint((w - bias) / scale), 0, 15) (ties to even; 0 when scale == 0), packed
 * as in cbt_linear.  w: device bf16 [rows][cols]; packed: device uint32 [rows][cols/8];
 * scales, biases: device bf16 [rows][cols/group].  cols % group == 0.  Queued on `stream`. */
cbt_status cbt_quantize_affine4(const void* w, int32_t rows, int32_t cols, int32_t group,
                                void* packed, void* scales, void* biases, void* stream);

/* ---- Operators on a caller-owned paged KV cache ------------------------------------------
 * The parts of a step that deal with the KV cache, for callers that run a model of their own on
 * caller-owned buffers: request lengths to block tables and slots (cbt_page_map), per-head
 * norms, rotary positions and the append of K and V (cbt_rope_append), and attention over the
 * pages (cbt_paged_attention).  Lengths, tables and the free stack live on the device and no
 * call reads them on the host, so a whole step can be captured in a CUDA graph and replayed
 * while sequences grow, join and retire.  An engine's own steps take the same rotary forms, norms,
 * window and sinks through cbt_engine_set_attention, which runs these operators.
 *
 * Conventions, besides those at the top of this file: all pointers are device pointers of the
 * current device except the descriptor structs, which are read during the call only; work is
 * queued on `stream` (cudaStream_t; NULL = legacy default) and nothing is allocated or
 * synchronised.  `err` is a device int32 [2] the caller set to zero: the first error a kernel
 * finds is left there as (CBT_DEV_* code, info) and stays until the caller clears it.  A call
 * with nothing to do (rows or tokens 0) returns CBT_OK and queues nothing. */

/* One layer's K and V in a pool of n_pages pages, page i at pool + i * page_bytes.  In a page, K
 * starts at k_offset and V at v_offset bytes, each n_kv_heads blocks of page_tokens * head_dim
 * bf16 in the layout of cbt_slab_bytes: K [position][head_dim], V [position / 64][head_dim][64].
 * A pool whose pages are cbt_slab_bytes(cfg, page_tokens) bytes with k_offset = 2 * layer * n,
 * v_offset = k_offset + n (n = n_kv_heads * page_tokens * head_dim * 2) is laid out as an
 * engine's pages are.  pool, page_bytes and the offsets are multiples of 256 bytes; page_tokens
 * is a multiple of 64; head_dim is 64 or 128; n_pages * page_tokens < 2^31 and pool_bytes <
 * 128 * 2^31 (CBT_ERR_LIMIT); the last page's blocks end within pool_bytes. */
typedef struct {
  void* pool;
  size_t pool_bytes;
  int64_t page_bytes;
  int64_t k_offset, v_offset;
  int32_t n_pages, page_tokens, n_kv_heads, head_dim;
} cbt_paged_kv;

/* Block tables and slot maps from request lengths: one step's page bookkeeping on the device.
 * Row b holds kv_lens[b] positions in pages block_table[b][0 .. ceil(kv_lens[b] / page_tokens)).
 *   new_lens[b] > 0   the row grows by that many positions, taking the pages it lacks;
 *   new_lens[b] == 0  the row stays as it is;
 *   new_lens[b] < 0   the row retires: its pages return to the free stack, its length becomes 0.
 * The free stack is free_pages[0 .. free_count[0]).  Retiring rows push their pages first, in
 * row and then position order; growing rows then pop theirs from its top in the same order.
 *   block_table  int32 [rows][max_pages]; entries taken are written, all others are left as
 *                they are (a retired row's entries too).
 *   free_pages   int32 [n_pages], or NULL: no page is taken or returned, growing rows find
 *                every page in their table already (free_count and free_count_out are unused).
 *   kv_lens_out, free_count_out  the lengths and the count afterwards; may be kv_lens and
 *                free_count themselves.
 *   cu_q         int32 [rows + 1]: exclusive prefix sums of the new tokens (row b's tokens are
 *                [cu_q[b], cu_q[b + 1])).
 *   positions, slots  int32 [max_tokens]: each new token's position in its row, and page id *
 *                page_tokens + position % page_tokens.  Both are -1 past the last token; a slot
 *                is -1 where its page id is outside [0, n_pages) (CBT_DEV_PAGE_ID, info: row).
 * All or nothing: if a row's length is negative or would pass max_pages * page_tokens
 * (CBT_DEV_LENGTH), the tokens pass max_tokens (CBT_DEV_TOKENS), the stack is short or its count
 * out of range (CBT_DEV_PAGES), or a page id that a retiring row returns is outside [0, n_pages)
 * (CBT_DEV_PAGE_ID, info: the row), then the lengths, count, table and stack stay as they were
 * (what free_pages holds from the count on is never specified), cu_q is all zero and positions and
 * slots are all -1, so the calls that follow find no tokens.
 * With rows 0 nothing is written, cu_q, positions and slots among it.
 * Output arrays may not overlap anything else the call reads, but for the two named pairs.
 * rows <= CBT_PAGE_MAP_MAX_ROWS, max_tokens and n_pages <= 2^30, max_pages * page_tokens < 2^31
 * and n_pages * page_tokens < 2^31 (CBT_ERR_LIMIT).  Other errors: CBT_ERR_NULL, CBT_ERR_INVALID,
 * CBT_ERR_CUDA. */
#define CBT_PAGE_MAP_MAX_ROWS 4096
typedef struct {
  int32_t* block_table;
  int32_t max_pages, page_tokens, n_pages, rows;
  const int32_t* kv_lens;
  const int32_t* new_lens;
  int32_t* free_pages;
  const int32_t* free_count;
  int32_t max_tokens;
  int32_t* kv_lens_out;
  int32_t* free_count_out;
  int32_t* cu_q;
  int32_t* positions;
  int32_t* slots;
  int32_t* err;
} cbt_page_map_args;
cbt_status cbt_page_map(const cbt_page_map_args* a, void* stream);

/* Rotary position embedding.  Pair i < rot_dim / 2 of a head is (x[i], x[i + rot_dim / 2])
 * (CBT_ROPE_HALF) or (x[2 i], x[2 i + 1]) (CBT_ROPE_INTERLEAVED), turned by position * f_i and
 * multiplied by mscale; dims from rot_dim on pass through.  With u_i = theta^(-2 i / rot_dim)
 * and s = factor:
 *   CBT_ROPE_NONE      f_i = u_i
 *   CBT_ROPE_LINEAR    f_i = u_i / s (positions interpolated)
 *   CBT_ROPE_BASE      f_i = u_i with theta * s^(rot_dim / (rot_dim - 2)) for theta
 *   CBT_ROPE_BY_PARTS  f_i = u_i (1 - r_i) + u_i / s r_i, r_i = clamp((i - lo) / (hi - lo), 0, 1),
 *                      lo = max(0, floor(c(beta_fast))), hi = min(rot_dim - 1, ceil(c(beta_slow))),
 *                      c(n) = rot_dim ln(original_len / (2 pi n)) / (2 ln theta), hi taken as
 *                      lo + 0.001 where it is not above lo: pairs that turn often over
 *                      original_len positions keep their frequency, slow ones are interpolated
 *                      (the published "YaRN" rule)
 * mscale 0 stands for the form's own: 0.1 ln s + 1 by parts (s > 1), else 1.
 * rot_dim is even, 2 <= rot_dim <= head_dim; theta > 1; factor >= 1; by parts also original_len >
 * 0 and beta_fast > beta_slow > 0 (0, 0: 32 and 1).  CBT_ERR_INVALID otherwise. */
#define CBT_ROPE_HALF 0
#define CBT_ROPE_INTERLEAVED 1
#define CBT_ROPE_NONE 0
#define CBT_ROPE_LINEAR 1
#define CBT_ROPE_BASE 2
#define CBT_ROPE_BY_PARTS 3
typedef struct {
  int32_t layout, rot_dim, scaling, original_len;
  double theta, factor, beta_fast, beta_slow, mscale;
} cbt_rope_config;

/* The frequencies a kernel turns by, filled on the host by cbt_rope_init: turns[i] = f_i / (2 pi)
 * as a fraction of a turn in 64-bit fixed point, so position * turns[i] modulo 2^64 is the angle
 * at any position without its whole turns. */
typedef struct {
  uint64_t turns[64];
  float mscale;
  int32_t layout, rot_dim, head_dim;
} cbt_rope;
cbt_status cbt_rope_init(const cbt_rope_config* c, int32_t head_dim, cbt_rope* out);

/* Element types of the rows below */
#define CBT_DTYPE_BF16 0
#define CBT_DTYPE_F32 1

/* Per-head norms, rotary positions and the KV append in one pass over QKV rows.  Token t's row
 * holds n_heads q heads, n_kv_heads k heads and n_kv_heads v heads of head_dim.  Every q and k
 * head is normalised (x / sqrt(mean(x^2) + eps) * gain, where a gain is given), then turned by
 * positions[t]; q goes to q_out in bf16, k and v in bf16 to slot slots[t] of the cache.
 *   qkv        bf16 or fp32 (qkv_dtype) [tokens], rows qkv_stride elements apart
 *   q_gain, k_gain  bf16 [head_dim] or NULL (that norm is left out)
 *   positions  int32 [tokens], >= 0 where the slot is
 *   slots      int32 [tokens]; a token whose slot or position is negative is skipped: its q_out
 *              row and the cache stay as they are.  A slot of n_pages * page_tokens or more is
 *              skipped too (CBT_DEV_PAGE_ID, info: token).  Where two tokens have one slot, each
 *              element of K and V there is one or the other's, unspecified which.
 *   q_out      bf16 [tokens][n_heads * head_dim], rows q_stride elements apart; no overlap with qkv
 * rope == NULL: no rotation.  Arithmetic is fp32 with one rounding to bf16 at the end.  qkv, q_out
 * and the gains are 16-byte aligned, the strides multiples of 8 elements.  Errors: CBT_ERR_NULL,
 * CBT_ERR_INVALID, CBT_ERR_UNSUPPORTED (head_dim), CBT_ERR_LIMIT (tokens above 2^30, n_heads + 2
 * n_kv_heads above 65535), CBT_ERR_CUDA. */
typedef struct {
  cbt_paged_kv kv;
  const cbt_rope* rope;
  const void* qkv;
  int32_t qkv_dtype;
  int64_t qkv_stride;
  int32_t tokens, n_heads;
  const void* q_gain;
  const void* k_gain;
  float eps;
  const int32_t* positions;
  const int32_t* slots;
  void* q_out;
  int64_t q_stride;
  int32_t* err;
} cbt_rope_append_args;
cbt_status cbt_rope_append(const cbt_rope_append_args* a, void* stream);

/* Attention over pages.  Row b has kv_lens[b] positions in the cache, the last n_b of them being
 * its query tokens [cu_q[b], cu_q[b + 1]) (cu_q NULL: token b alone, tokens == rows).  The query at
 * position p attends to positions j <= p with j > p - window or j < sinks (window 0: all j <= p):
 *   out = sum_j softmax_j(scale * q . k_j) v_j, q head h reading kv head h / (n_heads / n_kv_heads).
 * A query that sees nothing (its row holds fewer positions than query tokens) gets zeros; out rows
 * past cu_q[rows] are left as they are.  What positions hold that no query token of the row sees,
 * NaN and infinities among it, changes nothing.  (V that is not finite where one query token of a
 * row sees it may reach the row's other query tokens: their weight of it is 0, and 0 * NaN is NaN.)
 *   block_table  int32 [rows][max_pages]
 *   max_q, max_kv  upper bounds of n_b and kv_lens[b] that the caller vouches for: they size the
 *                launch and the workspace, and with max_q > 1 they decide whether rows are cut into
 *                runs (bounds far above the rows cost time, not results).  A row above either, or
 *                with more positions than its table, reports CBT_DEV_LENGTH; its outputs are
 *                unspecified.  So are those of a row with a page id outside the pool among the pages
 *                it reads (CBT_DEV_PAGE_ID).
 *   tokens       rows of q and out; a row whose cu_q range leaves [0, tokens] or runs backwards is
 *                skipped (CBT_DEV_LENGTH).  Where the ranges of other rows overlap (which takes one
 *                that runs backwards), the call's outputs are unspecified.
 *   q            bf16 [tokens][n_heads * head_dim], rows q_stride elements apart
 *   out          bf16 or fp32 (out_dtype), rows out_stride elements apart; no overlap with q
 *   workspace    cbt_paged_attention_workspace bytes, 256-byte aligned (NULL if that is 0).  Calls
 *                that overlap on the GPU, graph replays among them, need workspaces of their own.
 * scale is finite; window and sinks are >= 0 (sinks without a window change nothing).  Scores,
 * softmax sums and outputs are accumulated in fp32, in an order that the sizes fix: the same call
 * gives the same bits again.  The weights that multiply V have two bf16 parts (2^-16 relative) with
 * max_q == 1, and are rounded to bf16 once (2^-8) with more, rows of one token among them.
 * What the other rows hold never changes a row's result.  With max_q == 1 neither does how many there
 * are; with more, rows, max_q and max_kv decide whether long rows are summed in several runs, so
 * calls of different sizes may differ in the last bits.
 * n_heads / n_kv_heads <= 64, q and out 16-byte aligned, strides multiples of 8
 * elements, kv.head_dim 64 or 128 (CBT_ERR_UNSUPPORTED); rows <= CBT_PAGED_ATTENTION_MAX_ROWS,
 * max_kv + window and max_kv + sinks < 2^31, (rows + tokens) * n_heads < 2^29 and with max_q == 1
 * (rows + tokens) * n_heads * (max_kv / 128 + 2) < 2^31 (CBT_ERR_LIMIT).  Other errors:
 * CBT_ERR_NULL, CBT_ERR_INVALID (a workspace that is too small among it), CBT_ERR_CUDA. */
#define CBT_PAGED_ATTENTION_MAX_ROWS 4096
typedef struct {
  cbt_paged_kv kv;
  const int32_t* block_table;
  int32_t max_pages, rows;
  const int32_t* kv_lens;
  const int32_t* cu_q;
  int32_t tokens, max_q, max_kv, n_heads;
  const void* q;
  int64_t q_stride;
  float scale;
  int32_t window, sinks;
  void* out;
  int32_t out_dtype;
  int64_t out_stride;
  void* workspace;
  size_t workspace_bytes;
  int32_t* err;
} cbt_paged_attention_args;
cbt_status cbt_paged_attention(const cbt_paged_attention_args* a, void* stream);
/* Bytes of workspace the call described by a's sizes needs (pointers are not looked at); 0 where
 * it needs none or the sizes are not supported. */
size_t cbt_paged_attention_workspace(const cbt_paged_attention_args* a);

/* ---- The same operators on a cache in 8 bits ----------------------------------------------
 * cbt_rope_append_fp8, cbt_paged_attention_fp8 and cbt_paged_read_fp8 work on pages that hold K and V
 * as 8-bit floats (e4m3: four bits of exponent, three of mantissa, largest 448) with a scale for every
 * block of 64 positions of a kv head, K and V apart: half the bytes of a bf16 cache.  What such a cache
 * holds is off from what was appended by at most 2^-4 of each value, or 2^-10 of the block's scale where
 * that is more; where the scale has grown since, by at most 2^-4 of the value and 2^-9 of the scale
 * together.  (Values past 448 * 2^56 and infinities aside.)  Tables, slots and lengths are as for bf16 pages
 * (cbt_page_map serves both).
 *
 * A scale is a power of two, 2^e with e in [-56, 56]: the smallest that all of the block's values are
 * within 448 times of.  The steps of an 8-bit float are relative, so a finer scale would gain nothing,
 * and a block whose scale has to grow under later tokens is moved to the new one without another
 * rounding, but for codes below 2^-6.
 *
 * One layer in a pool of n_pages pages, page i at pool + i * page_bytes.  In a page, the codes of K
 * start at k_offset and those of V at v_offset bytes, each n_kv_heads blocks of page_tokens *
 * head_dim: K [position][head_dim], V [position / 64][head_dim][64].  The scales start at s_offset
 * bytes: fp32 [2 (K, V)][n_kv_heads][page_tokens / 64]; one that is not such a power of two is taken as
 * the one below it, and those out of range as the nearest in it.  pool, page_bytes and the offsets are
 * multiples of 256 bytes; page_tokens is a multiple of 64; head_dim is 64 or 128; n_pages * page_tokens
 * < 2^31 and pool_bytes < 256 * 2^31 (CBT_ERR_LIMIT); the last page's codes and scales end within
 * pool_bytes. */
#define CBT_FP8_BLOCK 64
typedef struct {
  void* pool;
  size_t pool_bytes;
  int64_t page_bytes;
  int64_t k_offset, v_offset, s_offset;
  int32_t n_pages, page_tokens, n_kv_heads, head_dim;
} cbt_paged_kv_fp8;

/* cbt_rope_append with K and V rounded to codes.  The norms, the rotation and q_out are those of
 * cbt_rope_append; k (rotated, in fp32) and v then go to slot slots[t] as codes.  For each block that
 * the call's tokens lie in, kv head, and K and V apart:
 *   - where a token lies in the block's first position (slot % 64 == 0) the block starts anew, and what
 *     its other positions held is lost; else it goes on from the scale that it has;
 *   - the scale becomes the largest of that and what the call's tokens need (their values that are
 *     finite); where it grows, the codes held there are rounded to the new one;
 *   - the tokens are rounded to it once, to nearest even.  An infinity becomes 448 times the scale, as
 *     does a value above 448 * 2^56; a NaN stays one.
 * k is formed in fp32, and to 2^-28 of the pair that is rotated where it lies beside the middle between two
 * codes, so that nearly every code is the one of k in full.
 * A block that is gone on with has to hold a scale: pages are taken from position 0 on, or zeroed first.
 * The tokens of one block stand next to each other in the call (as cbt_page_map deals them; tokens that
 * are skipped do not stand between them): where they do not, what the block then holds is unspecified.
 * Where two tokens have one slot, each element there is one or the other's.  Everything else is as in
 * cbt_rope_append, errors among it. */
typedef struct {
  cbt_paged_kv_fp8 kv;
  const cbt_rope* rope;
  const void* qkv;
  int32_t qkv_dtype;
  int64_t qkv_stride;
  int32_t tokens, n_heads;
  const void* q_gain;
  const void* k_gain;
  float eps;
  const int32_t* positions;
  const int32_t* slots;
  void* q_out;
  int64_t q_stride;
  int32_t* err;
} cbt_rope_append_fp8_args;
cbt_status cbt_rope_append_fp8(const cbt_rope_append_fp8_args* a, void* stream);

/* Reads positions back: row b's [first[b], first[b] + n_b), n_b = cu[b + 1] - cu[b], go to rows
 * [cu[b], cu[b + 1]) of k_out and v_out as code * scale (exact in either type).
 *   block_table, kv_lens  as in cbt_paged_attention; the positions lie within [0, kv_lens[b])
 *   first        int32 [rows], or NULL: 0
 *   cu           int32 [rows + 1]
 *   tokens       rows of k_out and v_out; those past cu[rows] are left as they are
 *   k_out, v_out bf16 or fp32 (out_dtype) [tokens][n_kv_heads * head_dim], rows out_stride elements
 *                apart; either may be NULL
 * A row whose positions leave the row or its table is skipped (CBT_DEV_LENGTH, info: the row); positions
 * in a page outside the pool are left as they were (CBT_DEV_PAGE_ID).  Where a row's range of cu leaves
 * [0, tokens] or runs backwards (CBT_DEV_LENGTH), the call's outputs are unspecified.  k_out and v_out
 * are 16-byte aligned, the stride a multiple of 8; rows <= CBT_PAGED_ATTENTION_MAX_ROWS, tokens <= 2^30
 * (CBT_ERR_LIMIT).  Other errors: CBT_ERR_NULL, CBT_ERR_INVALID, CBT_ERR_UNSUPPORTED, CBT_ERR_CUDA. */
typedef struct {
  cbt_paged_kv_fp8 kv;
  const int32_t* block_table;
  int32_t max_pages, rows;
  const int32_t* kv_lens;
  const int32_t* first;
  const int32_t* cu;
  int32_t tokens;
  void* k_out;
  void* v_out;
  int32_t out_dtype;
  int64_t out_stride;
  int32_t* err;
} cbt_paged_read_fp8_args;
cbt_status cbt_paged_read_fp8(const cbt_paged_read_fp8_args* a, void* stream);

/* cbt_paged_attention over codes: k_j and v_j are code * scale of position j.  Everything else is as there,
 * but for the roundings on the way:
 *   - q takes part to 2^-18 of the largest element of its head, or as bf16 holds it where that is finer;
 *     a head of q with an element that is not finite gets NaN;
 *   - the weights that multiply V are rounded to fp16 once: 2^-11 of each, and at most 2^-20 of the row's largest
 *     weight and, with V's scale in both, 2^-20 of the row's largest product of weight and scale, whichever is
 *     less.  (max_q > 1: where V's scales lie further apart than 2^64, 2^-84 of that product if that is more.) */
typedef struct {
  cbt_paged_kv_fp8 kv;
  const int32_t* block_table;
  int32_t max_pages, rows;
  const int32_t* kv_lens;
  const int32_t* cu_q;
  int32_t tokens, max_q, max_kv, n_heads;
  const void* q;
  int64_t q_stride;
  float scale;
  int32_t window, sinks;
  void* out;
  int32_t out_dtype;
  int64_t out_stride;
  void* workspace;
  size_t workspace_bytes;
  int32_t* err;
} cbt_paged_attention_fp8_args;
cbt_status cbt_paged_attention_fp8(const cbt_paged_attention_fp8_args* a, void* stream);
/* as cbt_paged_attention_workspace; the same sizes may need other bytes */
size_t cbt_paged_attention_fp8_workspace(const cbt_paged_attention_fp8_args* a);

/* The attention form of an engine's layers.  From now on every prefill and decode step of the
 * engine normalises q and k per head, rotates them, appends K and V and attends as cbt_rope_append
 * and cbt_paged_attention do, over the engine's own pages; NULL returns it to its built-in form
 * (no norms, half rotation of the whole head by rope_theta, all earlier positions seen).
 *   rope    rotary form (copied); NULL: the built-in one
 *   q_norm, k_norm  host arrays [n_layers] of device bf16 [head_dim] gains (the array is copied,
 *           the gains are borrowed), or NULL: that norm is left out
 *   window, sinks  as in cbt_paged_attention, any size: where either reaches the positions that all
 *           of the arena's pages hold, every earlier position is seen
 * q is rounded to bf16 for the attention, and in a prefill (of more than a token a prompt) the
 * softmax's weights too; the built-in form carries two parts of both.  Pages behind the window stay
 * held.  Of such an engine cbt_engine_stamps records the projections alone.
 * The calls' page table and the attention's partial sums grow inside the call that needs more, which
 * waits for the stream; cbt_stats.scratch_bytes counts them.  The table takes 4 bytes for each page of
 * the longest row, max_batch times; the sums of a decode step of B rows 4 * B * n_heads * head_dim bytes
 * for every 512 positions of the longest row (every 128 below 4096), those of a prefill at most 84 MB.
 * Where no memory is left the call returns CBT_ERR_CUDA and queues no step, and calls that fit
 * what is there go on.
 * Only before slabs exist (CBT_ERR_INVALID otherwise); a form that replaces one waits for the stream,
 * and the gains of before are the caller's again.  Needs a paged engine (kv_page_tokens > 0) with bf16
 * KV on the tensor-core path, max_batch <= CBT_PAGED_ATTENTION_MAX_ROWS and n_heads / n_kv_heads <= 64
 * (CBT_ERR_UNSUPPORTED).  Errors leave the engine's form as it was. */
typedef struct {
  const cbt_rope_config* rope;
  const void* const* q_norm;
  const void* const* k_norm;
  float qk_norm_eps;
  int32_t window, sinks;
} cbt_attention_config;
cbt_status cbt_engine_set_attention(cbt_engine* e, const cbt_attention_config* c);

/* ---- Greedy head without any allocation --------------------------------------------------
 * The pages have no counterpart to this call; it exists for callers that cannot allocate
 * device memory: code running where cudaMalloc is forbidden or unsafe (inside another
 * framework's memory pool or allocator hooks, a real-time loop that must not block on the
 * allocator, an embedding runtime that hands over pre-planned buffers only).  It runs the
 * last stage of a decode step on hidden states the caller already has:
 *   logits[r] = RMSNorm(hidden[r], final_norm, cfg->rms_eps) lm_head^T,
 *   next_tokens[r] = argmax(logits[r]) (lowest id on ties),
 * the operations decode_step_batch ends with, computed by the library's CUDA-core kernels
 * (an RMSNorm kernel, a split-K projection whose partial sums are added in a fixed order,
 * the argmax kernel) rather than the tensor-core projection of a decode step, so its logits
 * agree with decode_step_batch's within rounding, not bit for bit.  Its scratch (the
 * normalised rows and the split-K partial sums) lives in one fixed array in the library's
 * device memory, CBT_NOALLOC_SCRATCH_BYTES large.  Every GPU that loads the library holds
 * that array until the process exits.
 *   cfg          model config (d_model, vocab, rms_eps, weight_format, group_size are used)
 *   hidden       device float [n][d_model], the residual stream after the last layer
 *   n            rows, 0 <= n <= CBT_NOALLOC_MAX_ROWS (0 is a no-op)
 *   final_norm   device bf16 [d_model]
 *   lm_head      projection [vocab][d_model] as in cbt_linear (device pointers)
 *   logits       device float [n][vocab], written
 *   next_tokens  device int32 [n], written; may be NULL
 *   stream       cudaStream_t to queue on (NULL = legacy default stream)
 * Returns CBT_ERR_CUDA if one of its own launches fails (an error left by earlier, unrelated
 * work is neither reported nor cleared), and CBT_ERR_LIMIT, before queuing anything, when
 * n > CBT_NOALLOC_MAX_ROWS or when
 * n*d_model + (d_model/slice)*n*vocab floats (slice = 1024, 512 or 256, the largest that
 * divides d_model) exceed the fixed scratch.  It calls no cudaMalloc, cudaFree or any
 * allocating library routine.  The first call on each device looks up the array's device
 * address (cudaGetSymbolAddress, with that device current); make that first call before
 * any stream capture.  All calls share the one array and it keeps the last call's
 * contents, so calls that overlap on the GPU (different streams, or threads) race: queue
 * them on one stream, or order them with events. */
#define CBT_NOALLOC_MAX_ROWS 32
#define CBT_NOALLOC_SCRATCH_BYTES (20u << 20)
cbt_status cbt_greedy_head_noalloc(const cbt_model_config* cfg, const float* hidden, int32_t n,
                                   const void* final_norm, const cbt_linear* lm_head,
                                   float* logits, int32_t* next_tokens, void* stream);

#ifdef __cplusplus
}
#endif
#endif
