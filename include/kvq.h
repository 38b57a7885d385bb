/*
 * kvq.h -- decode attention over a quantized, paged KV cache (GB300, sm_103a).
 *
 * A C ABI: plain structs, pointers and sizes.  Every device pointer is caller
 * owned; the library never allocates, frees, or synchronizes the stream it is
 * given (kvq_get_device_error is the one call that waits, and says so).  All
 * compute calls are asynchronous on `stream` and take their grid and workspace
 * extents from host-side shapes only, so a sequence of calls can be captured
 * in a CUDA graph.
 *
 * The operations follow these pages:
 *  - onnxruntime issue #29783 (quantized KV cache in GroupQueryAttention):
 *    per-token scales, quantize the appended token on write, dequantize on
 *    read, no fp16 copy of the past.
 *  - onnxruntime PR #29912 "[CUDA] PagedAttention: quantized KV cache, XQA
 *    decode, MLA, QK-Norm and head sink", Summary of Changes: slot_mapping,
 *    head_sink, k_scale / v_scale with PER_TENSOR / PER_CHANNEL granularity,
 *    int8 / float8e4m3fn cache types, ReshapeAndCache (quantize on write),
 *    split-KV paged decode with softcap and sliding window, ApplyHeadSink, and
 *    the attention_metadata upper bound that keeps a step capturable.
 *  - onnxruntime PR #32515 "[CUDA] Add INT4 paged KV cache with per-channel
 *    scales", Description: int4 packed two per byte, cache head dimension
 *    (head_size+1)/2, per-channel scale folded into Q and re-applied to the
 *    output, speculative decode with several query tokens.
 *  - "kv-quant-attn" page, sections "Method" and "Correctness": per-row absmax
 *    scales, one block per (batch, kv head) resolving the whole GQA group from
 *    one read, warp-private softmax state, fixed-order merge (bitwise
 *    reproducible), GQA ratio at most 8, head dimension at most 256; section
 *    "Requirements and limits": the group-wise scaling it leaves undone, here
 *    as PER_GROUP.
 *
 * Data layout (all tensors dense, row-major, innermost last):
 *   codes       uint8  [num_blocks, num_kv_heads, block_size, Dp]
 *               Dp = head_dim (int8, e4m3) or head_dim/2 (int4: channel 2j in
 *               the low nibble of byte j, channel 2j+1 in the high nibble,
 *               two's-complement nibbles)
 *   PER_ROW     scales fp32 [num_blocks, num_kv_heads, block_size]
 *   PER_TENSOR  scale  fp32 [1]
 *   PER_CHANNEL scales fp32 [num_kv_heads, head_dim]
 *   PER_GROUP   scales fp32 [num_blocks, num_kv_heads, block_size, head_dim / group_size]
 *   cache slot  s = block * block_size + row
 *   q, out      bf16   [batch, q_tokens, num_q_heads, head_dim]
 *   k_new/v_new bf16   [n_tokens, num_kv_heads, head_dim]
 *   block_table int32  [batch, max_blocks_per_seq]
 *   seq_lens    int32  [batch]   (each includes the q_tokens new tokens)
 *   lse_out     fp32   [batch, q_tokens, num_q_heads] (natural log)
 *
 * Supported on the GPU path: head_dim in {64, 128, 256}, and 576 for a LATENT
 * cache (absorbed MLA, e.g. 512 latent + 64 rotary channels) with int8 or
 * e4m3 codes and per-row, per-tensor or per-channel scales, at most 48 query
 * rows per kv head; num_q_heads a multiple of num_kv_heads with a ratio of at
 * most 8; q_tokens in [1, 8]; block_size a power of two >= 16; batch <= 1024.
 * Pointers 16-byte aligned.
 */
#ifndef KVQ_H
#define KVQ_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define KVQ_API __attribute__((visibility("default")))

/* A cudaStream_t (the same type: a pointer to the runtime's stream object);
 * NULL is the legacy default stream. */
typedef struct CUstream_st* kvq_stream_t;

typedef enum {
  KVQ_OK = 0,
  KVQ_ERR_INVALID_ARG = 1,         /* bad enum, shape, null or misaligned pointer */
  KVQ_ERR_UNSUPPORTED = 2,         /* valid, but outside what the GPU path covers */
  KVQ_ERR_WORKSPACE_TOO_SMALL = 3, /* workspace_bytes < kvq_decode_workspace_size */
  KVQ_ERR_CUDA = 4,                /* a CUDA runtime call or a launch failed */
  KVQ_ERR_DEVICE_TIMEOUT = 5       /* a bounded device-side wait gave up */
} kvq_status;

/* Cache element types (PR #29912: int8, float8e4m3fn; PR #32515: packed int4). */
typedef enum { KVQ_INT8 = 1, KVQ_FP8_E4M3 = 2, KVQ_INT4 = 3 } kvq_dtype;

/* Scale granularity: PER_ROW is one absmax scale per (token, kv head) row,
 * computed on append (kv-quant-attn "Method"; issue #29783 per-token);
 * PER_TENSOR and PER_CHANNEL are static caller-given scales (PR #29912);
 * PER_GROUP applies the PER_ROW rule to each run of kvq_cache.group_size
 * consecutive channels of a row, one scale per group (the group-wise scaling
 * the kv-quant-attn page lists under "Requirements and limits" as not done
 * there, which would narrow the int4 error around outlier channels). */
typedef enum {
  KVQ_SCALE_PER_ROW = 1,
  KVQ_SCALE_PER_TENSOR = 2,
  KVQ_SCALE_PER_CHANNEL = 3,
  KVQ_SCALE_PER_GROUP = 4
} kvq_scale_mode;

/* Device-side data violations, OR-ed into a per-device flag word.  The
 * offending access is skipped (never trapped); outputs that depend on it are
 * unspecified.  Read with kvq_get_device_error. */
#define KVQ_DEVERR_SLOT 0x1u      /* append: slot_mapping[n] >= num_blocks * block_size */
#define KVQ_DEVERR_BLOCK_ID 0x2u  /* decode: block_table entry outside [0, num_blocks) */
#define KVQ_DEVERR_SEQ_LEN 0x4u   /* decode: seq_len < 0, > capacity, or > max_seq_len */
#define KVQ_DEVERR_TIMEOUT 0x8u   /* a bounded pipeline wait gave up */
#define KVQ_DEVERR_POSITION 0x10u /* norm/RoPE prologue: position outside [0, max_position) */
#define KVQ_DEVERR_KEEP_INDEX 0x20u /* kvq_evict_compact: a kept row outside [0, capacity), or in
                                       * place before its destination */
#define KVQ_DEVERR_NO_BLOCKS 0x40u  /* kvq_pages_step: a sequence got no pages (the pool is short) */

/* Cache layouts (PR #29912, kv_cache_layout and v_head_size): SEPARATE K and V
 * caches, or LATENT (absorbed MLA): one cache whose rows serve as K, and whose
 * leading v_head_size channels serve as V. */
typedef enum { KVQ_LAYOUT_SEPARATE = 0, KVQ_LAYOUT_LATENT = 1 } kvq_layout;

/* The paged cache: one descriptor per layer (kv-quant-attn "Usage": one cache
 * object per layer).  All pointers are device memory owned by the caller.
 * k_scale / v_scale: PER_ROW fp32 [num_blocks, Hkv, block_size] or PER_GROUP
 * fp32 [num_blocks, Hkv, block_size, head_dim / group_size] arrays written by
 * kvq_append (16-byte aligned), or the static scales (PER_TENSOR [1],
 * PER_CHANNEL [Hkv, head_dim]; finite and > 0: the precondition the PR #447
 * scale loader checks). */
typedef struct {
  int32_t dtype;        /* kvq_dtype */
  int32_t k_mode;       /* kvq_scale_mode of K */
  int32_t v_mode;       /* kvq_scale_mode of V */
  int32_t num_blocks;   /* pool size in blocks */
  int32_t block_size;   /* tokens per block (power of two >= 16) */
  int32_t num_kv_heads; /* Hkv */
  int32_t head_dim;     /* D */
  void* k_codes;        /* uint8 [num_blocks, Hkv, block_size, Dp] */
  void* v_codes;
  float* k_scale;
  float* v_scale;
  int32_t layout;       /* kvq_layout; LATENT: v_codes, v_scale, v_mode are ignored (V is the K
                           row, with K's scales) and may be NULL / 0; kvq_append writes K only
                           and ignores v_new; kvq_combine writes out [B, T, Hq, v_head_size] */
  int32_t v_head_size;  /* LATENT: channels of V, a multiple of 8 in [8, head_dim]; 0 = head_dim
                           (the pages' DeepSeek-V3 example: head_dim 576, v_head_size 512) */
  int32_t group_size;   /* PER_GROUP on either side: channels per scale group, 32, 64 or 128
                           and at most head_dim (one group size for both sides); otherwise
                           ignored.  Decode with a PER_GROUP side runs on the mma.sync
                           kernel's grouped layout for every query-row count. */
} kvq_cache;

/* One decode call (PagedAttention's inputs, PR #29912 Summary of Changes). */
typedef struct {
  int32_t batch;              /* B (<= 1024) */
  int32_t num_q_heads;        /* Hq; Hq / Hkv <= 8; query head i reads kv head i / (Hq/Hkv) */
  int32_t q_tokens;           /* T in [1, 8]: 1, or 1 + drafts (PR #32515, speculative
                                 decode); draft t sits at position seq_len - T + t and
                                 sees keys 0..that position (causal among drafts) */
  int32_t max_blocks_per_seq; /* block_table row length; capacity = it * block_size */
  int32_t max_seq_len;        /* host upper bound on seq_lens, like attention_metadata
                                 [max_kv_len] (PR #29912); 0 = capacity.  Sizes the grid,
                                 never read back from the device. */
  float sm_scale;             /* logit scale; <= 0 selects 1/sqrt(head_dim) */
  float softcap;              /* > 0: logit s -> softcap * tanh(s / softcap); 0 = off */
  int32_t window;             /* > 0: keep the `window` most recent keys up to and
                                 including the query position; 0 = off */
  uint32_t flags;             /* KVQ_DECODE_* bits below; 0 = the defaults */
} kvq_decode_params;

/* kvq_decode_params.flags.
 *
 * KVQ_DECODE_EARLY_INPUTS: every kvq kernel may start while the kernel enqueued
 * just before it on the stream finishes (programmatic dependent launch).  By
 * default kvq_decode reads nothing until that preceding kernel has completed.
 * With this bit it reads q, block_table, seq_lens and the static scales
 * (PER_TENSOR / PER_CHANNEL) while the preceding kernel is still running, and
 * waits only before it reads the cache and writes the workspace: the split plan
 * and the query prologue then overlap that kernel's tail.  Set it only when
 * none of those inputs is written by the operation enqueued just before
 * kvq_decode on the stream: e.g. they were copied from the host, or that
 * operation is kvq_append (which writes only the cache) and the one before
 * the append writes none of them either (kvq_append lets the decode start
 * while that one finishes: a kvq_combine, say, which writes only out and
 * lse).  It must not be set when that operation is kvq_norm_rope_apply
 * producing q, or any kernel that writes q, block_table or seq_lens.
 *
 * KVQ_DECODE_NO_TCGEN05: keep shapes of 17..64 query rows per kv head on the
 * mma.sync kernel's layouts instead of the tensor-memory (tcgen05) kernel
 * (for comparing the two; results agree within the parity tolerance). */
#define KVQ_DECODE_EARLY_INPUTS 0x1u
#define KVQ_DECODE_NO_TCGEN05 0x2u
/* KVQ_DECODE_EARLY_CACHE (with KVQ_DECODE_EARLY_INPUTS): the operation
 * enqueued just before kvq_decode writes no cache row other than the step's
 * new tokens (positions seq_lens[b] - q_tokens .. seq_lens[b] - 1): e.g. it
 * is kvq_append of exactly those tokens, or it writes no cache at all.  The
 * decode then loads every older row while that operation is still running and
 * waits for it only before the 64- or 128-key tile that holds the new tokens,
 * so the first cache reads overlap its tail.  Without KVQ_DECODE_EARLY_INPUTS
 * the bit has no effect.  A kvq_evict_compact must not be among the last two
 * operations before such a decode: it moves older rows. */
#define KVQ_DECODE_EARLY_CACHE 0x4u

/* Human-readable name of a status code (static storage). */
KVQ_API const char* kvq_status_string(kvq_status status);

/* kvq_append -- quantize-on-write of new K/V rows into their cache slots
 * (ReshapeAndCache, PR #29912; per-row absmax, kv-quant-attn "Method";
 * int4 nibble packing, PR #32515).
 * For each token n and kv head h, the D bf16 values of k_new[n, h, :] (and of
 * v_new) are quantized: PER_ROW scale = absmax / qmax (IEEE fp32 division,
 * qmax 127 / 7 / 448, an all-zero row stores scale 0 and zero codes; PER_GROUP
 * the same over each group of group_size channels), then
 * code = clamp(round_half_even(x / scale), -qmax, qmax) for int8 / int4, or
 * the nearest e4m3 value (ties to even, finite overflow saturated to 448).
 * slot_mapping int64 [n_tokens] (device): slot < 0 skips the token (padding);
 * slot >= num_blocks * block_size sets KVQ_DEVERR_SLOT and skips it.
 * Rows already in the cache are never touched.  n_tokens == 0 is a no-op.
 * Its kernel lets the next kernel on the stream be scheduled at once (that
 * kernel may then run while this one and the one before it finish); every
 * kvq kernel waits for its predecessor before it reads what that one writes,
 * so only a decode with KVQ_DECODE_EARLY_INPUTS reads anything early. */
KVQ_API kvq_status kvq_append(const kvq_cache* cache, const void* k_new, const void* v_new,
                              const int64_t* slot_mapping, int32_t n_tokens,
                              kvq_stream_t stream);

/* The prologue before the cache write: QK-RMSNorm, then RoPE (QkNormRotaryTNH
 * in onnxruntime PR #29912, Summary of Changes: q_norm_weight / k_norm_weight
 * inputs, qk_norm_epsilon with default 1e-6, rotary_offset, which rotates
 * channels [rotary_offset, rotary_offset + rotary_dim)).  For each (token,
 * head) row x of head_dim bf16 values:
 *   RMSNorm (norm_weight != NULL): y_d = (x_d * r) * w_d,
 *     r = 1 / sqrt(sum_d x_d^2 / head_dim + eps);
 *   RoPE (rotary_dim > 0): the pair (a, b) of angle index i in
 *     [0, rotary_dim/2) becomes (a cos - b sin, b cos + a sin), with
 *     cos = cos_cache[pos, i], sin = sin_cache[pos, i] for the token's
 *     position pos; pairs are (off + i, off + i + rotary_dim/2) (half split)
 *     or (off + 2i, off + 2i + 1) (rotary_interleaved);
 * then one round-to-nearest-even to bf16 per value.  Arithmetic is IEEE fp32,
 * one rounding per operation in a fixed order, so results are reproducible
 * bit for bit: with E = head_dim / 32, the squares of channels
 * l*E .. l*E + E - 1 are summed in order into partial l (l = 0..31), then for
 * o = 16, 8, 4, 2, 1 each partial l becomes partial l + partial (l xor o);
 * each rotated value is (y * cos) -+ (partner * sin) with both products
 * rounded.  The pages fix neither the rotation layout nor the tables: both
 * are the caller's, as here. */
typedef struct {
  const void* norm_weight;    /* bf16 [head_dim] (device), or NULL: no RMSNorm */
  float norm_eps;             /* <= 0 selects 1e-6 */
  int32_t rotary_dim;         /* 0: no RoPE; else even, rotary_offset + rotary_dim <= head_dim */
  int32_t rotary_offset;      /* first rotated channel (>= 0) */
  int32_t rotary_interleaved; /* 0: half-split pairs; 1: adjacent pairs */
  const float* cos_cache;     /* fp32 [max_position, rotary_dim/2] (device) */
  const float* sin_cache;     /* fp32 [max_position, rotary_dim/2] (device) */
  int32_t max_position;       /* rows of the tables (> 0 when rotary_dim > 0) */
  int32_t hadamard;           /* 1: then rotate the row by the orthonormal Walsh-Hadamard
                                 matrix (Sylvester order, entry (i, j) =
                                 (-1)^popcount(i & j) / sqrt(head_dim)): butterflies of
                                 span 1, 2, 4, ... in fp32, then times
                                 fl32(1 / fl32(sqrt(head_dim))).  Apply it to Q and K alike:
                                 dot products are unchanged while an outlier channel is
                                 spread over the row before quantization (the rotation
                                 PR #32515 names as the follow-up for the int4 cache) */
} kvq_norm_rope;

/* kvq_norm_rope_apply -- the prologue on x [n_tokens, num_heads, head_dim]
 * bf16 (device) into y (same shape; y == x is allowed), e.g. the queries
 * before kvq_decode.  positions int64 [n_tokens] (device; may be NULL when
 * rotary_dim == 0): a position outside [0, max_position) sets
 * KVQ_DEVERR_POSITION and leaves that token's rows of y unwritten.
 * head_dim in {64, 128, 256, 576} (the Hadamard rotation: powers of two only);
 * x, y 16-byte aligned. */
KVQ_API kvq_status kvq_norm_rope_apply(const kvq_norm_rope* prologue, const void* x, void* y,
                                       const int64_t* positions, int32_t n_tokens,
                                       int32_t num_heads, int32_t head_dim, kvq_stream_t stream);

/* kvq_append_norm_rope -- kvq_append with the prologue fused in front of the
 * K quantizer: each K row is normalized and rotated as kvq_norm_rope_apply
 * would (same fp32 arithmetic, same bf16 rounding) and the resulting bf16 row
 * is quantized exactly as kvq_append quantizes its input; V rows are
 * quantized as given (the prologue acts on Q and K only).  A token with a
 * negative slot is skipped; one whose position is outside the tables sets
 * KVQ_DEVERR_POSITION and neither its K nor its V rows are written. */
KVQ_API kvq_status kvq_append_norm_rope(const kvq_cache* cache, const kvq_norm_rope* k_prologue,
                                        const void* k_new, const void* v_new,
                                        const int64_t* slot_mapping, const int64_t* positions,
                                        int32_t n_tokens, kvq_stream_t stream);

/* Bytes of workspace kvq_decode needs for these shapes on the current device
 * (split partials and the device-side split plan).  Host-only arithmetic plus
 * one cached device-attribute query. */
KVQ_API kvq_status kvq_decode_workspace_size(const kvq_cache* cache,
                                             const kvq_decode_params* params,
                                             size_t* workspace_bytes);

/* kvq_decode -- split-KV flash-decoding over the quantized pages
 * (PagedAttention paged decode, PR #29912; kv-quant-attn "Method").
 * Reads q, block_table, seq_lens and the cache on the device, dequantizes on
 * the fly, and writes per-split partials (log-sum-exp and normalized output)
 * plus the split plan into `workspace` (device, caller owned, at least
 * kvq_decode_workspace_size bytes, 256-byte aligned).  The result is
 * completed by kvq_combine with the same cache, params and workspace on the
 * same stream.  Per query row, logits are sm_scale * <q, k_j>, capped by
 * softcap, masked to keys j <= pos (and j > pos - window when set).
 * The kvq kernels let the next kernel on the stream start early
 * (programmatic dependent launch); kvq_decode itself waits for the preceding
 * kernel to complete before it reads any input, unless params->flags has
 * KVQ_DECODE_EARLY_INPUTS (see there for when that is allowed). */
KVQ_API kvq_status kvq_decode(const kvq_cache* cache, const kvq_decode_params* params,
                              const void* q, const int32_t* block_table,
                              const int32_t* seq_lens, void* workspace,
                              size_t workspace_bytes, kvq_stream_t stream);

/* kvq_combine -- fixed-order log-sum-exp merge of the split partials
 * (kv-quant-attn "Method": partials merged in a fixed order, bitwise
 * reproducible), then the exact head-sink rescale o *= 1/(1+exp(s_h - lse))
 * (ApplyHeadSink, PR #29912), the static V scale (PER_TENSOR, or PER_CHANNEL
 * per output channel: the fold of PR #32515), and a round-to-nearest-even
 * bf16 store to out [B, T, Hq, D].
 * head_sink fp32 [Hq] or NULL; lse_out fp32 [B, T, Hq] or NULL (natural-log
 * LSE of the logits, before the sink; -inf for an empty key set, whose output
 * row is zero). */
KVQ_API kvq_status kvq_combine(const kvq_cache* cache, const kvq_decode_params* params,
                               const void* workspace, size_t workspace_bytes,
                               const float* head_sink, void* out, float* lse_out,
                               kvq_stream_t stream);

/* kvq_prefill -- attention of a chunk of C = params->q_tokens new query tokens
 * per sequence over the quantized cache (chunked prefill / prompt attention:
 * PR #29912 and PR #32515 testing name prefill and chunked prefill; the head
 * sink applies as in decode).  The chunk's K/V rows are appended first
 * (kvq_append); token c of sequence b sits at position seq_lens[b] - C + c
 * and sees keys 0..that position (and the window, when set).  q, out bf16
 * [B, C, Hq, D]; lse_out fp32 [B, C, Hq] or NULL; head_sink as in
 * kvq_combine.  The chunk is cut into groups of T tokens (virtual
 * sequences; sequence b's j-th group sees the prefix seq_lens[b] - C + T
 * (j + 1)), run as one attention pass and one combine; B * C / T <= 1024.
 * With head_dim 128 or 256, no group-wise scales and KVQ_DECODE_NO_TCGEN05
 * unset, T is the largest divisor of C with T x (Hq / Hkv) <= 128 when that
 * gives at least 64 query rows per kv head: a group's rows are the M
 * dimension of tcgen05 MMAs and each key tile of its prefix is dequantized
 * once for all of them (the kv-quant-attn page, "Requirements and limits":
 * prefill wants a tiled attention kernel).  Otherwise T is the largest of 8,
 * 4, 2, 1 dividing C and the groups run on the decode kernels.  Each group
 * reads its prefix, so a chunk costs C / T passes over the cache, shared
 * through L2 where they coincide.  C >= 1 (no upper bound besides the
 * virtual batch).  workspace: at least kvq_prefill_workspace_size bytes,
 * 256-byte aligned. */
KVQ_API kvq_status kvq_prefill_workspace_size(const kvq_cache* cache, const kvq_decode_params* params,
                                              size_t* workspace_bytes);
KVQ_API kvq_status kvq_prefill(const kvq_cache* cache, const kvq_decode_params* params, const void* q,
                               const int32_t* block_table, const int32_t* seq_lens, const float* head_sink,
                               void* out, float* lse_out, void* workspace, size_t workspace_bytes,
                               kvq_stream_t stream);

/* The score rule of a masked call: a bias that depends on distance, and an
 * interval of visible keys per query token.  Query token c of sequence b sits
 * at position pos = seq_lens[b] - C + c (C = params->q_tokens) and sees the
 * keys j with key_begin[b, c] <= j < key_end[b, c] (cut to [0, seq_lens[b]);
 * NULL: 0 and pos + 1, the causal rule) and, with params->window > 0,
 * j > pos - window.  Intervals say:
 *   document mask  key_begin = first position of the token's document
 *   prefix mask    key_end = max(pos + 1, prefix length): the prefix is seen
 *                  in both directions
 *   padding        key_end <= key_begin: the token sees nothing; its output
 *                  rows are zero and their lse is -inf
 * The logit of query head h and key j is softcap(sm_scale <q, k_j>) -
 * slopes[h] * |pos - j| (the bias comes after the cap and is not capped).
 * Positions and distances count cache rows.  After kvq_evict_compact they are
 * those of the rows that were kept, and every kv head kept its own: a distance
 * shrinks by the evicted rows between query and key, and key_begin, key_end and
 * window cut other tokens in each head.  Only the rows that sinks and recent
 * protect lie at the same places in all of them.  The reference's pages name
 * neither rule; both are the usual ones of models with linear distance biases,
 * packed documents and bidirectional prefixes. */
typedef struct {
  const float* slopes;      /* fp32 [Hq] (device; finite, any sign), or NULL: no bias */
  const int32_t* key_begin; /* int32 [B, C] (device; any values), or NULL */
  const int32_t* key_end;   /* int32 [B, C] (device; any values), or NULL */
} kvq_score_mask;

/* kvq_attend_masked -- attention of C = params->q_tokens >= 1 query tokens per
 * sequence under a score rule: one call for a decode step (C = 1, or 1 +
 * drafts) and for a prompt's chunk (any C, not only multiples of a tile).
 * Arguments and results as in kvq_prefill; mask may be NULL (causal, no
 * bias).  Sequences are cut into groups of tokens; of a group's keys those
 * before the first and behind the last that some token of it sees are not read,
 * and their pages need not be in the table.  (Those between are read, seen or
 * not.)  With head_dim 128 or 256, no group-wise scales,
 * KVQ_DECODE_NO_TCGEN05 unset and more than 16 query rows per kv head, the
 * groups are tiles of up to 128 rows on tcgen05 MMAs; otherwise of up to 8
 * tokens on the mma.sync kernel.  (Under a softcap tiles from 64 rows on; with
 * a per-channel K scale, an lse_out and head_dim 256 tiles have up to 64 rows,
 * from 56 on under a softcap.)  KVQ_DECODE_EARLY_INPUTS and
 * KVQ_DECODE_EARLY_CACHE have no effect here.  lse_out is fp32-accurate (on the
 * tiles a bias counts to 2^-14 of its slope): with a per-channel K scale the
 * query operand is then carried in two f16 parts, which costs time (a prompt's
 * tiles about half as much again at head_dim 128 and twice at 256); lse_out NULL
 * leaves that out.  batch <= 1024; batch * C <= 2^30.  out must not overlap q.
 * workspace: at least
 * kvq_attend_masked_workspace_size bytes, 256-byte aligned; it belongs to
 * this call until the call's kernels have run. */
KVQ_API kvq_status kvq_attend_masked_workspace_size(const kvq_cache* cache, const kvq_decode_params* params,
                                                    size_t* workspace_bytes);
KVQ_API kvq_status kvq_attend_masked(const kvq_cache* cache, const kvq_decode_params* params,
                                     const kvq_score_mask* mask, const void* q, const int32_t* block_table,
                                     const int32_t* seq_lens, const float* head_sink, void* out, float* lse_out,
                                     void* workspace, size_t workspace_bytes, kvq_stream_t stream);

/* kvq_key_mass -- the attention weight that every cached key receives from
 * this step's query tokens, accumulated: for each sequence b, kv head g and
 * position j in [0, seq_lens[b]), with slot(j) the key's place in the pages,
 *   mass[slot(j)] = old + sum over tokens c and query heads h of group g that
 *                   see j of exp(s[b, c, h, j] - lse[b, c, h]),
 *   old = 0 for the last `fresh` positions (the step's new tokens, which held
 *         no weight before), else decay * mass[slot(j)].
 * s and the visible keys are those of kvq_attend_masked with the same params
 * and mask (of kvq_decode / kvq_prefill with mask NULL); lse fp32
 * [B, C, Hq] is their lse_out (before the head sink; -inf rows add nothing).
 * For the weights beside a head sink pass log(e^lse + e^sink) in its place.
 * kvq_attend_masked's is fp32-accurate; the unmasked calls' is a few 1e-7 of a
 * softcap off, and kvq_decode's with 17 or more query rows per kv head up to
 * 2^-11 (weights summed as f16), which the weights of the row then show.
 * mass fp32 [num_blocks, Hkv, block_size] (device), laid out like per-row
 * scales; slots of other positions are left as they are.  C = q_tokens >= 1:
 * one decode step, or the last tokens of a prompt looking back over it.
 * decay in [0, 1]: 1 sums, 0 overwrites (mass is then not read).  The scores
 * are fp32-accurate (a folded per-channel K scale enters as two f16 parts).
 * Each key is written by one thread in a fixed order: repeated calls give the
 * same bits.  A page must not be shared by two sequences of the call.  Every
 * page of [0, seq_lens[b]) is needed: an unreadable block id sets
 * KVQ_DEVERR_BLOCK_ID, and its keys keep what they held.
 * workspace: at least kvq_key_mass_workspace_size bytes, 256-byte aligned; it
 * belongs to this call until the call's kernels have run. */
KVQ_API kvq_status kvq_key_mass_workspace_size(const kvq_cache* cache, const kvq_decode_params* params,
                                               size_t* workspace_bytes);
KVQ_API kvq_status kvq_key_mass(const kvq_cache* cache, const kvq_decode_params* params, const kvq_score_mask* mask,
                                const void* q, const int32_t* block_table, const int32_t* seq_lens,
                                const float* lse, float decay, int32_t fresh, float* mass, void* workspace,
                                size_t workspace_bytes, kvq_stream_t stream);

/* An eviction: every sequence longer than `budget` rows is cut to `budget`. */
typedef struct {
  int32_t batch;              /* B */
  int32_t max_blocks_per_seq; /* block_table row length; capacity = it * block_size */
  int32_t max_seq_len;        /* host upper bound on seq_lens; 0 = capacity */
  int32_t num_blocks;         /* pool size in blocks */
  int32_t block_size;         /* tokens per block (power of two >= 16) */
  int32_t num_kv_heads;       /* Hkv */
  int32_t budget;             /* rows kept per sequence (>= 1) */
  int32_t sinks;              /* the first `sinks` rows always stay */
  int32_t recent;             /* the last `recent` rows always stay; sinks + recent <= budget */
} kvq_evict_params;

/* kvq_evict_select -- the rows that stay, for each sequence and kv head on its
 * own: of a sequence of L > budget rows the first `sinks`, the last `recent`,
 * and of the rest the budget - sinks - recent with the largest mass; among
 * equal masses the lower row stays, -0 equals +0, and a NaN ranks below every
 * number.  A sequence of at most `budget` rows stays whole.
 * keep int32 [B, Hkv, budget]: the kept rows in ascending order, then -1.
 * kept_lens int32 [B]: min(seq_lens[b], budget), the lengths after
 * kvq_evict_compact.  keep and kept_lens may overlap neither one another nor
 * an input (refused).  An unreadable block id sets KVQ_DEVERR_BLOCK_ID and
 * ranks its rows as NaN.
 * num_kv_heads * block_size <= 2^29; batch * num_kv_heads <= 2^24. */
KVQ_API kvq_status kvq_evict_select(const kvq_evict_params* params, const float* mass, const int32_t* block_table,
                                    const int32_t* seq_lens, int32_t* keep, int32_t* kept_lens,
                                    kvq_stream_t stream);

/* kvq_evict_compact -- moves the kept rows together: position i of sequence b
 * and kv head g becomes what position keep[b, g, i] was, for i < kept_lens[b]
 * (at most budget): K and V codes, per-row or per-group scales, and mass when
 * it is given.  keep must be strictly ascending with keep[i] >= i, as
 * kvq_evict_select writes it.  The cache's block size, pool size and kv heads
 * must be the params'.
 * dst_table NULL or equal to block_table: in place; positions behind
 * kept_lens[b] keep their contents, and the pages behind the last kept row
 * are free for other use.  Otherwise dst_table [B, max_blocks_per_seq] names
 * other pages, none of which is a source page of this call: for sequences
 * whose pages are shared, which in-place moves would change for everyone.
 * A kept row outside the capacity, or in place one with keep[i] < i, sets
 * KVQ_DEVERR_KEEP_INDEX and is not moved (its destination's contents are
 * unspecified).
 * K is moved as it was written: with rotary positions it keeps the rotation
 * of its first position.
 * In place the kernel's blocks wait for one another (a cooperative launch with
 * bounded waits; KVQ_DEVERR_TIMEOUT).  The tables, keep and kept_lens may not
 * overlap the cache's arrays, mass or the part of the workspace that is needed
 * (refused).  workspace: at
 * least kvq_evict_compact_workspace_size bytes, 256-byte aligned (used in place
 * only, but checked always); it belongs to this call until its kernel has
 * run. */
KVQ_API kvq_status kvq_evict_compact_workspace_size(const kvq_cache* cache, const kvq_evict_params* params,
                                                    size_t* workspace_bytes);
KVQ_API kvq_status kvq_evict_compact(const kvq_cache* cache, const kvq_evict_params* params,
                                     const int32_t* block_table, const int32_t* dst_table, const int32_t* keep,
                                     const int32_t* kept_lens, float* mass, void* workspace,
                                     size_t workspace_bytes, kvq_stream_t stream);

/* kvq_attend_prompt -- attention of whole prompts over the bf16 K and V at
 * hand, before (or without) a cache: N = total_tokens rows hold the tokens of
 * B sequences one after another, sequence b in rows cu_seqlens[b] ..
 * cu_seqlens[b + 1] - 1.  Token i of a sequence sees its tokens j <= i (with
 * window > 0: j > i - window), so it is what kvq_prefill of the whole sequence
 * gives without the cache's rounding.  Logits, softcap, window, head_sink,
 * lse_out and the order of heads are those of kvq_decode_params.
 *   q    bf16 [N, Hq, D]    out bf16 [N, Hq, D] (dense)
 *   k, v bf16 [N, Hkv, D]   lse_out fp32 [N, Hq] (dense) or NULL
 *   cu_seqlens int32 [B + 1], ascending (device)
 * head_dim in {64, 128, 256}; Hq a multiple of Hkv, at most 8 times it.
 * q, k and v may be slices of a wider projection: q_stride, k_stride and
 * v_stride are the elements from one token to the next (a multiple of 8; 0:
 * dense); the heads of a token are dense.  Lengths are on the device: rows of
 * out and lse_out that belong to no sequence (before cu_seqlens[0], behind
 * cu_seqlens[B], an empty sequence) are left as they were, and what q, k and v
 * hold there, NaN included, changes nothing.  A sequence whose bounds descend,
 * leave [0, N] or exceed max_seq_len sets KVQ_DEVERR_SEQ_LEN and is skipped; so
 * is, behind such bounds, a sequence that begins before the end of an earlier
 * one whose own bounds are right (no row belongs to two sequences).
 * Inf or NaN in a token's K or V row reaches the tokens that see it, and no
 * other (tiles of rows whose results hold NaN are computed twice).
 * Weights enter the product with V as bf16; sums, maxima and lse are fp32.
 * Repeated calls give the same bits.  out must not overlap q, k or v.
 * batch <= 1024.  workspace: at least kvq_attend_prompt_workspace_size bytes,
 * 256-byte aligned; it belongs to this call until the call's kernels have
 * run. */
typedef struct {
  int32_t batch;        /* B (<= 1024) */
  int32_t total_tokens; /* N: rows of q, k, v and out */
  int32_t num_q_heads;  /* Hq */
  int32_t num_kv_heads; /* Hkv */
  int32_t head_dim;     /* D */
  int32_t max_seq_len;  /* host upper bound on a sequence's tokens; 0 = total_tokens */
  int32_t q_stride;     /* elements between tokens of q; 0 = Hq * D */
  int32_t k_stride;     /* 0 = Hkv * D */
  int32_t v_stride;     /* 0 = Hkv * D */
  float sm_scale;       /* <= 0 selects 1/sqrt(head_dim) */
  float softcap;        /* > 0: logit s -> softcap * tanh(s / softcap); 0 = off */
  int32_t window;       /* > 0: the `window` most recent tokens, the query's own among them; 0 = off */
} kvq_prompt_params;

KVQ_API kvq_status kvq_attend_prompt_workspace_size(const kvq_prompt_params* params, size_t* workspace_bytes);
KVQ_API kvq_status kvq_attend_prompt(const kvq_prompt_params* params, const void* q, const void* k, const void* v,
                                     const int32_t* cu_seqlens, const float* head_sink, void* out, float* lse_out,
                                     void* workspace, size_t workspace_bytes, kvq_stream_t stream);

/* A tree of drafted tokens per sequence (speculative decode with several
 * candidates; the drafts of kvq_decode are its case of one chain).  The last
 * num_nodes[b] rows of sequence b are the nodes, node i at row P + i with
 * P = seq_lens[b] - num_nodes[b]; their K and V rows are appended first
 * (kvq_append), like any tokens.  parents[b, i] is the node that node i
 * follows; one outside [0, i) (-1, say) makes i a root, which follows the
 * prefix alone.  Node i stands at position P + depth(i), a root's depth being
 * 0: the position its rotary angle wants (kvq_pages_step gives it). */
#define KVQ_MAX_TREE_NODES 256
typedef struct {
  const int32_t* parents;   /* int32 [B, T] (device), T = params->q_tokens <= KVQ_MAX_TREE_NODES */
  const int32_t* num_nodes; /* int32 [B] (device), or NULL: T nodes each.  Outside [0, T], or more
                               than seq_lens[b]: KVQ_DEVERR_SEQ_LEN, and cut to that range */
} kvq_tree;

/* kvq_attend_tree -- attention of the nodes of each sequence's tree over the
 * quantized cache: node i sees the prefix rows j < P and, of the nodes, its
 * ancestors and itself.  With params->window > 0 a key counts when its
 * position (a prefix row's is its row, a node's P + depth) is above the
 * node's own minus window.  q, out bf16 [B, T, Hq, D]; nodes i >= num_nodes[b]
 * are padding: their output rows are zero and their lse -inf.  A node whose
 * cached row has a scale of inf or NaN reaches its descendants only (their
 * results are NaN, as those of a query that holds NaN), and a finite one,
 * however large, takes nothing of the others' precision: weights are relative
 * to the largest V scale of the rows that a node itself sees.
 * Everything else is as in kvq_attend_masked.
 * batch <= 1024.  workspace: at least kvq_attend_tree_workspace_size bytes,
 * 256-byte aligned; it belongs to this call until the call's kernels have
 * run. */
KVQ_API kvq_status kvq_attend_tree_workspace_size(const kvq_cache* cache, const kvq_decode_params* params,
                                                  size_t* workspace_bytes);
KVQ_API kvq_status kvq_attend_tree(const kvq_cache* cache, const kvq_decode_params* params, const kvq_tree* tree,
                                   const void* q, const int32_t* block_table, const int32_t* seq_lens,
                                   const float* head_sink, void* out, float* lse_out, void* workspace,
                                   size_t workspace_bytes, kvq_stream_t stream);

/* kvq_tree_accept -- the path through each tree that the model agrees with,
 * and its rows moved together.  Node 0 is accepted (the step's own token);
 * after an accepted node n the lowest child c of n with drafts[b, c] ==
 * chosen[b, n] is, until there is none.  chosen[b, n] is what the model
 * answers after node n (an argmax or a sample of its logits).
 *   path [B, T] int32         the accepted nodes in order, then -1
 *   accepted [B] int32        how many (0 for a sequence without nodes)
 *   new_lens [B] int32        P + accepted: the lengths after the call
 *   next_tokens [B] int64     chosen after the last accepted node (-1: no nodes)
 * Row P + path[i] of the cache (K and V codes, per-row or per-group scales,
 * and mass fp32 [num_blocks, Hkv, block_size] when it is given) moves to row
 * P + i; the rows behind keep their contents.  The moves read block_table
 * entries of the nodes' rows only; an unreadable block id sets
 * KVQ_DEVERR_BLOCK_ID and its row is not moved.  A page that holds nodes must
 * not be shared by two sequences.  Of params only batch, q_tokens (T),
 * max_blocks_per_seq and max_seq_len are used.  drafts, chosen int64 [B, T].
 * The outputs may overlap neither an input nor one another (refused). */
KVQ_API kvq_status kvq_tree_accept(const kvq_cache* cache, const kvq_decode_params* params, const kvq_tree* tree,
                                   const int64_t* drafts, const int64_t* chosen, const int32_t* block_table,
                                   const int32_t* seq_lens, int32_t* path, int32_t* accepted, int32_t* new_lens,
                                   int64_t* next_tokens, float* mass, kvq_stream_t stream);

/* kvq_pages_step -- the bookkeeping of a step on the device: which pages each
 * sequence gives back or gets, where its new rows lie, and at which positions.
 * Sequence b holds the pages of held_lens[b] rows (ceil(held / block_size)
 * entries of its block_table row); the first start_lens[b] <= held_lens[b]
 * rows stay (start_lens NULL: all) and new_tokens[b] rows come behind them.
 * With want = start + new it gives back the pages behind ceil(want /
 * block_size) or gets those it lacks.  A finished sequence is start = new = 0,
 * a fresh one held = 0, a step after kvq_tree_accept start = its new_lens.
 * The pool is a stack: free_blocks[0 .. free_count) are free, the last on top.
 * Given-back pages are pushed in order of sequence and page, then the pages
 * that are asked for popped in that order; a call with the same inputs gives
 * the same tables, and entries of free_blocks below free_count and of a table
 * row below its held pages are never changed.
 * A sequence is refused, and left as it was, when its rows would exceed its
 * table row or the new tokens up to and with it max_tokens
 * (KVQ_DEVERR_SEQ_LEN), or when it needs pages and the pages asked for up to
 * and with it exceed the pool (KVQ_DEVERR_NO_BLOCKS); the sums count refused
 * sequences too, the pool the pages that sequences not refused by the first
 * two give back.  Its length stays held_lens[b] and it gets no tokens, so
 * that the call can be made again with the same values.  held < 0 or above
 * the table row, start outside [0, held] or new < 0: KVQ_DEVERR_SEQ_LEN,
 * refused and not counted.
 *   block_table [B, max_blocks_per_seq] int32  entries behind the held pages
 *                are written for the pages that were got; others stay
 *   seq_lens [B] int32        start + new (refused: held)
 *   free_left [1] int32       free_count after the call
 *   cu_seqlens [B + 1] int32  prefix sums of the tokens that were granted
 *   slot_mapping [max_tokens] int64   slot of each new row, sequence after
 *                sequence (kvq_append's); -1 behind the last
 *   positions [max_tokens] int64      start + i for the i-th new row of a
 *                sequence, or with parents [B, tree_nodes] (as in kvq_tree)
 *                start + depth(i) for i < tree_nodes; 0 behind the last
 * seq_lens may be held_lens or start_lens itself, free_left free_count itself
 * (in place); otherwise outputs overlap neither an input nor one another
 * (refused).  A page id outside [0, num_blocks) is passed on as it is, sets
 * KVQ_DEVERR_BLOCK_ID, and its rows get slot -1; a free_count outside
 * [0, num_blocks], or more pages given back than the pool has, sets it too.
 * With batch 0 the [B] arrays may be NULL; with batch 0 and max_tokens 0 the
 * call does nothing.  batch <= 1024; max_tokens <= 2^30. */
typedef struct {
  int32_t batch;              /* B (<= 1024) */
  int32_t max_blocks_per_seq; /* block_table row length; capacity = it * block_size */
  int32_t num_blocks;         /* pool size in blocks; entries of free_blocks */
  int32_t block_size;         /* tokens per block (power of two >= 16) */
  int32_t max_tokens;         /* entries of slot_mapping and positions */
  int32_t tree_nodes;         /* row length of parents (<= KVQ_MAX_TREE_NODES); unused without parents */
} kvq_pages_params;

KVQ_API kvq_status kvq_pages_step(const kvq_pages_params* params, const int32_t* held_lens,
                                  const int32_t* start_lens, const int32_t* new_tokens, const int32_t* parents,
                                  int32_t* block_table, int32_t* free_blocks, const int32_t* free_count,
                                  int32_t* seq_lens, int32_t* free_left, int32_t* cu_seqlens,
                                  int64_t* slot_mapping, int64_t* positions, kvq_stream_t stream);

/* kvq_attend_noalloc -- kvq_decode then kvq_combine, with the split-partial
 * scratch in a library-owned 16 MiB device array instead of a caller
 * workspace.  The pages have no counterpart: this exists for callers that
 * cannot allocate device memory where they run attention (a plugin inside a
 * runtime that owns all device memory and offers no scratch allocator, or a
 * loop that must not pay cudaMalloc's implicit synchronization).  It allocates
 * and frees nothing.  Arguments and results are those of kvq_decode and
 * kvq_combine; KVQ_ERR_WORKSPACE_TOO_SMALL when the shapes need more than
 * 16 MiB of scratch (kvq_decode_workspace_size tells).  The first call on a
 * device looks up the array's device address (cudaGetSymbolAddress); make
 * that first call before any stream capture.  The array holds the previous
 * call's contents and is shared by all calls on the device: calls that
 * overlap on the GPU (different streams without ordering) race. */
KVQ_API kvq_status kvq_attend_noalloc(const kvq_cache* cache, const kvq_decode_params* params,
                                      const void* q, const int32_t* block_table,
                                      const int32_t* seq_lens, const float* head_sink, void* out,
                                      float* lse_out, kvq_stream_t stream);

/* kvq_check_wait_timeout -- failure-detection check of the bounded waits.
 * Launches one thread that waits on an mbarrier nothing ever arrives on, with
 * the same bounded wait the decode pipelines use (there bounded at 1.5 s),
 * here given limit_us microseconds (1 .. 2,000,000).  The wait gives up,
 * KVQ_DEVERR_TIMEOUT is set in the device flag word, and the context stays
 * usable: kvq_get_device_error then returns KVQ_ERR_DEVICE_TIMEOUT.  Nothing
 * is faulted or trapped.  Asynchronous on `stream`. */
KVQ_API kvq_status kvq_check_wait_timeout(uint32_t limit_us, kvq_stream_t stream);

/* Reads the current device's KVQ_DEVERR_* flag word into *flags (host).  This
 * call synchronizes `stream` before reading.  clear != 0 resets the word. */
KVQ_API kvq_status kvq_get_device_error(uint32_t* flags, int32_t clear, kvq_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* KVQ_H */
