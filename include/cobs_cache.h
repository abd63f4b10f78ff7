/* Cache and prompt calls of the COBS library: putting tokens into the KV
 * cache (rotary positions, bf16 or E4M3 storage), attention of a prompt or
 * of an appended chunk over the cache, reading an E4M3 cache back as bf16
 * pages, and the sparse decode over either kind of cache.
 *
 * With the calls of cobs.h they form one path: cobs_append_tokens writes the
 * new tokens' keys and values, cobs_prompt_attention computes the new tokens'
 * attention, cobs_build_block_stats(_paged) makes the records of the blocks
 * that became complete, and every decode step appends one token, selects and
 * decodes.  With an E4M3 cache, cobs_read_cache gives the bf16 pages that the
 * statistics and the prompt attention read.
 *
 * Everything cobs.h says of its calls holds here: streams, ownership (the
 * caller owns all memory, nothing is allocated), host checks before any
 * launch, the status word of the workspace, cobs_last_error(), 16-byte
 * alignment of every device pointer, and thread safety.  The kernels launch
 * on the current device, which must be the one the pointers belong to: a
 * buffer that begins in another device's memory, or in host memory that the
 * CUDA runtime does not know, is refused (INVALID_ARG).
 * The calls can be captured into CUDA graphs.
 *
 * One workspace, initialised once with cobs_workspace_init, may serve all
 * calls of the same batch and num_kv_heads, those of cobs.h among them, when it
 * is as large as the largest of cobs_workspace_bytes and
 * cobs_prompt_workspace_bytes asks for.  Where its counters lie depends on
 * batch and num_kv_heads: selection, decode and prompt attention of another
 * batch or other kv-heads need another workspace, or this one initialised
 * again.  (cobs_append_tokens and cobs_read_cache use the status word alone.)
 *
 * Packed tokens.  n_tokens rows hold the new tokens of all sequences, one
 * sequence after the other; cu_tokens (device int32 [batch + 1], ascending
 * from 0) gives sequence b the rows [cu_tokens[b], cu_tokens[b + 1]).  A
 * sequence may have no row.  Rows before cu_tokens[0] and rows at or past
 * cu_tokens[batch] belong to nobody: they reach no result and their outputs are
 * left as they were.  Bounds that point outside [0, n_tokens] are cut to it, and
 * reported as COBS_ERR_DEVICE, as are bounds that descend.
 * cu_tokens NULL: one token per sequence, n_tokens == batch.  With n_tokens 0
 * (or no blocks to read) nothing is done, and buffers of rows may be NULL. */
#ifndef COBS_CACHE_H_
#define COBS_CACHE_H_

#include "cobs.h"

#ifdef __cplusplus
extern "C" {
#endif

#define COBS_CACHE_BF16 0   /* keys and values in bf16                        */
#define COBS_CACHE_E4M3 1   /* E4M3 codes and one fp32 scale per row (below)  */

/* A KV cache, contiguous (block_table NULL) or paged:
 *   k, v          [batch][num_kv_heads][capacity_tokens][d], or page pools
 *                 [n_pages][num_kv_heads][B][d]; bf16, or E4M3 codes (one
 *                 byte each)
 *   k_scale,      COBS_CACHE_E4M3: fp32 [batch][num_kv_heads]
 *   v_scale       [capacity_tokens], or [n_pages][num_kv_heads][B]
 *   block_table   device int32 [batch][table_stride]: the page of block j of
 *                 sequence b; a negative entry is a block without a page
 * An E4M3 row (one token of one kv-head) stores scale = max |x| / 448 over
 * its finite components, and per component the code of the fp32 quotient
 * x / scale, rounded to nearest, ties to even; the value it stands for is
 * code * scale.  A row whose largest finite magnitude is below 448 * 2^-126
 * stores scale 0 and zero codes; a component that is not finite stores the NaN
 * code. */
typedef struct cobs_kv_cache {
  void* k;
  void* v;
  float* k_scale;
  float* v_scale;
  const int32_t* block_table;
  int64_t n_pages;
  int32_t table_stride;
  int32_t format;             /* COBS_CACHE_BF16 or COBS_CACHE_E4M3           */
} cobs_kv_cache;

/* Scaling of the rotary frequencies for long contexts. */
#define COBS_ROPE_PLAIN 0     /* f_t = base^(-2 t / rotary_dim)               */
#define COBS_ROPE_LINEAR 1    /* f_t / factor                                 */
#define COBS_ROPE_BY_PARTS 2  /* f_t (g + (1 - g) / factor), where
                                 g = clamp((turns - low) / (high - low), 0, 1)
                                 and turns = original_context f_t / (2 pi), the
                                 turns pair t makes over the original context:
                                 fast pairs keep their frequency, slow ones are
                                 interpolated                                  */
#define COBS_ROPE_CUSTOM 3    /* frequencies[t], radians per token            */

typedef struct cobs_rope_params {
  int32_t rotary_dim;         /* leading dimensions that are rotated: a
                                 multiple of 8, 0 <= rotary_dim <= 128          */
  int32_t interleaved;        /* 0: pairs (t, t + rotary_dim / 2);
                                 1: pairs (2 t, 2 t + 1)                        */
  int32_t scaling;            /* COBS_ROPE_*                                    */
  int32_t reserved;           /* 0                                              */
  double base;                /* > 1                                            */
  double factor;              /* LINEAR, BY_PARTS: >= 1                         */
  double original_context;    /* BY_PARTS: > 0                                  */
  double low, high;           /* BY_PARTS: 0 <= low < high                      */
  double attention_factor;    /* cos and sin are multiplied by it, > 0          */
  const double* frequencies;  /* CUSTOM: host [rotary_dim / 2], 0 <= f <= pi    */
} cobs_rope_params;

/* A rotary table, filled by cobs_rope_init and kept by the caller (host
 * memory, plain data): the turns pair t makes per token in units of 2^-64, so
 * that position times turns modulo 2^64 is the fraction of a turn with no
 * rounding that grows with the position. */
typedef struct cobs_rope {
  int32_t rotary_dim;
  int32_t interleaved;
  float attention_factor;
  int32_t reserved;
  uint64_t turns[64];
} cobs_rope;

/* Fill *rope from *params (host only, no GPU work).
 * Errors: INVALID_ARG. */
COBS_API cobs_status cobs_rope_init(const cobs_rope_params* params, cobs_rope* rope);

/* Rotate the queries and keys of the packed new tokens and store their keys
 * and values in the cache:
 *   position of row i of sequence b = start[b] + i - cu_tokens[b]
 *   (y1, y2) = attention_factor * (x1 cos a - x2 sin a, x2 cos a + x1 sin a),
 *   a = position * f_t, for every rotated pair; the other dimensions are
 *   copied.  q_out and a bf16 cache hold the result rounded to bf16; an E4M3
 *   cache is coded from the unrounded fp32 result.  Values are not rotated.
 *   rope        NULL: nothing is rotated (q, if given, is copied)
 *   q, k, v     device bf16, rows of [num_q_heads][d] or [num_kv_heads][d];
 *               row i starts at element i * q_stride (k_stride, v_stride), so
 *               that the parts of one fused projection can be given.  Strides
 *               are multiples of 8 and at least a row.  q may be NULL (keys
 *               and values only), then q_out is NULL too.
 *   start       device int64 [batch]: tokens already in each sequence's cache
 *   q_out       device bf16 [n_tokens][num_q_heads][d]; may be q itself when
 *               q_stride is num_q_heads * d, otherwise it overlaps no input
 * Cache rows of other positions are left as they were.  A token whose
 * position lies outside [0, capacity_tokens), whose block lies past
 * table_stride, has no page, or names a page >= n_pages, is not stored and
 * is reported as COBS_ERR_DEVICE through the status word (its query is still
 * rotated).  Two tokens must not name the same cache row.
 * ws: status word only (256 bytes).
 * Errors: INVALID_ARG, UNSUPPORTED, WORKSPACE, CUDA. */
COBS_API cobs_status cobs_append_tokens(const cobs_dims* dims, const cobs_kv_cache* cache,
                                        const cobs_rope* rope, const void* q, int64_t q_stride,
                                        const void* k, int64_t k_stride, const void* v,
                                        int64_t v_stride, const int32_t* cu_tokens,
                                        int64_t n_tokens, const int64_t* start, void* q_out,
                                        void* ws, size_t ws_bytes, void* stream);

/* Read blocks [block_begin, block_end) of every sequence out of a cache of
 * either format as bf16 pages:
 *   k_out, v_out  device bf16 [batch * n][num_kv_heads][B][d] with
 *                 n = block_end - block_begin; block j of sequence b is page
 *                 b * n + j - block_begin.  Either may be NULL (not both).
 *                 These are page pools for cobs_build_block_stats_paged and
 *                 cobs_prompt_attention with a table that says so.
 *   seq_lens      device int64 [batch] or NULL: rows at or past a sequence's
 *                 length are left as they were (NULL: every row is read)
 * A value is code * scale in fp32, rounded to bf16 (bf16 caches: copied).  A
 * block without a page is left as it was; a page >= n_pages too, and is
 * reported as COBS_ERR_DEVICE.  ws: status word only (256 bytes).
 * Errors: INVALID_ARG, UNSUPPORTED, WORKSPACE, CUDA. */
COBS_API cobs_status cobs_read_cache(const cobs_dims* dims, const cobs_kv_cache* cache,
                                     const int64_t* seq_lens, int64_t block_begin,
                                     int64_t block_end, void* k_out, void* v_out, void* ws,
                                     size_t ws_bytes, void* stream);

/* Bytes of workspace that cobs_prompt_attention needs for up to n_tokens
 * packed rows over sequences of up to max_seq_len tokens (the status word, room
 * for the counters of the selection and the decode, and the partial results of
 * split rows; it does not depend on the device).
 * Returns 0 (and sets the last error) for invalid arguments. */
COBS_API size_t cobs_prompt_workspace_bytes(const cobs_dims* dims, int64_t n_tokens,
                                            int64_t max_seq_len);

/* Causal attention of the packed new tokens over the cache that already holds
 * them: row i of sequence b with c = cu_tokens[b + 1] - cu_tokens[b] rows has
 * position p = seq_lens[b] - c + i - cu_tokens[b] and attends to the tokens
 * [0, p]:
 *   out = softmax(q K^T * softmax_scale) V, lse = ln sum exp(q K^T *
 *   softmax_scale), per query head over its kv-head.
 *   cache        COBS_CACHE_BF16 (an E4M3 cache: UNSUPPORTED, read it back
 *                with cobs_read_cache); contiguous or paged
 *   q            device bf16 [n_tokens][num_q_heads][d]
 *   seq_lens     device int64 [batch]: tokens of each sequence in the cache,
 *                the new ones among them, each in [0, max_seq_len] (a value
 *                outside is clamped and reported as COBS_ERR_DEVICE)
 *   max_seq_len  host bound of every length, in [1, capacity_tokens]
 *   out          device bf16 [n_tokens][num_q_heads][d]
 *   lse          device fp32 [n_tokens][num_q_heads] or NULL
 * A row with a negative position (more rows than tokens) attends to nothing:
 * out 0, lse -inf.  A row one of whose logits is NaN or +inf (its query, or a
 * product with it, is not finite) is NaN in out and lse; one whose logits are
 * all -inf is as one without keys.  Keys and values at or past a sequence's
 * length are never read into a result, whatever they hold.  Keys and values
 * inside a sequence must be finite: a value that is not may also reach rows up
 * to 382 tokens before it.  A block inside a sequence whose page is missing or
 * >= n_pages counts as tokens that are not there, and is reported as
 * COBS_ERR_DEVICE.  Weights are rounded to bf16 before they meet the values
 * (off by 2^-8 of each at most), not before they are summed.
 *   ws           at least cobs_prompt_workspace_bytes(dims, n_tokens,
 *                max_seq_len), initialised once with cobs_workspace_init;
 *                calls that share it must not overlap on the GPU
 * Errors: INVALID_ARG, UNSUPPORTED, WORKSPACE, CUDA. */
COBS_API cobs_status cobs_prompt_attention(const cobs_dims* dims, const cobs_kv_cache* cache,
                                           const void* q, const int32_t* cu_tokens,
                                           int64_t n_tokens, const int64_t* seq_lens,
                                           int64_t max_seq_len, float softmax_scale, void* out,
                                           float* lse, void* ws, size_t ws_bytes, void* stream);

/* cobs_sparse_decode over a cache of either format, contiguous or paged:
 * arguments, list checks, results and workspace (cobs_workspace_bytes) as
 * there; seq_lens as in cobs_sparse_decode_varlen, or NULL (every sequence is
 * max_seq_len tokens long).  A bf16 cache runs the kernels of
 * cobs_sparse_decode(_varlen, _paged), bit for bit.  Over an E4M3 cache
 *   logit_j = softmax_scale * k_scale_j * (q . k_code_j),
 *   out = sum_j e^(logit_j - m) v_scale_j v_code_j / sum_j e^(logit_j - m),
 * with q split into three E4M3 parts that hold every component exactly down
 * to 2^-16 of the row's largest (components below it are rounded by at most
 * 2^-24 of the largest), and each weight e^(logit_j - m) v_scale_j rounded by
 * at most 2^-16 of itself or 2^-24 of the pair's largest, whichever is more.
 * A query row with a component that is not finite is NaN in out and lse.  Codes
 * of tokens inside a sequence must not be NaN, and their scales must be as
 * cobs_append_tokens stores them: 0, or finite and at least 2^-126.
 * Errors: INVALID_ARG, UNSUPPORTED, WORKSPACE, CUDA. */
COBS_API cobs_status cobs_sparse_decode_cache(const cobs_dims* dims, const cobs_kv_cache* cache,
                                              const void* q, const int32_t* idx,
                                              const int32_t* n_sel, int32_t idx_stride,
                                              const int64_t* seq_lens, int64_t max_seq_len,
                                              float softmax_scale, float* out, float* lse,
                                              void* ws, size_t ws_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* COBS_CACHE_H_ */
