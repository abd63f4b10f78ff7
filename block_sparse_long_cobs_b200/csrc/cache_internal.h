// Declarations of the cache and prompt kernels (include/cobs_cache.h).
#pragma once

#include "../../include/cobs_cache.h"
#include "cobs_internal.h"

namespace cobs {

// A cache as the kernels see it (contiguous when table is null).
struct CacheView {
  void* k;
  void* v;
  float* ks;               // E4M3 caches: one scale per row
  float* vs;
  const int32_t* table;    // [batch][table_stride] or null
  int64_t n_pages;
  int64_t cap;             // capacity_tokens
  int32_t table_stride;
  int32_t hkv;
  int32_t format;          // COBS_CACHE_*
};

struct AppendArgs {
  CacheView c;
  cobs_rope rope;          // rotary_dim 0: nothing is rotated
  const uint16_t* q;       // null: keys and values only
  const uint16_t* k;
  const uint16_t* v;
  int64_t q_stride, k_stride, v_stride;   // elements between rows
  uint16_t* q_out;         // [n_tokens][hq][d]
  const int32_t* cu;       // [batch + 1] or null (one token per sequence)
  const int64_t* start;    // [batch]
  int32_t* status;
  int64_t n_tokens;
  int32_t batch, hq, d;    // hq 0 when q is null
  int32_t rows_per_warp;   // head rows of one token that a warp takes
  int32_t chunks;          // warps per token
};

struct ReadArgs {
  CacheView c;
  const int64_t* seq_lens; // [batch] or null
  uint16_t* k_out;         // [batch * n][hkv][64][d] or null
  uint16_t* v_out;
  int32_t* status;
  int64_t block_begin, n;  // blocks per sequence
  int32_t batch, d;
};

struct PromptArgs {
  CacheView c;
  const uint16_t* q;       // [n_tokens][hq][d]
  const int32_t* cu;       // [batch + 1] or null (one token per sequence)
  const int64_t* seq_lens; // [batch]
  uint16_t* out;           // [n_tokens][hq][d]
  float* lse;              // [n_tokens][hq] or null
  float* partials;         // notes and rows of units that were cut
  int32_t* status;
  int64_t n_tokens, max_seq_len;
  int32_t batch, hq, d;
  float scale_log2;        // softmax_scale * log2(e)
};

cudaError_t launch_append(const AppendArgs& a, cudaStream_t stream);
cudaError_t launch_read_cache(const ReadArgs& a, cudaStream_t stream);
cudaError_t launch_prompt(const PromptArgs& a, cudaStream_t stream);
size_t prompt_partial_bytes(const cobs_dims* d, int64_t n_tokens, int64_t max_seq_len);
// decode over an E4M3 cache: d.k / d.v hold codes, ks / vs the row scales
cudaError_t launch_decode_e4m3(const DecodeArgs& d, const float* ks, const float* vs,
                               cudaStream_t stream);

}  // namespace cobs
