// C ABI of the cache and prompt calls (include/cobs_cache.h): argument checks
// and launch arguments.  Everything that can be checked on the host is
// checked here, before any CUDA call.
#include <cmath>
#include <cuda.h>
#include <initializer_list>

#include "abi_common.h"
#include "cache_internal.h"

using namespace cobs;

namespace {

constexpr int64_t kMaxRows = int64_t(1) << 31;

// Descriptor of a cache whose blocks [0, blocks) a call may address.
cobs_status check_cache(const cobs_dims* dims, const cobs_kv_cache* c, int64_t blocks) {
  if (!c) return fail(COBS_ERR_INVALID_ARG, "cache is NULL");
  if (c->format != COBS_CACHE_BF16 && c->format != COBS_CACHE_E4M3)
    return fail(COBS_ERR_INVALID_ARG, "cache format must be COBS_CACHE_BF16 or _E4M3 (got %d)",
                int(c->format));
  if (!c->k || !c->v) return fail(COBS_ERR_INVALID_ARG, "cache k and v must not be NULL");
  if (!aligned16(c->k) || !aligned16(c->v))
    return fail(COBS_ERR_INVALID_ARG, "cache pointers must be 16-byte aligned");
  if (c->format == COBS_CACHE_E4M3) {
    if (!c->k_scale || !c->v_scale)
      return fail(COBS_ERR_INVALID_ARG, "an E4M3 cache needs k_scale and v_scale");
    if (!aligned16(c->k_scale) || !aligned16(c->v_scale))
      return fail(COBS_ERR_INVALID_ARG, "cache pointers must be 16-byte aligned");
  }
  return check_paging(dims, c->block_table, c->table_stride, c->n_pages, blocks);
}

CacheView view_of(const cobs_dims* dims, const cobs_kv_cache* c) {
  CacheView v{};
  v.k = c->k;
  v.v = c->v;
  v.ks = c->k_scale;
  v.vs = c->v_scale;
  v.table = c->block_table;
  v.n_pages = c->n_pages;
  v.cap = dims->capacity_tokens;
  v.table_stride = c->table_stride;
  v.hkv = dims->num_kv_heads;
  v.format = c->format;
  return v;
}

// Number of packed rows.
cobs_status check_count(const cobs_dims* dims, int64_t n_tokens) {
  if (n_tokens < 0) return fail(COBS_ERR_INVALID_ARG, "n_tokens must be >= 0");
  if (n_tokens > (kMaxRows - 1) / (int64_t(dims->num_q_heads) + 2 * int64_t(dims->num_kv_heads)))
    return fail(COBS_ERR_UNSUPPORTED, "n_tokens * head rows must be < 2^31");
  return COBS_OK;
}

// Packed rows of new tokens.
cobs_status check_tokens(const cobs_dims* dims, const int32_t* cu_tokens, int64_t n_tokens) {
  const cobs_status st = check_count(dims, n_tokens);
  if (st != COBS_OK) return st;
  if (cu_tokens && !aligned16(cu_tokens))
    return fail(COBS_ERR_INVALID_ARG, "cu_tokens must be 16-byte aligned");
  if (!cu_tokens && n_tokens != dims->batch)
    return fail(COBS_ERR_INVALID_ARG,
                "without cu_tokens there is one token per sequence: n_tokens %lld, batch %d",
                (long long)n_tokens, dims->batch);
  return COBS_OK;
}

cobs_status check_rows(const char* name, const void* p, int64_t stride, int64_t row) {
  if (!p || !aligned16(p))
    return fail(COBS_ERR_INVALID_ARG, "%s must not be NULL and must be 16-byte aligned", name);
  if (stride % 8 != 0 || stride < row || stride >= (int64_t(1) << 31))
    return fail(COBS_ERR_INVALID_ARG,
                "%s_stride %lld must be a multiple of 8 and at least a row of %lld", name,
                (long long)stride, (long long)row);
  return COBS_OK;
}

// Whether every buffer of a call (null: not given) is memory of the current
// device, or memory that it can reach: the last check before a launch.  A host
// pointer, or another device's, would fault in the kernel.
struct Buffer {
  const char* name;
  const void* p;
};
// The driver's query of one attribute: 28 ns a buffer, where the runtime's of
// all takes 66, and a call has up to twelve.  (Null: not found.)
typedef CUresult (*PointerAttributeFn)(void*, CUpointer_attribute, CUdeviceptr);
PointerAttributeFn pointer_attribute_fn() {
  static const PointerAttributeFn fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q{};
    if (cudaGetDriverEntryPoint("cuPointerGetAttribute", &p, cudaEnableDefault, &q) !=
            cudaSuccess ||
        q != cudaDriverEntryPointSuccess) {
      (void)cudaGetLastError();
      p = nullptr;
    }
    return reinterpret_cast<PointerAttributeFn>(p);
  }();
  return fn;
}

cobs_status check_device(std::initializer_list<Buffer> buffers) {
  const PointerAttributeFn ask = pointer_attribute_fn();
  int dev = 0;
  bool known = cudaGetDevice(&dev) == cudaSuccess;
  for (const Buffer& x : buffers) {
    if (!x.p) continue;
    int on = -1;
    if (known && ask &&
        ask(&on, CU_POINTER_ATTRIBUTE_DEVICE_ORDINAL, reinterpret_cast<CUdeviceptr>(x.p)) ==
            CUDA_SUCCESS &&
        on == dev)
      continue;
    cudaPointerAttributes at{};
    known = known && cudaPointerGetAttributes(&at, x.p) == cudaSuccess;
    if (!known || at.type == cudaMemoryTypeUnregistered) {
      (void)cudaGetLastError();   // not sticky: leave no error behind
      return fail(COBS_ERR_INVALID_ARG, "%s is not a device pointer", x.name);
    }
    if (at.type == cudaMemoryTypeDevice && at.device != dev)
      return fail(COBS_ERR_INVALID_ARG, "%s lies on device %d, the current device is %d", x.name,
                  at.device, dev);
  }
  return COBS_OK;
}

// A cache's scales, where its format has them.
const void* scale_of(const cobs_kv_cache* c, const float* s) {
  return c->format == COBS_CACHE_E4M3 ? s : nullptr;
}

}  // namespace

extern "C" {

cobs_status cobs_rope_init(const cobs_rope_params* p, cobs_rope* rope) {
  if (!p || !rope) return fail(COBS_ERR_INVALID_ARG, "params and rope must not be NULL");
  if (p->rotary_dim < 0 || p->rotary_dim > 128 || p->rotary_dim % 8 != 0)
    return fail(COBS_ERR_INVALID_ARG, "rotary_dim must be a multiple of 8 in [0, 128] (got %d)",
                p->rotary_dim);
  if (p->interleaved != 0 && p->interleaved != 1)
    return fail(COBS_ERR_INVALID_ARG, "interleaved must be 0 or 1");
  if (p->reserved != 0) return fail(COBS_ERR_INVALID_ARG, "reserved must be 0");
  if (p->scaling < COBS_ROPE_PLAIN || p->scaling > COBS_ROPE_CUSTOM)
    return fail(COBS_ERR_INVALID_ARG, "scaling must be one of COBS_ROPE_* (got %d)", p->scaling);
  if (!std::isfinite(p->attention_factor) || !(p->attention_factor > 0.0) ||
      p->attention_factor > 1e30)
    return fail(COBS_ERR_INVALID_ARG, "attention_factor must be finite and > 0");
  const bool custom = p->scaling == COBS_ROPE_CUSTOM;
  if (!custom && (!std::isfinite(p->base) || !(p->base > 1.0)))
    return fail(COBS_ERR_INVALID_ARG, "base must be finite and > 1");
  if ((p->scaling == COBS_ROPE_LINEAR || p->scaling == COBS_ROPE_BY_PARTS) &&
      (!std::isfinite(p->factor) || !(p->factor >= 1.0)))
    return fail(COBS_ERR_INVALID_ARG, "factor must be finite and >= 1");
  if (p->scaling == COBS_ROPE_BY_PARTS &&
      (!std::isfinite(p->original_context) || !(p->original_context > 0.0) ||
       !std::isfinite(p->high) || !(p->low >= 0.0) || !(p->high > p->low)))
    return fail(COBS_ERR_INVALID_ARG, "BY_PARTS needs original_context > 0 and 0 <= low < high");
  if (custom && p->rotary_dim > 0 && !p->frequencies)
    return fail(COBS_ERR_INVALID_ARG, "COBS_ROPE_CUSTOM needs frequencies");
  constexpr long double kTwoPi = 6.283185307179586476925286766559L;
  cobs_rope r{};
  r.rotary_dim = p->rotary_dim;
  r.interleaved = p->interleaved;
  r.attention_factor = float(p->attention_factor);
  for (int t = 0; t < p->rotary_dim / 2; ++t) {
    long double f;
    if (custom) {
      const double g = p->frequencies[t];
      if (!std::isfinite(g) || g < 0.0 || g > 3.1415926535897932)
        return fail(COBS_ERR_INVALID_ARG, "frequency %d outside [0, pi]", t);
      f = g;
    } else {
      f = powl(p->base, -2.0L * t / p->rotary_dim);
    }
    if (p->scaling == COBS_ROPE_LINEAR) f /= p->factor;
    if (p->scaling == COBS_ROPE_BY_PARTS) {
      long double g = (p->original_context * f / kTwoPi - p->low) / (p->high - p->low);
      g = g < 0.0L ? 0.0L : (g > 1.0L ? 1.0L : g);
      f = f * g + f / p->factor * (1.0L - g);
    }
    r.turns[t] = uint64_t(llroundl(f / kTwoPi * 18446744073709551616.0L));
  }
  *rope = r;
  return ok();
}

cobs_status cobs_append_tokens(const cobs_dims* dims, const cobs_kv_cache* cache,
                               const cobs_rope* rope, const void* q, int64_t q_stride,
                               const void* k, int64_t k_stride, const void* v, int64_t v_stride,
                               const int32_t* cu_tokens, int64_t n_tokens, const int64_t* start,
                               void* q_out, void* ws, size_t ws_bytes, void* stream) {
  cobs_status st = check_dims(dims);
  if (st != COBS_OK) return st;
  if ((st = check_tokens(dims, cu_tokens, n_tokens)) != COBS_OK) return st;
  // a table shorter than the capacity is allowed: tokens past it are reported
  if ((st = check_cache(dims, cache, 0)) != COBS_OK) return st;
  const int64_t kv_row = int64_t(dims->num_kv_heads) * dims->head_dim;
  const int64_t q_row = int64_t(dims->num_q_heads) * dims->head_dim;
  if (n_tokens > 0) {   // (empty tensors have no address)
    if ((st = check_rows("k", k, k_stride, kv_row)) != COBS_OK) return st;
    if ((st = check_rows("v", v, v_stride, kv_row)) != COBS_OK) return st;
    if (q) {
      if ((st = check_rows("q", q, q_stride, q_row)) != COBS_OK) return st;
      if (!q_out || !aligned16(q_out))
        return fail(COBS_ERR_INVALID_ARG, "q_out must not be NULL and must be 16-byte aligned");
      if (q_out == q && q_stride != q_row)
        return fail(COBS_ERR_INVALID_ARG, "in place, q_stride must be num_q_heads * head_dim");
    } else if (q_out) {
      return fail(COBS_ERR_INVALID_ARG, "q_out without q");
    }
  }
  if (!start || !aligned16(start))
    return fail(COBS_ERR_INVALID_ARG, "start must not be NULL and must be 16-byte aligned");
  if (rope) {
    if (rope->rotary_dim < 0 || rope->rotary_dim > dims->head_dim || rope->rotary_dim % 8 != 0)
      return fail(COBS_ERR_INVALID_ARG, "rotary_dim %d is not a multiple of 8 in [0, head_dim]",
                  rope->rotary_dim);
    if (!std::isfinite(rope->attention_factor))
      return fail(COBS_ERR_INVALID_ARG, "attention_factor must be finite");
  }
  if ((st = check_ws(ws, ws_bytes, kStatusBytes)) != COBS_OK) return st;
  if (n_tokens == 0) return ok();
  st = check_device({{"cache k", cache->k}, {"cache v", cache->v},
                     {"k_scale", scale_of(cache, cache->k_scale)},
                     {"v_scale", scale_of(cache, cache->v_scale)},
                     {"block_table", cache->block_table}, {"q", q}, {"k", k}, {"v", v},
                     {"cu_tokens", cu_tokens}, {"start", start}, {"q_out", q_out}, {"ws", ws}});
  if (st != COBS_OK) return st;
  AppendArgs a{};
  a.c = view_of(dims, cache);
  if (rope) a.rope = *rope;
  a.q = static_cast<const uint16_t*>(q);
  a.k = static_cast<const uint16_t*>(k);
  a.v = static_cast<const uint16_t*>(v);
  a.q_stride = q_stride;
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  a.q_out = static_cast<uint16_t*>(q_out);
  a.cu = cu_tokens;
  a.start = start;
  a.status = static_cast<int32_t*>(ws);
  a.n_tokens = n_tokens;
  a.batch = dims->batch;
  a.hq = q ? dims->num_q_heads : 0;
  a.d = dims->head_dim;
  const cudaError_t e = launch_append(a, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "append launch");
  return ok();
}

cobs_status cobs_read_cache(const cobs_dims* dims, const cobs_kv_cache* cache,
                            const int64_t* seq_lens, int64_t block_begin, int64_t block_end,
                            void* k_out, void* v_out, void* ws, size_t ws_bytes, void* stream) {
  cobs_status st = check_dims(dims);
  if (st != COBS_OK) return st;
  const int64_t nb_cap = dims->capacity_tokens / kBlock;
  if (block_begin < 0 || block_end < block_begin || block_end > nb_cap)
    return fail(COBS_ERR_INVALID_ARG, "block range [%lld, %lld) outside [0, %lld]",
                (long long)block_begin, (long long)block_end, (long long)nb_cap);
  if ((st = check_cache(dims, cache, block_end)) != COBS_OK) return st;
  if (!k_out && !v_out && block_end > block_begin)
    return fail(COBS_ERR_INVALID_ARG, "k_out and v_out are both NULL");
  if ((k_out && !aligned16(k_out)) || (v_out && !aligned16(v_out)) ||
      (seq_lens && !aligned16(seq_lens)))
    return fail(COBS_ERR_INVALID_ARG, "device pointers must be 16-byte aligned");
  if ((st = check_ws(ws, ws_bytes, kStatusBytes)) != COBS_OK) return st;
  if (block_end == block_begin) return ok();
  st = check_device({{"cache k", cache->k}, {"cache v", cache->v},
                     {"k_scale", scale_of(cache, cache->k_scale)},
                     {"v_scale", scale_of(cache, cache->v_scale)},
                     {"block_table", cache->block_table}, {"seq_lens", seq_lens},
                     {"k_out", k_out}, {"v_out", v_out}, {"ws", ws}});
  if (st != COBS_OK) return st;
  ReadArgs a{};
  a.c = view_of(dims, cache);
  a.seq_lens = seq_lens;
  a.k_out = static_cast<uint16_t*>(k_out);
  a.v_out = static_cast<uint16_t*>(v_out);
  a.status = static_cast<int32_t*>(ws);
  a.block_begin = block_begin;
  a.n = block_end - block_begin;
  a.batch = dims->batch;
  a.d = dims->head_dim;
  const cudaError_t e = launch_read_cache(a, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "cache read launch");
  return ok();
}

static cobs_status check_prompt_sizes(const cobs_dims* dims, int64_t n_tokens,
                                      int64_t max_seq_len) {
  cobs_status st = check_dims(dims);
  if (st != COBS_OK) return st;
  if ((st = check_count(dims, n_tokens)) != COBS_OK) return st;
  if (max_seq_len < 1 || max_seq_len > dims->capacity_tokens)
    return fail(COBS_ERR_INVALID_ARG, "max_seq_len %lld outside [1, capacity_tokens]",
                (long long)max_seq_len);
  return COBS_OK;
}

// The split rows lie where the selection and the decode keep scores and their
// own partial rows, behind the counters that those calls leave for the next
// one: a workspace may serve them all.
static size_t prompt_partials_at(const cobs_dims* dims) { return layout(dims, 0).scores; }

static size_t prompt_need(const cobs_dims* dims, int64_t n_tokens, int64_t max_seq_len) {
  const size_t rows = prompt_partial_bytes(dims, n_tokens, max_seq_len);
  return rows == 0 ? kStatusBytes : prompt_partials_at(dims) + rows;
}

size_t cobs_prompt_workspace_bytes(const cobs_dims* dims, int64_t n_tokens, int64_t max_seq_len) {
  if (check_prompt_sizes(dims, n_tokens, max_seq_len) != COBS_OK) return 0;
  ok();
  return prompt_need(dims, n_tokens, max_seq_len);
}

cobs_status cobs_prompt_attention(const cobs_dims* dims, const cobs_kv_cache* cache,
                                  const void* q, const int32_t* cu_tokens, int64_t n_tokens,
                                  const int64_t* seq_lens, int64_t max_seq_len,
                                  float softmax_scale, void* out, float* lse, void* ws,
                                  size_t ws_bytes, void* stream) {
  cobs_status st = check_prompt_sizes(dims, n_tokens, max_seq_len);
  if (st != COBS_OK) return st;
  if ((st = check_tokens(dims, cu_tokens, n_tokens)) != COBS_OK) return st;
  if ((st = check_cache(dims, cache, ceil_div(max_seq_len, kBlock))) != COBS_OK) return st;
  if (cache->format != COBS_CACHE_BF16)
    return fail(COBS_ERR_UNSUPPORTED,
                "prompt attention reads a bf16 cache: read an E4M3 cache back with "
                "cobs_read_cache first");
  if (!seq_lens || (n_tokens > 0 && (!q || !out)))
    return fail(COBS_ERR_INVALID_ARG, "q, seq_lens and out must not be NULL");
  if (!aligned16(q) || !aligned16(seq_lens) || !aligned16(out) || (lse && !aligned16(lse)))
    return fail(COBS_ERR_INVALID_ARG, "device pointers must be 16-byte aligned");
  if (!(std::isfinite(softmax_scale)) || softmax_scale <= 0.f)
    return fail(COBS_ERR_INVALID_ARG, "softmax_scale must be finite and > 0");
  if ((st = check_ws(ws, ws_bytes, prompt_need(dims, n_tokens, max_seq_len))) != COBS_OK)
    return st;
  if (n_tokens == 0) return ok();
  st = check_device({{"cache k", cache->k}, {"cache v", cache->v},
                     {"block_table", cache->block_table}, {"q", q}, {"cu_tokens", cu_tokens},
                     {"seq_lens", seq_lens}, {"out", out}, {"lse", lse}, {"ws", ws}});
  if (st != COBS_OK) return st;
  PromptArgs a{};
  a.c = view_of(dims, cache);
  a.q = static_cast<const uint16_t*>(q);
  a.cu = cu_tokens;
  a.seq_lens = seq_lens;
  a.out = static_cast<uint16_t*>(out);
  a.lse = lse;
  a.partials = reinterpret_cast<float*>(static_cast<char*>(ws) + prompt_partials_at(dims));
  a.status = static_cast<int32_t*>(ws);
  a.n_tokens = n_tokens;
  a.max_seq_len = max_seq_len;
  a.batch = dims->batch;
  a.hq = dims->num_q_heads;
  a.d = dims->head_dim;
  a.scale_log2 = softmax_scale * 1.4426950408889634f;
  const cudaError_t e = launch_prompt(a, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "prompt attention launch");
  return ok();
}

cobs_status cobs_sparse_decode_cache(const cobs_dims* dims, const cobs_kv_cache* cache,
                                     const void* q, const int32_t* idx, const int32_t* n_sel,
                                     int32_t idx_stride, const int64_t* seq_lens,
                                     int64_t max_seq_len, float softmax_scale, float* out,
                                     float* lse, void* ws, size_t ws_bytes, void* stream) {
  cobs_status st = check_dims(dims);
  if (st != COBS_OK) return st;
  if (max_seq_len < 1 || max_seq_len > dims->capacity_tokens)
    return fail(COBS_ERR_INVALID_ARG, "max_seq_len %lld outside [1, capacity_tokens]",
                (long long)max_seq_len);
  if ((st = check_cache(dims, cache, ceil_div(max_seq_len, kBlock))) != COBS_OK) return st;
  DecodeArgs a{};
  st = decode_args(dims, q, cache->k, cache->v, cache->block_table, cache->table_stride,
                   cache->n_pages, idx, n_sel, idx_stride, seq_lens, max_seq_len, softmax_scale,
                   out, lse, ws, ws_bytes, &a);
  if (st != COBS_OK) return st;
  st = check_device({{"cache k", cache->k}, {"cache v", cache->v},
                     {"k_scale", scale_of(cache, cache->k_scale)},
                     {"v_scale", scale_of(cache, cache->v_scale)},
                     {"block_table", cache->block_table}, {"q", q}, {"idx", idx},
                     {"n_sel", n_sel}, {"seq_lens", seq_lens}, {"out", out}, {"lse", lse},
                     {"ws", ws}});
  if (st != COBS_OK) return st;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e = cache->format == COBS_CACHE_BF16
                            ? launch_decode(a, s)
                            : launch_decode_e4m3(a, cache->k_scale, cache->v_scale, s);
  if (e != cudaSuccess) return cuda_fail(e, "sparse decode launch");
  return ok();
}

}  // extern "C"
