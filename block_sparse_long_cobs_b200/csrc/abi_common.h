// Host helpers shared by the C-ABI files: error reporting and the checks that
// every call makes before it touches the GPU.
#pragma once

#include "cobs_internal.h"

namespace cobs {

// Smallest workspace: the status word and its padding.
constexpr size_t kStatusBytes = 256;

// Set the thread's last error and return st; ok() clears it.
cobs_status fail(cobs_status st, const char* fmt, ...);
cobs_status ok();
cobs_status cuda_fail(cudaError_t e, const char* what);

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
inline size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

cobs_status check_dims(const cobs_dims* d);
cobs_status check_ws(void* ws, size_t have, size_t need);

// block_table null: the contiguous cache [batch, Hkv, capacity_tokens, d];
// else a page pool [n_pages, Hkv, 64, d] addressed through the table.
cobs_status check_paging(const cobs_dims* dims, const int32_t* block_table, int32_t table_stride,
                         int64_t n_pages, int64_t blocks_needed);

WorkspaceLayout layout(const cobs_dims* d, int32_t n_sel_max);

// Checked launch arguments of a decode (block_table null: contiguous caches;
// seq_lens null: every sequence is seq_len tokens long).
cobs_status decode_args(const cobs_dims* dims, const void* q, const void* k, const void* v,
                        const int32_t* block_table, int32_t table_stride, int64_t n_pages,
                        const int32_t* idx, const int32_t* n_sel, int32_t idx_stride,
                        const int64_t* seq_lens, int64_t seq_len, float softmax_scale,
                        float* out, float* lse, void* ws, size_t ws_bytes, DecodeArgs* args);

}  // namespace cobs
