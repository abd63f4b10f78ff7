// Device helpers of the cache and prompt kernels: rows of a cache, sequences
// of packed tokens, E4M3 codes.
#pragma once

#include <cuda_fp8.h>

#include "cache_internal.h"
#include "device_common.cuh"

namespace cobs {

// Row (in rows of d components) of token `pos` of (sequence b, kv-head h);
// -1 where the cache has no place for it.
__device__ __forceinline__ int64_t cache_row(const CacheView& c, int64_t b, int h, int64_t pos) {
  if (pos < 0 || pos >= c.cap) return -1;
  if (c.table == nullptr) return (b * c.hkv + h) * c.cap + pos;
  const int64_t j = pos / kBlock;
  if (j >= c.table_stride) return -1;
  const int32_t page = __ldg(c.table + b * c.table_stride + j);
  if (page < 0 || page >= c.n_pages) return -1;
  return (int64_t(page) * c.hkv + h) * kBlock + pos % kBlock;
}

// Sequence of packed row i: the b with cu[b] <= i < cu[b + 1], `batch` when
// the row belongs to nobody (i >= cu[batch]).  Whole warp, i warp-uniform:
// each step looks at 32 evenly spaced bounds of the range that is left.
__device__ __forceinline__ int warp_find_sequence(const int32_t* cu, int batch, int64_t i,
                                                  int lane) {
  if (cu == nullptr) return int(i < batch ? i : batch);
  int lo = 0, n = batch;   // the number of ends cu[b + 1] <= i is lo + [0, n]
  while (n > 0) {
    const int step = (n + 31) / 32;
    const int at = lo + (lane + 1) * step;       // ends below this one
    const bool below = at <= lo + n && int64_t(__ldg(cu + at)) <= i;
    const int k = __popc(__ballot_sync(0xffffffffu, below));
    lo += k * step;
    // the answer lies in the next group of `step` ends, its last one above i
    const int left = n - k * step;
    n = left < step ? left : step - 1;
  }
  return lo;
}

// Bounded mbarrier wait like wait_or_abort, for waits on the critical path:
// the clock is first read after 64 tries (reading the global timer on every
// wait that does not succeed at once adds its latency to each step of a
// pipeline).
__device__ __forceinline__ bool wait_step(uint64_t* bar, uint32_t parity, int32_t* status,
                                          volatile int* abort_flag) {
  uint64_t t0 = 0;
  for (uint32_t it = 1; !mbar_try_wait(bar, parity); ++it) {
    if ((it & 63u) == 0) {
      if (*abort_flag) return false;
      const uint64_t now = global_timer_ns();
      if (t0 == 0) {
        t0 = now;
      } else if (now - t0 > kWaitLimitNs) {
        report(status, COBS_ERR_TIMEOUT);
        *abort_flag = 1;
        return false;
      }
    }
  }
  return true;
}

// Packed fp32 pairs.
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// Two fp32 -> packed bf16 (low half: x), nearest even, NaN kept.
__device__ __forceinline__ uint32_t bf16x2_bits(float x, float y) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(y), "f"(x));
  return r;
}

// Two floats -> two E4M3 codes (low byte: x), nearest even, saturating.
__device__ __forceinline__ uint32_t e4m3x2(float x, float y) {
  return __nv_cvt_float2_to_fp8x2(make_float2(x, y), __NV_SATFINITE, __NV_E4M3);
}
// Two E4M3 codes (low byte first) -> fp32 (exact).
__device__ __forceinline__ float2 e4m3x2_to_float2(uint32_t codes) {
  return __half22float2(__half2(
      __nv_cvt_fp8x2_to_halfraw2(__nv_fp8x2_storage_t(codes & 0xffffu), __NV_E4M3)));
}

}  // namespace cobs
