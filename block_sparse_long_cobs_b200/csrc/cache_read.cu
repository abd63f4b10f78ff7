// Reading blocks of a cache back as bf16 pages (include/cobs_cache.h,
// cobs_read_cache): value = code * scale, rounded to bf16.
//
// Bound by memory (d + 4 bytes read and 2 d written per row).  One CTA per
// (block, kv-head): d / 8 lanes share a row, each with 8 codes.
#include "cache_device.cuh"

namespace cobs {
namespace {

constexpr int kReadThreads = 256;

template <int D, int kFormat>
__global__ void __launch_bounds__(kReadThreads) read_cache_kernel(const ReadArgs a) {
  constexpr int kLanes = D / 8;
  pdl_wait();
  pdl_launch_dependents();
  const int h = int(blockIdx.x % a.c.hkv);
  const int64_t page_out = blockIdx.x / a.c.hkv;      // batch * n pages
  const int64_t b = page_out / a.n, j = a.block_begin + page_out % a.n;
  int64_t rows = kBlock;
  if (a.seq_lens != nullptr) rows = min(rows, __ldg(a.seq_lens + b) - j * kBlock);
  int64_t row0;
  if (a.c.table == nullptr) {
    row0 = (b * a.c.hkv + h) * a.c.cap + j * kBlock;
  } else {
    const int32_t page = __ldg(a.c.table + b * a.c.table_stride + j);
    if (page >= a.c.n_pages) {
      if (threadIdx.x == 0 && rows > 0) report(a.status, COBS_ERR_DEVICE);
      return;
    }
    if (page < 0) return;
    row0 = (int64_t(page) * a.c.hkv + h) * kBlock;
  }
  const int li = threadIdx.x % kLanes;
  for (int which = 0; which < 2; ++which) {
    uint16_t* out = which ? a.v_out : a.k_out;
    if (out == nullptr) continue;
    const void* src = which ? a.c.v : a.c.k;
    const float* scales = which ? a.c.vs : a.c.ks;
    for (int r = threadIdx.x / kLanes; r < rows; r += kReadThreads / kLanes) {
      uint4 w;
      if (kFormat == COBS_CACHE_BF16) {
        w = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(src) +
                                            (row0 + r) * D + 8 * li);
      } else {
        const uint2 codes = *reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(src) +
                                                            (row0 + r) * D + 8 * li);
        const float sc = scales[row0 + r];
        const uint32_t c[4] = {codes.x & 0xffffu, codes.x >> 16, codes.y & 0xffffu, codes.y >> 16};
        uint32_t o[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const float2 f = e4m3x2_to_float2(c[u]);
          o[u] = bf16x2_bits(f.x * sc, f.y * sc);
        }
        w = make_uint4(o[0], o[1], o[2], o[3]);
      }
      *reinterpret_cast<uint4*>(out + ((page_out * a.c.hkv + h) * kBlock + r) * D + 8 * li) = w;
    }
  }
}

}  // namespace

cudaError_t launch_read_cache(const ReadArgs& a, cudaStream_t stream) {
  const int64_t ctas = int64_t(a.batch) * a.n * a.c.hkv;
  if (ctas >= (int64_t(1) << 31)) return cudaErrorInvalidValue;
  auto kern = a.d == 128 ? (a.c.format == COBS_CACHE_E4M3 ? read_cache_kernel<128, 1> : read_cache_kernel<128, 0>)
                         : (a.c.format == COBS_CACHE_E4M3 ? read_cache_kernel<64, 1> : read_cache_kernel<64, 0>);
  return launch_pdl(kern, dim3(unsigned(ctas)), dim3(kReadThreads), 0, stream, a);
}

}  // namespace cobs
