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
  // all loads of K and V first, then the conversions and stores
  constexpr int kStep = kReadThreads / kLanes, kPer = kBlock / kStep;
  const int li = threadIdx.x % kLanes, r0 = threadIdx.x / kLanes;
  uint4 w[2][kPer];
  float sc[2][kPer];
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    const void* src = which ? a.c.v : a.c.k;
    const float* scales = which ? a.c.vs : a.c.ks;
    const bool wanted = (which ? a.v_out : a.k_out) != nullptr;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int r = r0 + i * kStep;
      w[which][i] = make_uint4(0u, 0u, 0u, 0u);
      sc[which][i] = 0.f;
      if (!wanted || r >= rows) continue;
      const int64_t at = (row0 + r) * D + 8 * li;
      if (kFormat == COBS_CACHE_BF16) {
        w[which][i] = __ldcs(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(src) + at));
      } else {
        const uint2 c = __ldcs(reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(src) + at));
        w[which][i].x = c.x;
        w[which][i].y = c.y;
        sc[which][i] = __ldg(scales + row0 + r);
      }
    }
  }
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    uint16_t* out = which ? a.v_out : a.k_out;
    if (out == nullptr) continue;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int r = r0 + i * kStep;
      if (r >= rows) continue;
      uint4 o = w[which][i];
      if (kFormat == COBS_CACHE_E4M3) {
        const float s = sc[which][i];
        const uint32_t c[4] = {o.x & 0xffffu, o.x >> 16, o.y & 0xffffu, o.y >> 16};
        uint32_t v[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const float2 f = e4m3x2_to_float2(c[u]);
          v[u] = bf16x2_bits(f.x * s, f.y * s);
        }
        o = make_uint4(v[0], v[1], v[2], v[3]);
      }
      *reinterpret_cast<uint4*>(out + ((page_out * a.c.hkv + h) * kBlock + r) * D + 8 * li) = o;
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
