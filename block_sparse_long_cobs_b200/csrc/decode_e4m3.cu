// Sparse decode over an E4M3 cache (include/cobs_cache.h,
// cobs_sparse_decode_cache): exact attention over the tokens of the selected
// blocks, whose keys and values are E4M3 codes with one fp32 scale per row.
//
// One warp per query head: the keys of 32 tokens at a time, one per lane,
// with a running maximum and sum.
#include "cache_device.cuh"

namespace cobs {
namespace {

constexpr int kWarps = 4;

template <int D>
__global__ void __launch_bounds__(32 * kWarps)
decode_rows_e4m3_kernel(const DecodeArgs a, const float* ks, const float* vs) {
  constexpr int kE = D / 32;
  __shared__ float qs[kWarps][D];
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t row = int64_t(blockIdx.x) * kWarps + warp;   // b * hq + head
  if (row >= int64_t(a.batch) * a.hq) return;
  const int64_t b = row / a.hq;
  const int group = a.hq / a.hkv;
  const int kvh = int(row % a.hq) / group;
  const bool first = int(row % a.hq) % group == 0 && lane == 0;
  const int64_t pair = b * a.hkv + kvh;
  const int64_t len = sequence_length(a.seq_lens, a.seq_len, b, a.status, first);
  const int64_t nblk = (len + kBlock - 1) / kBlock;
  int n_sel = a.n_sel[pair];
  if (n_sel < 1 || n_sel > a.idx_stride) {
    if (first) report(a.status, COBS_ERR_DEVICE);
    n_sel = n_sel < 0 ? 0 : (n_sel > a.idx_stride ? a.idx_stride : n_sel);
  }
  for (int t = lane; t < D; t += 32)
    qs[warp][t] = __uint_as_float(uint32_t(a.q[row * D + t]) << 16);
  __syncwarp();
  float m = -INFINITY, l = 0.f, o[kE];
#pragma unroll
  for (int e = 0; e < kE; ++e) o[e] = 0.f;
  for (int s2 = 0; s2 < 2 * n_sel; ++s2) {
    const int j = a.idx[pair * a.idx_stride + (s2 >> 1)];
    int64_t r0 = -1;
    if (j >= 0 && j < nblk) {
      if (a.block_table == nullptr) {
        r0 = pair * a.cap + int64_t(j) * kBlock;
      } else {
        const int32_t page = a.block_table[b * a.table_stride + j];
        if (page >= 0 && page < a.n_pages) r0 = (int64_t(page) * a.hkv + kvh) * kBlock;
      }
    }
    if (r0 < 0) {
      if (first) report(a.status, COBS_ERR_DEVICE);
      continue;
    }
    const int64_t t0 = int64_t(j) * kBlock + 32 * (s2 & 1);
    r0 += 32 * (s2 & 1);
    const int n = int(len - t0 < 32 ? len - t0 : 32);
    if (n <= 0) continue;
    float s = -INFINITY, vsc = 0.f;
    if (lane < n) {
      const uint2* kp = reinterpret_cast<const uint2*>(
          reinterpret_cast<const uint8_t*>(a.k) + (r0 + lane) * D);
      float acc = 0.f;
#pragma unroll 4
      for (int t = 0; t < D / 8; ++t) {
        const uint2 w = kp[t];
        const uint32_t wv[4] = {w.x & 0xffffu, w.x >> 16, w.y & 0xffffu, w.y >> 16};
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const float2 f = e4m3x2_to_float2(wv[u]);
          acc = fmaf(f.x, qs[warp][8 * t + 2 * u], acc);
          acc = fmaf(f.y, qs[warp][8 * t + 2 * u + 1], acc);
        }
      }
      s = acc * ks[r0 + lane] * a.scale_log2;
      vsc = vs[r0 + lane];
    }
    const float mn = fmaxf(m, warp_max(s));
    const float alpha = m == -INFINITY ? 0.f : exp2f(m - mn);
    const float p = lane < n ? exp2f(s - mn) : 0.f;
    l = l * alpha + warp_sum(p);
    m = mn;
#pragma unroll
    for (int e = 0; e < kE; ++e) o[e] *= alpha;
    const float wgt = p * vsc;
    for (int i = 0; i < n; ++i) {
      const float wi = __shfl_sync(0xffffffffu, wgt, i);
      const uint8_t* vp = reinterpret_cast<const uint8_t*>(a.v) + (r0 + i) * D + lane * kE;
#pragma unroll
      for (int e = 0; e < kE; e += 2) {
        const float2 f = e4m3x2_to_float2(*reinterpret_cast<const uint16_t*>(vp + e));
        o[e] = fmaf(wi, f.x, o[e]);
        o[e + 1] = fmaf(wi, f.y, o[e + 1]);
      }
    }
  }
  const float inv = l > 0.f ? 1.f / l : 0.f;
#pragma unroll
  for (int e = 0; e < kE; ++e) a.out[row * D + lane * kE + e] = o[e] * inv;
  if (lane == 0) a.lse[row] = l > 0.f ? (m + log2f(l)) * 0.69314718055994530942f : -INFINITY;
}

}  // namespace

cudaError_t launch_decode_e4m3(const DecodeArgs& a, const float* ks, const float* vs,
                               cudaStream_t stream) {
  const int64_t ctas = (int64_t(a.batch) * a.hq + kWarps - 1) / kWarps;
  auto kern = a.d == 128 ? decode_rows_e4m3_kernel<128> : decode_rows_e4m3_kernel<64>;
  return launch_pdl(kern, dim3(unsigned(ctas)), dim3(32 * kWarps), 0, stream, a, ks, vs);
}

}  // namespace cobs
