// Causal attention of packed new tokens over the bf16 cache
// (include/cobs_cache.h, cobs_prompt_attention).
//
// One warp per (token, query head): the keys of 32 tokens at a time, one per
// lane, then p = 2^(s - m) with a running maximum m and sum l, and the values
// summed with the output dimensions spread over the lanes.
#include "cache_device.cuh"

namespace cobs {
namespace {

constexpr int kPromptWarps = 4;

template <int D>
__global__ void __launch_bounds__(32 * kPromptWarps) prompt_rows_kernel(const PromptArgs a) {
  constexpr int kE = D / 32;   // output dimensions of a lane
  __shared__ float qs[kPromptWarps][D];
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t row = int64_t(blockIdx.x) * kPromptWarps + warp;
  const int64_t token = row / a.hq;
  const int hq = int(row % a.hq);
  if (token >= a.n_tokens) return;
  const int b = warp_find_sequence(a.cu, a.batch, token, lane);
  if (b >= a.batch) return;
  const int kvh = hq / (a.hq / a.c.hkv);
  int64_t len = __ldg(a.seq_lens + b);
  if (len < 0 || len > a.max_seq_len) {
    if (lane == 0) report(a.status, COBS_ERR_DEVICE);
    len = len < 0 ? 0 : a.max_seq_len;
  }
  const int64_t last = a.cu != nullptr ? __ldg(a.cu + b + 1) : token + 1;
  const int64_t pos = len - (last - token);
  for (int t = lane; t < D; t += 32)
    qs[warp][t] = __uint_as_float(uint32_t(a.q[row * D + t]) << 16);
  __syncwarp();
  float m = -INFINITY, l = 0.f, o[kE];
#pragma unroll
  for (int e = 0; e < kE; ++e) o[e] = 0.f;
  for (int64_t j0 = 0; j0 <= pos; j0 += 32) {
    const int64_t r0 = cache_row(a.c, b, kvh, j0);
    if (r0 < 0) {
      if (lane == 0) report(a.status, COBS_ERR_DEVICE);
      continue;
    }
    const int n = int(pos + 1 - j0 < 32 ? pos + 1 - j0 : 32);
    float s = -INFINITY;
    if (lane < n) {
      const uint4* kp = reinterpret_cast<const uint4*>(
          static_cast<const uint16_t*>(a.c.k) + (r0 + lane) * D);
      float acc = 0.f;
#pragma unroll 4
      for (int t = 0; t < D / 8; ++t) {
        const uint4 w = kp[t];
        const uint32_t wv[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const float2 f = bf16x2_to_float2(wv[u]);
          acc = fmaf(f.x, qs[warp][8 * t + 2 * u], acc);
          acc = fmaf(f.y, qs[warp][8 * t + 2 * u + 1], acc);
        }
      }
      s = acc * a.scale_log2;
    }
    const float mn = fmaxf(m, warp_max(s));
    const float alpha = m == -INFINITY ? 0.f : exp2f(m - mn);
    const float p = lane < n ? exp2f(s - mn) : 0.f;
    l = l * alpha + warp_sum(p);
    m = mn;
#pragma unroll
    for (int e = 0; e < kE; ++e) o[e] *= alpha;
    for (int i = 0; i < n; ++i) {
      const float pi = __shfl_sync(0xffffffffu, p, i);
      const uint16_t* vp = static_cast<const uint16_t*>(a.c.v) + (r0 + i) * D + lane * kE;
#pragma unroll
      for (int e = 0; e < kE; ++e)
        o[e] = fmaf(pi, __uint_as_float(uint32_t(vp[e]) << 16), o[e]);
    }
  }
  const float inv = l > 0.f ? 1.f / l : 0.f;
#pragma unroll
  for (int e = 0; e < kE; e += 2)
    *reinterpret_cast<uint32_t*>(a.out + row * D + lane * kE + e) =
        bf16x2_bits(o[e] * inv, o[e + 1] * inv);
  if (lane == 0 && a.lse != nullptr)
    a.lse[row] = l > 0.f ? (m + log2f(l)) * 0.69314718055994530942f : -INFINITY;
}

}  // namespace

size_t prompt_partial_bytes(const cobs_dims*, int64_t, int64_t) { return 0; }

cudaError_t launch_prompt(const PromptArgs& a, cudaStream_t stream) {
  const int64_t ctas = (a.n_tokens * a.hq + kPromptWarps - 1) / kPromptWarps;
  if (ctas >= (int64_t(1) << 31)) return cudaErrorInvalidValue;
  auto kern = a.d == 128 ? prompt_rows_kernel<128> : prompt_rows_kernel<64>;
  return launch_pdl(kern, dim3(unsigned(ctas)), dim3(32 * kPromptWarps), 0, stream, a);
}

}  // namespace cobs
