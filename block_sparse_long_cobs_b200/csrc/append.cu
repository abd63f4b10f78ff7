// Appending tokens: rotary positions on queries and keys, and the cache rows
// of the new keys and values, in one pass (include/cobs_cache.h,
// cobs_append_tokens).
//
// For a rotated pair (x1, x2) at position p with frequency f,
//   (y1, y2) = A (x1 cos pf - x2 sin pf, x2 cos pf + x1 sin pf).
// The angle is taken in turns: the table holds f / 2 pi as a 64-bit fraction
// of a turn, so p times it modulo 2^64 is the exact fraction of the turn (its
// error is p 2^-64 turns), whatever the position; a product in fp32 would be
// off by p f 2^-24 radians, 0.016 at 2^18 tokens.
//
// Bound by memory: every row is read once and written once.  A warp takes
// some head rows of one token, so the sines and cosines (they depend on the
// token alone) are computed once for all of them; d / 8 lanes share a row,
// each with four pairs, in two 8-byte pieces.
#include "cache_device.cuh"

namespace cobs {
namespace {

constexpr int kAppendWarps = 4;

__device__ __forceinline__ float finite_or_zero_abs(float x) {
  const float a = fabsf(x);
  return a <= 3.402823466e38f ? a : 0.f;   // NaN and infinities count as 0
}

template <int D, int kFormat>
__global__ void __launch_bounds__(32 * kAppendWarps) append_kernel(const __grid_constant__ AppendArgs a) {
  constexpr int kLanes = D / 8;          // lanes of a row
  constexpr int kRows = 32 / kLanes;     // rows of a warp at a time
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int64_t item = int64_t(blockIdx.x) * kAppendWarps + (threadIdx.x >> 5);
  const int64_t token = item / a.chunks;
  if (token >= a.n_tokens) return;
  const int b = warp_find_sequence(a.cu, a.batch, token, lane);
  if (b >= a.batch) return;
  const int64_t pos = __ldg(a.start + b) + (a.cu != nullptr ? token - __ldg(a.cu + b) : 0);
  const int hkv = a.c.hkv;
  const int n_rows = a.hq + 2 * hkv;
  const int r0 = int(item % a.chunks) * a.rows_per_warp;
  const int r1 = min(r0 + a.rows_per_warp, n_rows);

  // this lane's four pair slots of a row
  const int li = lane % kLanes, sub = lane / kLanes;
  const int half_rot = a.rope.rotary_dim >> 1;
  const int slot = 4 * li;
  const bool rot = slot < half_rot;
  const bool inter = a.rope.interleaved != 0;
  int e1, e2;                            // first elements of its two pieces
  if (inter || !rot) {
    e1 = inter ? 2 * slot : 2 * half_rot + 2 * (slot - half_rot);
    e2 = e1 + 4;
  } else {
    e1 = slot;
    e2 = half_rot + slot;
  }
  float cs[4], sn[4];
  if (rot) {
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const uint64_t turn = uint64_t(pos) * a.rope.turns[slot + u];
      // the fraction as half turns in [-1, 1)
      const float x = float(int32_t(uint32_t(turn >> 32))) * 4.656612873077393e-10f;
      sincospif(x, &sn[u], &cs[u]);
      cs[u] *= a.rope.attention_factor;
      sn[u] *= a.rope.attention_factor;
    }
  }
  bool stored = true;
  for (int r = r0 + sub; r - sub < r1; r += kRows) {
    const bool act = r < r1;
    const int which = r < a.hq ? 0 : (r < a.hq + hkv ? 1 : 2);   // q, k, v
    const int h = which == 0 ? r : (which == 1 ? r - a.hq : r - a.hq - hkv);
    const uint16_t* src = which == 0   ? a.q + token * a.q_stride
                          : which == 1 ? a.k + token * a.k_stride
                                       : a.v + token * a.v_stride;
    src += int64_t(h) * D;
    const int f1 = which == 2 ? 8 * li : e1, f2 = which == 2 ? 8 * li + 4 : e2;
    uint2 w1 = make_uint2(0u, 0u), w2 = w1;
    if (act) {
      w1 = *reinterpret_cast<const uint2*>(src + f1);
      w2 = *reinterpret_cast<const uint2*>(src + f2);
    }
    float x[8];
    {
      const float2 p0 = bf16x2_to_float2(w1.x), p1 = bf16x2_to_float2(w1.y);
      const float2 p2 = bf16x2_to_float2(w2.x), p3 = bf16x2_to_float2(w2.y);
      x[0] = p0.x; x[1] = p0.y; x[2] = p1.x; x[3] = p1.y;
      x[4] = p2.x; x[5] = p2.y; x[6] = p3.x; x[7] = p3.y;
    }
    const bool turn_it = rot && which < 2;
    if (turn_it) {
      if (inter) {
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const float p = x[2 * u], q = x[2 * u + 1];
          x[2 * u] = p * cs[u] - q * sn[u];
          x[2 * u + 1] = q * cs[u] + p * sn[u];
        }
      } else {
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const float p = x[u], q = x[4 + u];
          x[u] = p * cs[u] - q * sn[u];
          x[4 + u] = q * cs[u] + p * sn[u];
        }
      }
    }
    uint16_t* dst16 = nullptr;
    int64_t row = 0;
    if (which == 0) {
      dst16 = a.q_out + (token * a.hq + h) * int64_t(D);
    } else {
      row = cache_row(a.c, b, h, pos);
      stored &= row >= 0 || !act;
      dst16 = reinterpret_cast<uint16_t*>(which == 1 ? a.c.k : a.c.v) + row * D;
    }
    if (kFormat == COBS_CACHE_E4M3) {
      float top = 0.f;
#pragma unroll
      for (int u = 0; u < 8; ++u) top = fmaxf(top, finite_or_zero_abs(x[u]));
#pragma unroll
      for (int m = kLanes / 2; m > 0; m >>= 1)
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, m));
      if (which != 0) {
        float scale = top / 448.f;
        if (scale < 1.17549435e-38f) scale = 0.f;
        const float inv = scale > 0.f ? 1.f / scale : 0.f;
#pragma unroll
        for (int u = 0; u < 8; ++u)
          x[u] = fabsf(x[u]) <= 3.402823466e38f ? x[u] * inv : __uint_as_float(0x7fffffffu);
        if (act && row >= 0) {
          uint8_t* dst = reinterpret_cast<uint8_t*>(which == 1 ? a.c.k : a.c.v) + row * D;
          *reinterpret_cast<uint32_t*>(dst + f1) = e4m3x2(x[0], x[1]) | (e4m3x2(x[2], x[3]) << 16);
          *reinterpret_cast<uint32_t*>(dst + f2) = e4m3x2(x[4], x[5]) | (e4m3x2(x[6], x[7]) << 16);
          if (li == 0) (which == 1 ? a.c.ks : a.c.vs)[row] = scale;
        }
        continue;
      }
    }
    if (act && (which == 0 || row >= 0)) {
      if (turn_it) {
        w1 = make_uint2(bf16x2_bits(x[0], x[1]), bf16x2_bits(x[2], x[3]));
        w2 = make_uint2(bf16x2_bits(x[4], x[5]), bf16x2_bits(x[6], x[7]));
      }
      *reinterpret_cast<uint2*>(dst16 + f1) = w1;
      *reinterpret_cast<uint2*>(dst16 + f2) = w2;
    }
  }
  if (!stored) report(a.status, COBS_ERR_DEVICE);
}

}  // namespace

cudaError_t launch_append(const AppendArgs& a0, cudaStream_t stream) {
  AppendArgs a = a0;
  const int n_rows = a.hq + 2 * a.c.hkv;
  a.rows_per_warp = 8;
  a.chunks = (n_rows + a.rows_per_warp - 1) / a.rows_per_warp;
  const int64_t ctas = (a.n_tokens * a.chunks + kAppendWarps - 1) / kAppendWarps;
  if (ctas >= (int64_t(1) << 31)) return cudaErrorInvalidValue;
  auto kern = a.d == 128 ? (a.c.format == COBS_CACHE_E4M3 ? append_kernel<128, 1> : append_kernel<128, 0>)
                         : (a.c.format == COBS_CACHE_E4M3 ? append_kernel<64, 1> : append_kernel<64, 0>);
  return launch_pdl(kern, dim3(unsigned(ctas)), dim3(32 * kAppendWarps), 0, stream, a);
}

}  // namespace cobs
