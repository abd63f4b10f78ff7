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
// token alone), the sequence and the page are found once for all of them;
// d / 8 lanes share a row, each with four pairs, in two 8-byte pieces, and
// the loads of kBatch rows are issued together.
#include "cache_device.cuh"

namespace cobs {
namespace {

constexpr int kAppendWarps = 4;
constexpr int kBatch = 4;                // rows (of a sub-warp) loaded together

template <int K>
struct Kind {
  static constexpr int value = K;
};

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
  // bounds outside the rows, or descending, are reported: the first warps look
  // at 32 sequences each
  if (a.cu != nullptr)
    for (int64_t s = item * 32 + lane; s < a.batch; s += int64_t(gridDim.x) * kAppendWarps * 32) {
      const int64_t c0 = __ldg(a.cu + s), c1 = __ldg(a.cu + s + 1);
      if (c0 < 0 || c1 < c0 || c1 > a.n_tokens) report(a.status, COBS_ERR_DEVICE);
    }
  if (token >= a.n_tokens) return;
  int b;
  int64_t pos, first = token;            // of the sequence, its bound cut to the rows
  if (a.cu != nullptr && a.batch <= 32) {
    // bounds and lengths of all sequences at once: one trip to memory, not two
    const bool in = lane < a.batch;
    const int32_t c0 = in ? __ldg(a.cu + lane) : 0, c1 = in ? __ldg(a.cu + lane + 1) : 0;
    const int64_t st = in ? __ldg(a.start + lane) : 0;
    b = __popc(__ballot_sync(0xffffffffu, in && int64_t(c1) <= token));
    if (b >= a.batch) return;
    first = max(__shfl_sync(0xffffffffu, c0, b), 0);
    pos = __shfl_sync(0xffffffffu, st, b) + token - first;
  } else {
    b = warp_find_sequence(a.cu, a.batch, token, lane);
    if (b >= a.batch) return;
    if (a.cu != nullptr) first = max(__ldg(a.cu + b), 0);
    pos = __ldg(a.start + b) + token - first;
  }
  if (token < first) return;             // before the first bound: nobody's
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
  float cs[4] = {}, sn[4] = {};
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
  // cache row of kv-head 0 (-1: no place) and the rows between heads
  const int64_t row0 = cache_row(a.c, b, 0, pos);
  const int64_t head_rows = a.c.table != nullptr ? int64_t(kBlock) : a.c.cap;
  if (row0 < 0 && r1 > a.hq && lane == 0) report(a.status, COBS_ERR_DEVICE);
  const uint64_t cs2[2] = {pack2(make_float2(cs[0], cs[1])), pack2(make_float2(cs[2], cs[3]))};
  const uint64_t sn2[2] = {pack2(make_float2(sn[0], sn[1])), pack2(make_float2(sn[2], sn[3]))};
  const uint64_t ns2[2] = {pack2(make_float2(-sn[0], -sn[1])), pack2(make_float2(-sn[2], -sn[3]))};

  // n head rows of one kind (0 queries, 1 keys, 2 values) from src on; row i
  // goes to row `row + i step` of dst (and of scales).
  auto rows = [&](auto kind, const uint16_t* src, int n, void* dst, float* scales, int64_t row,
                  int64_t step) {
    constexpr int kKind = decltype(kind)::value;
    constexpr bool kCode = kKind != 0 && kFormat == COBS_CACHE_E4M3;
    const bool turn = kKind != 2 && rot;
    const int f1 = kKind == 2 ? 8 * li : e1, f2 = kKind == 2 ? 8 * li + 4 : e2;
    for (int rb = sub; rb - sub < n; rb += kBatch * kRows) {
      uint2 w1[kBatch], w2[kBatch];
      const uint16_t* p = src + rb * D;
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        w1[i] = w2[i] = make_uint2(0u, 0u);
        if (rb + i * kRows < n) {
          w1[i] = *reinterpret_cast<const uint2*>(p + i * kRows * D + f1);
          w2[i] = *reinterpret_cast<const uint2*>(p + i * kRows * D + f2);
        }
      }
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        if (rb - sub + i * kRows >= n) break;    // the same in every lane
        const bool act = rb + i * kRows < n;
        if (turn || kCode) {
          uint64_t x[4] = {pack2(bf16x2_to_float2(w1[i].x)), pack2(bf16x2_to_float2(w1[i].y)),
                           pack2(bf16x2_to_float2(w2[i].x)), pack2(bf16x2_to_float2(w2[i].y))};
          if (turn) {
            if (inter) {   // pairs side by side: x1 of two pairs, x2 of two pairs
#pragma unroll
              for (int u = 0; u < 4; u += 2) {
                const float2 m = unpack2(x[u]), q = unpack2(x[u + 1]);
                x[u] = pack2(make_float2(m.x, q.x));
                x[u + 1] = pack2(make_float2(m.y, q.y));
              }
            }
#pragma unroll
            for (int u = 0; u < 2; ++u) {
              const uint64_t x1 = inter ? x[2 * u] : x[u], x2 = inter ? x[2 * u + 1] : x[2 + u];
              const uint64_t y1 = fma2(x2, ns2[u], mul2(x1, cs2[u]));
              const uint64_t y2 = fma2(x1, sn2[u], mul2(x2, cs2[u]));
              if (inter) {
                const float2 m = unpack2(y1), q = unpack2(y2);
                x[2 * u] = pack2(make_float2(m.x, q.x));
                x[2 * u + 1] = pack2(make_float2(m.y, q.y));
              } else {
                x[u] = y1;
                x[2 + u] = y2;
              }
            }
          }
          const float2 v0 = unpack2(x[0]), v1 = unpack2(x[1]), v2 = unpack2(x[2]), v3 = unpack2(x[3]);
          if constexpr (kCode) {
            float v[8] = {v0.x, v0.y, v1.x, v1.y, v2.x, v2.y, v3.x, v3.y};
            float top = 0.f;
#pragma unroll
            for (int u = 0; u < 8; ++u) top = fmaxf(top, finite_or_zero_abs(v[u]));
            __syncwarp();
#pragma unroll
            for (int m = kLanes / 2; m > 0; m >>= 1)
              top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, m));
            float scale = top / 448.f;
            if (scale < 1.17549435e-38f) scale = 0.f;
            // Codes of x / scale: x times y = 1 / scale alone falls on the other
            // side of the middle between two codes now and then, so that the
            // quotient q = x y is put right by its exact remainder, q + (x - q
            // scale) y (Markstein, IBM J. Res. Dev. 34, 1990).  That is x / scale
            // to the last bit for every bf16 x, and for 10^9 fp32 ones but one.
            // (4096 tokens: 33.2 us, with q alone 33.2, with a division 35.5.)  What
            // is not finite becomes NaN on the way, scale 0 gives zeros.
            float by = scale;
            if (scale < 0x1p-60f) {       // remainders above the subnormal numbers
              const uint64_t up = pack2(make_float2(0x1p64f, 0x1p64f));
#pragma unroll
              for (int u = 0; u < 4; ++u) x[u] = mul2(x[u], up);
              by *= 0x1p64f;
            }
            const float inv = by > 0.f ? 1.f / by : 0.f;
            const uint64_t inv2 = pack2(make_float2(inv, inv)), nb2 = pack2(make_float2(-by, -by));
            uint32_t code[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) {
              const uint64_t q = mul2(x[u], inv2);
              const float2 c = unpack2(fma2(fma2(q, nb2, x[u]), inv2, q));
              code[u] = e4m3x2(c.x, c.y);
            }
            if (act) {
              const int64_t r = row + (rb + i * kRows) * step;
              uint8_t* d = static_cast<uint8_t*>(dst) + r * D;
              *reinterpret_cast<uint32_t*>(d + f1) = code[0] | (code[1] << 16);
              *reinterpret_cast<uint32_t*>(d + f2) = code[2] | (code[3] << 16);
              if (li == 0) scales[r] = scale;
            }
          } else {
            w1[i] = make_uint2(bf16x2_bits(v0.x, v0.y), bf16x2_bits(v1.x, v1.y));
            w2[i] = make_uint2(bf16x2_bits(v2.x, v2.y), bf16x2_bits(v3.x, v3.y));
          }
        }
        if (!kCode && act) {
          uint16_t* d = static_cast<uint16_t*>(dst) + (row + (rb + i * kRows) * step) * D;
          *reinterpret_cast<uint2*>(d + f1) = w1[i];
          *reinterpret_cast<uint2*>(d + f2) = w2[i];
        }
      }
    }
  };
  const int q1 = min(r1, a.hq);
  if (r0 < q1)
    rows(Kind<0>(), a.q + token * a.q_stride + r0 * D, q1 - r0, a.q_out, nullptr,
         token * a.hq + r0, 1);
  if (row0 < 0) return;
  const int k0 = max(r0 - a.hq, 0), k1 = min(r1 - a.hq, hkv);
  if (k0 < k1)
    rows(Kind<1>(), a.k + token * a.k_stride + k0 * D, k1 - k0, a.c.k, a.c.ks,
         row0 + k0 * head_rows, head_rows);
  const int v0 = max(r0 - a.hq - hkv, 0), v1 = min(r1 - a.hq - hkv, hkv);
  if (v0 < v1)
    rows(Kind<2>(), a.v + token * a.v_stride + v0 * D, v1 - v0, a.c.v, a.c.vs,
         row0 + v0 * head_rows, head_rows);
}

}  // namespace

cudaError_t launch_append(const AppendArgs& a0, cudaStream_t stream) {
  AppendArgs a = a0;
  const int n_rows = a.hq + 2 * a.c.hkv;
  // Few tokens: a pass of one row per sub-warp, so that the GPU is filled and
  // nothing waits in turn (32 tokens of 48 rows: 3.3 us, with 32 rows a warp
  // 5.0); many: up to kBatch loads' worth four times over, so that the sines are
  // shared (4096 tokens of 80 rows: 33.0 us, with 16 rows a warp 37.6).  About
  // 32 warps per SM lie between the two.
  const int per_pass = 32 / (a.d / 8);
  int64_t rows = a.n_tokens * n_rows / (int64_t(148) * 32);
  rows = rows < per_pass ? per_pass : (rows > 4 * kBatch * per_pass ? 4 * kBatch * per_pass : rows);
  a.rows_per_warp = int32_t(rows / per_pass * per_pass);
  a.chunks = (n_rows + a.rows_per_warp - 1) / a.rows_per_warp;
  const int64_t ctas = (a.n_tokens * a.chunks + kAppendWarps - 1) / kAppendWarps;
  if (ctas >= (int64_t(1) << 31)) return cudaErrorInvalidValue;
  auto kern = a.d == 128 ? (a.c.format == COBS_CACHE_E4M3 ? append_kernel<128, 1> : append_kernel<128, 0>)
                         : (a.c.format == COBS_CACHE_E4M3 ? append_kernel<64, 1> : append_kernel<64, 0>);
  return launch_pdl(kern, dim3(unsigned(ctas)), dim3(32 * kAppendWarps), 0, stream, a);
}

}  // namespace cobs
