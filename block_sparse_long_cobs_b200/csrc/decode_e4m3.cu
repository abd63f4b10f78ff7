// Sparse decode over an E4M3 cache (include/cobs_cache.h,
// cobs_sparse_decode_cache) on the tensor cores: exact attention over the
// tokens of the selected blocks, whose keys and values are E4M3 codes with one
// fp32 scale per row, read by kind::f8f6f4 products as they are stored.
//
//   logit_j = scale ks_j (q . kc_j),  out = sum_j e^(logit_j - m) vs_j vc_j / l,
//   l = sum_j e^(logit_j - m).
//
// Operands.  A query row times a power of two is split into three E4M3 parts,
// q = h0 + h1 / 16 + h2 / 256 (a part takes 4 significant bits; the last one's
// smallest step is 2^-23 to 2^-24 of the row's largest), so that S = K [h0; h1; h2]^T
// (M = 128 keys) loses nothing of a bf16 query.  The weights of the values,
// w = vs 2^(s - M), are split into four parts in the same way (2^-16 of the
// weight, 2^-24 of the largest), and O^T = V^T [w0; w1; w2; w3]^T (M = 128
// dimensions) is put together when it is read back.  The value scales take
// part in the running maximum of O (M, over s + floor(log2 vs)), so that rows
// of any magnitude keep those bits; l has its own (m, over s), both raised
// only when a tile exceeds them by more than 2^8 or 2^7.75.  M is set to a quarter
// of the largest weight: what the last part rounds is relative to 2^M, and the
// first part has room above it.  (Outputs of 32 sequences at 32k against 64 bits:
// 4 to 5 10^-7, with M the largest 7 to 12 10^-7, with an eighth 4 10^-7.  Time:
// 22.3, 22.2 and 22.4 us at 4 heads per kv-head, 28.1, 27.5 and 28.8 at 8, where
// tiles raise M more often.)
//
// Bound by memory: d + 4 bytes per key and per value row.  Work split, ring
// and merge are those of the bf16 decode: a persistent grid (two CTAs per SM)
// takes chunks of the pairs' block lists off a counter, a tile is two blocks,
//   warps 0-3  softmax (one key per thread) and output
//   warp 4     TMA: K_t with the scales of both, V_t, through a 5-slot ring
//   warp 5     products, one tile of scores ahead of the softmax
//   warp 6     the query parts of the next chunk
// head_dim 64 runs the same kernel: the tensor maps fill the other 64 columns
// with zeros (shared memory only, no traffic).
//
// Keys at or past a sequence's length are masked, and their V rows zeroed where
// the tensor maps do not (a zero weight times a NaN code is not zero).  Every
// wait is bounded; a CTA that gives up records COBS_ERR_TIMEOUT, lets its
// copies and products finish, frees its tensor memory and returns.
#include "tcgen05_issue.cuh"

namespace cobs {
namespace {

constexpr int kW = 128;                  // bytes of a tile row (head_dim 64: half zeros)
constexpr int kThreads = 224;
constexpr int kSoftThreads = 128;
constexpr int kStages = 5;
constexpr int kStageBytes = 128 * kW;
constexpr int kScaleSlots = 4;           // tiles whose scales are in flight
constexpr int kPSlots = 2;
// Row scales of the query parts (and their barriers) live four chunks: they are
// written for chunk n + 4 after the products of chunk n + 2 began, which wait
// until the softmax has taken the scores of chunk n.
constexpr int kQRing = 4;
constexpr int kChunkQ = 4;
constexpr float kRaiseM = 8.f;           // l's maximum is raised beyond 2^8
constexpr float kRaiseO = 7.75f;         // O's beyond 2^7.75: a weight, up to twice that, below 448
constexpr float kBelowO = 2.f;           // O's unit is 2^-2 of the largest
constexpr float kLn2 = 0.69314718055994530942f;

template <int G>
struct Shape {
  static constexpr int kHeads = G <= 4 ? 4 : 8;     // head rows of an operand part
  static constexpr int kN = 4 * kHeads;             // operand rows: part x head
  static constexpr int kOpBytes = kN * kW;
  static constexpr uint32_t kTmemCols = 4 * kN;     // two score and two output buffers
  static constexpr int kOffQ = kStages * kStageBytes;
  static constexpr int kOffP = kOffQ + 2 * kOpBytes;
  static constexpr int kDynSmem = kOffP + kPSlots * kOpBytes + 1024;
};

// Instruction descriptors: D fp32, A and B E4M3, N >> 3 at bit 17, M >> 4 at
// bit 24; bit 15: A is MN-major.
constexpr uint32_t idesc_e4m3(int M, int N) {
  return (1u << 4) | (uint32_t(N >> 3) << 17) | (uint32_t(M >> 4) << 24);
}

// Byte of (operand row n, column c) in the K-major 128-byte-swizzled layout.
__device__ __forceinline__ uint32_t op_offset(int n, int c) {
  return uint32_t((n >> 3) * 1024 + (n & 7) * 128 + ((((c >> 4) ^ n) & 7) << 4) + (c & 15));
}

struct Chunk {
  int64_t pair;
  int seg, nb, s0;
  bool bad;   // n_sel outside [1, idx_stride]
};

__device__ __forceinline__ Chunk chunk_of(int64_t c, const DecodeArgs& a) {
  Chunk g;
  g.pair = c / a.chunks_per_pair;
  g.seg = int(c % a.chunks_per_pair);
  int n = __ldg(a.n_sel + g.pair);
  g.bad = n < 1 || n > a.idx_stride;
  n = n < 0 ? 0 : (n > a.idx_stride ? a.idx_stride : n);
  g.s0 = g.seg * a.chunk_slots;
  const int s1 = min(min(g.s0 + a.chunk_slots, a.idx_stride), n);
  g.nb = s1 > g.s0 ? s1 - g.s0 : 0;
  return g;
}

// The parts of two weights, scaled: w = p0 + p1 / 16 + p2 / 256 + p3 / 4096.
template <int kParts>
__device__ __forceinline__ void split2(float x, float y, uint32_t (&code)[kParts]) {
#pragma unroll
  for (int p = 0; p < kParts; ++p) {
    code[p] = e4m3x2(x, y);
    if (p + 1 < kParts) {
      const float2 f = e4m3x2_to_float2(code[p]);
      x = (x - f.x) * 16.f;
      y = (y - f.y) * 16.f;
    }
  }
}

// kMode: 0 one length for the batch, contiguous cache (the maps' row bound is
// the length); 1 per-sequence lengths; 2 page pools.
template <int G, int kMode>
__global__ void __launch_bounds__(kThreads, 2)
decode_e4m3_kernel(const __grid_constant__ CUtensorMap kmap,
                   const __grid_constant__ CUtensorMap vmap, const __grid_constant__ DecodeArgs a,
                   const float* __restrict__ ks_g, const float* __restrict__ vs_g) {
  using S = Shape<G>;
  constexpr int H = S::kHeads, N = S::kN;
  extern __shared__ uint8_t dyn_smem[];
  uint8_t* base = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(dyn_smem) + 1023) & ~uintptr_t(1023));
  __shared__ __align__(8) uint64_t full[kStages], empty[kStages];
  __shared__ __align__(8) uint64_t s_full[2], s_free[2], p_full[kPSlots], p_free[kPSlots];
  __shared__ __align__(8) uint64_t o_full[2], q_full[kQRing], q_empty[2], sc_full[kScaleSlots], drain;
  __shared__ __align__(8) uint64_t cq_full[kChunkQ], cq_empty[kChunkQ];
  __shared__ long long cq_val[kChunkQ];
  __shared__ __align__(16) float scales[kScaleSlots][2][128];   // of keys, of values
  __shared__ float q_inv[kQRing][8];
  __shared__ float red[4][2 * 8];
  __shared__ uint32_t tmem_slot;
  __shared__ volatile int abort_s;

  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  const int64_t seq_blocks = (a.seq_len + kBlock - 1) / kBlock;

  if (tid == 0) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&kmap)) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&vmap)) : "memory");
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&s_full[s], 1);
      mbar_init(&s_free[s], 4);
      mbar_init(&p_full[s], 4);
      mbar_init(&p_free[s], 1);
      mbar_init(&o_full[s], 1);
      mbar_init(&q_empty[s], 1);
    }
    for (int s = 0; s < kScaleSlots; ++s) mbar_init(&sc_full[s], 1);
    for (int s = 0; s < kQRing; ++s) mbar_init(&q_full[s], 1);
    for (int s = 0; s < kChunkQ; ++s) {
      mbar_init(&cq_full[s], 1);
      mbar_init(&cq_empty[s], 6);   // four softmax warps, products, queries
    }
    mbar_init(&drain, 1);
    fence_barrier_init();
    abort_s = 0;
  }
  if (warp == 0) tmem_alloc(&tmem_slot, S::kTmemCols);
  // operand rows that no head or part fills stay zero
  for (int e = tid; e < 4 * S::kOpBytes / 16; e += kThreads)
    reinterpret_cast<uint4*>(base + S::kOffQ)[e] = make_uint4(0u, 0u, 0u, 0u);
  fence_proxy_async_smem();
  pdl_wait();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  pdl_launch_dependents();
  const uint32_t tmem = tmem_slot;
  const uint32_t o_col = tmem + 2u * N;

  // the ci-th chunk of this CTA; -1: give up, n_chunks or more: no work left
  auto next_chunk = [&](uint32_t ci) -> int64_t {
    const int qs = ci % kChunkQ;
    if (!warp_wait(&cq_full[qs], (ci / kChunkQ) & 1, a.status, &abort_s)) return -1;
    const int64_t c = cq_val[qs];
    __syncwarp();
    if (lane == 0) mbar_arrive(&cq_empty[qs]);
    return c;
  };

  if (warp == 4) {
    // ============================ TMA producer ============================
    if (lane == 0) {
      uint32_t it = 0, gt = 0;
      bool ok = true;
      for (uint32_t ci = 0; ok; ++ci) {
        const int qs = ci % kChunkQ;
        if (ci >= kChunkQ &&
            !wait_step(&cq_empty[qs], ((ci / kChunkQ) - 1) & 1, a.status, &abort_s))
          break;
        const int64_t c = ci == 0 ? int64_t(blockIdx.x)
                                  : int64_t(gridDim.x) + int64_t(atomicAdd(&a.work[0], 1u));
        cq_val[qs] = c;
        mbar_arrive(&cq_full[qs]);
        if (c >= a.n_chunks) {
          // the last CTA to run out of work puts the counters back
          __threadfence();
          if (atomicAdd(&a.work[1], 1u) == gridDim.x - 1) {
            a.work[0] = 0u;
            a.work[1] = 0u;
            __threadfence();
          }
          break;
        }
        // the blocks of the next tile are asked for one tile ahead, those of the
        // first together with the count
        const int s0 = int(c % a.chunks_per_pair) * a.chunk_slots;
        const int32_t* row = a.idx + (c / a.chunks_per_pair) * a.idx_stride + s0;
        int jn[2] = {__ldg(row), s0 + 1 < a.idx_stride ? __ldg(row + 1) : -1};
        const Chunk g = chunk_of(c, a);
        const int64_t b = g.pair / a.hkv;
        const int64_t len_b =
            kMode == 0 ? a.seq_len : sequence_length(a.seq_lens, a.seq_len, b, a.status, false);
        const int64_t blocks_b = kMode == 0 ? seq_blocks : (len_b + kBlock - 1) / kBlock;
        for (int t = 0; 2 * t < g.nb && ok; ++t, ++gt) {
          const int nh = 2 * t + 1 < g.nb ? 2 : 1;
          const int jc[2] = {jn[0], jn[1]};
          if (2 * t + 2 < g.nb) jn[0] = __ldg(row + 2 * t + 2);
          if (2 * t + 3 < g.nb) jn[1] = __ldg(row + 2 * t + 3);
          int y[2] = {0, 0}, z[2] = {0, 0};
          int64_t r0[2] = {-1, -1};       // first row of the block's scales
          for (int h2 = 0; h2 < nh; ++h2) {
            const int j = jc[h2];
            bool in = j >= 0 && j < blocks_b;
            if constexpr (kMode == 2) {
              const int32_t page = in ? __ldg(a.block_table + b * a.table_stride + j) : -1;
              const bool good = page >= 0 && page < a.n_pages;
              if (in && !good) report(a.status, COBS_ERR_DEVICE);
              in = in && good;
              z[h2] = in ? int(int64_t(page) * a.hkv + g.pair % a.hkv) : 0;
              y[h2] = in ? 0 : kBlock;    // past the map's rows: reads as zero
              r0[h2] = in ? int64_t(z[h2]) * kBlock : -1;
            } else {
              z[h2] = int(g.pair);
              y[h2] = in ? j * kBlock : int(seq_blocks * kBlock);
              r0[h2] = in ? g.pair * a.cap + int64_t(j) * kBlock : -1;
            }
          }
          for (int kv = 0; kv < 2; ++kv, ++it) {
            const int st = it % kStages;
            if (it >= uint32_t(kStages) &&
                !wait_step(&empty[st], ((it / kStages) - 1) & 1, a.status, &abort_s)) {
              ok = false;
              break;
            }
            mbar_arrive_expect_tx(&full[st], uint32_t(nh) * 64u * kW);
            for (int h2 = 0; h2 < nh; ++h2)
              tma_load_3d(base + st * kStageBytes + h2 * 64 * kW, kv ? &vmap : &kmap, 0, y[h2],
                          z[h2], &full[st]);
            if (kv == 0) {
              // (K_t took the slot after V_{t - 3}'s: the softmax is done with
              // tile t - 3, nobody reads the scales of tile t - 4 any more)
              const int sl = gt % kScaleSlots;
              const int n = int(r0[0] >= 0) + int(r0[1] >= 0);
              mbar_arrive_expect_tx(&sc_full[sl], uint32_t(n) * 512u);
              for (int h2 = 0; h2 < nh; ++h2)
                if (r0[h2] >= 0) {
                  bulk_g2s(&scales[sl][0][64 * h2], ks_g + r0[h2], 256u, &sc_full[sl]);
                  bulk_g2s(&scales[sl][1][64 * h2], vs_g + r0[h2], 256u, &sc_full[sl]);
                }
            }
          }
        }
      }
      // copies of the last items may still be landing
      for (uint32_t x = it > uint32_t(kStages) ? it - kStages : 0u; x < it; ++x)
        (void)mbar_wait_bounded(&full[x % kStages], (x / kStages) & 1, a.status);
      const uint32_t tiles = (it + 1) / 2;   // tiles whose scales were asked for
      for (uint32_t x = tiles > uint32_t(kScaleSlots) ? tiles - kScaleSlots : 0u; x < tiles; ++x)
        (void)mbar_wait_bounded(&sc_full[x % kScaleSlots], (x / kScaleSlots) & 1, a.status);
    }
    __syncwarp();
  } else if (warp == 6) {
    // ============================ query parts =============================
    uint32_t n = 0;
    for (uint32_t ci = 0;; ++ci) {
      const int64_t c = next_chunk(ci);
      if (c < 0 || c >= a.n_chunks) break;
      const Chunk g = chunk_of(c, a);
      if (g.nb == 0) continue;
      const int buf = n & 1;
      const int64_t hq0 = (g.pair / a.hkv) * a.hq + (g.pair % a.hkv) * G;
      // lane: components 8 ch .. 8 ch + 7 of heads 2 i + lane / 16
      const int ch = lane & 15;
      const bool in = 8 * ch < a.d;
      uint4 w[(G + 1) / 2];
#pragma unroll
      for (int i = 0; i < (G + 1) / 2; ++i) {
        const int h = 2 * i + (lane >> 4);
        w[i] = make_uint4(0u, 0u, 0u, 0u);
        if (in && h < G)
          w[i] = __ldg(reinterpret_cast<const uint4*>(a.q + (hq0 + h) * a.d + 8 * ch));
      }
      if (n >= 2 && !warp_wait(&q_empty[buf], ((n >> 1) - 1) & 1, a.status, &abort_s)) break;
      uint8_t* op = base + S::kOffQ + buf * S::kOpBytes;
#pragma unroll
      for (int i = 0; i < (G + 1) / 2; ++i) {
        const int h = 2 * i + (lane >> 4);
        const uint32_t wv[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
        float x[8], top = 0.f;
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const float2 f = bf16x2_to_float2(wv[u]);
          x[2 * u] = f.x;
          x[2 * u + 1] = f.y;
          top = fmaxf(top, fmaxf(fabsf(f.x), fabsf(f.y)));
        }
#pragma unroll
        for (int m = 8; m > 0; m >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, m));
        // the row times 2^(6 - E): its largest in [2^6, 2^7)
        int E = int((__float_as_uint(top) >> 23) & 0xFFu) - 127;
        E = E < -100 ? -100 : (E > 120 ? 120 : E);
        const float sc = __uint_as_float(uint32_t(133 - E) << 23);
        if (h < G) {
          uint32_t lo[3] = {0u, 0u, 0u}, hi[3] = {0u, 0u, 0u};
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            uint32_t code[3];
            // x 0 is NaN for what is not finite: its code must not saturate
            split2<3>(fmaf(x[2 * u], 0.f, x[2 * u] * sc),
                      fmaf(x[2 * u + 1], 0.f, x[2 * u + 1] * sc), code);
#pragma unroll
            for (int p = 0; p < 3; ++p) (u < 2 ? lo[p] : hi[p]) |= (code[p] & 0xffffu) << (16 * (u & 1));
          }
#pragma unroll
          for (int p = 0; p < 3; ++p)
            *reinterpret_cast<uint2*>(op + op_offset(p * H + h, 8 * ch)) = make_uint2(lo[p], hi[p]);
          if (ch == 0) q_inv[n % kQRing][h] = __uint_as_float(uint32_t(121 + E) << 23);   // 2^(E - 6)
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&q_full[n % kQRing]);
      ++n;
    }
  } else if (warp == 5) {
    // ============================== products ==============================
    constexpr uint32_t idesc_qk = idesc_e4m3(128, N);
    constexpr uint32_t idesc_pv = idesc_e4m3(128, N) | (1u << 15);
    const uint32_t elected = elect_one();
    const uint32_t ring0 = smem_addr(base);
    const uint32_t op_q = ring0 + S::kOffQ, op_p = ring0 + S::kOffP;
    uint32_t it = 0, gt = 0, pt = 0, n = 0;
    bool ok = true, issued = false;
    auto wait = [&](uint64_t* bar, uint32_t parity) {
      return warp_wait(bar, parity, a.status, &abort_s);
    };
    auto qk = [&](uint32_t item, int buf) {
      const uint32_t sb = gt & 1, st = item % kStages;
      if (gt >= 2 && !wait(&s_free[sb], ((gt >> 1) - 1) & 1)) return false;
      if (!wait(&full[st], (item / kStages) & 1)) return false;
      tc_fence_after();
      const uint64_t ad = umma_desc_sw128(ring0 + st * kStageBytes);
      const uint64_t bd = umma_desc_sw128(op_q + buf * S::kOpBytes);
#pragma unroll
      for (int k = 0; k < kW / 32; ++k)
        umma_f8_if(elected, tmem + uint32_t(N) * sb, ad + 2 * k, bd + 2 * k, idesc_qk,
                   k > 0 ? 1u : 0u);
      umma_commit_if(elected, &empty[st]);
      umma_commit_if(elected, &s_full[sb]);
      issued = true;
      ++gt;
      return true;
    };
    for (uint32_t ci = 0; ok; ++ci) {
      const int64_t c = next_chunk(ci);
      if (c < 0 || c >= a.n_chunks) break;
      const int nb = __shfl_sync(0xffffffffu, chunk_of(c, a).nb, 0);
      if (nb == 0) continue;
      const int T = (nb + 1) >> 1, buf = n & 1;
      const uint32_t it0 = it;     // K_t is item it0 + 2 t, V_t the next
      ok = wait(&q_full[n % kQRing], (n / kQRing) & 1) && qk(it0, buf);
      if (!ok) break;
      if (T == 1) umma_commit_if(elected, &q_empty[buf]);
      for (int t = 0; t < T; ++t) {
        // the scores of the next tile, one step ahead of the softmax
        if (t + 1 < T) {
          ok = qk(it0 + 2 * (t + 1), buf);
          if (!ok) break;
          if (t + 2 == T) umma_commit_if(elected, &q_empty[buf]);
        }
        const uint32_t slot = pt % kPSlots, vi = it0 + 2 * t + 1, st = vi % kStages;
        ok = wait(&p_full[slot], (pt / kPSlots) & 1) && wait(&full[st], (vi / kStages) & 1);
        if (!ok) break;
        tc_fence_after();
        const uint64_t ad = umma_desc_sw128_mn(ring0 + st * kStageBytes, 1024);
        const uint64_t bd = umma_desc_sw128(op_p + slot * S::kOpBytes);
        const int steps = 2 * t + 1 < nb ? 4 : 2;   // a lone block: its 64 keys only
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (k < steps)
            umma_f8_if(elected, o_col + uint32_t(N) * buf, ad + k * (32 * kW >> 4), bd + 2 * k,
                       idesc_pv, (t > 0 || k > 0) ? 1u : 0u);
        umma_commit_if(elected, &empty[st]);
        umma_commit_if(elected, &p_free[slot]);
        ++pt;
      }
      if (!ok) break;
      it = it0 + 2u * uint32_t(T);
      umma_commit_if(elected, &o_full[buf]);
      ++n;
    }
    if (issued) {   // every product must be complete before TMEM is freed
      umma_commit_if(elected, &drain);
      (void)mbar_wait_bounded(&drain, 0, a.status);
    }
  } else if (warp < 4) {
    // ====================== softmax and output warps ======================
    const int r = tid;                 // key of a tile; later the output dimension
    const int half = r >> 6, kk = r & 63;
    const uint32_t lane_base = uint32_t(warp * 32) << 16;
    const int64_t hstride = int64_t(a.part_stride) * (a.d + 2);
    uint32_t gt = 0, n = 0;
    bool ok = true;

    // Output rows of the chunk before (its products have had a chunk's time to
    // complete).  A pair that is one chunk is normalised here; otherwise the
    // rows go to the partials.
    bool pend = false;
    Chunk pg{};
    int p_buf = 0;
    uint32_t p_use = 0;
    float pm[G], pM[G], pl[G];
    auto output = [&]() -> bool {
      const bool has_o = pg.nb > 0;
#pragma unroll
      for (int h = 0; h < G; ++h) {
        const float sum = warp_sum(pl[h]);
        if (lane == 0) red[warp][h] = sum;
      }
      bool fail = abort_s != 0;
      if (has_o) fail = !warp_wait(&o_full[p_buf], p_use & 1, a.status, &abort_s);
      if (named_bar_or(1, kSoftThreads, fail)) return false;
      float o[G];
#pragma unroll
      for (int h = 0; h < G; ++h) o[h] = 0.f;
      if (has_o) {
        tc_fence_after();
        float v[32];
        if constexpr (N == 32) {
          tmem_ld32(o_col + lane_base + uint32_t(N) * p_buf, v);
        } else {
          float v16[16];
          tmem_ld16(o_col + lane_base + uint32_t(N) * p_buf, v16);
#pragma unroll
          for (int e = 0; e < 16; ++e) v[e] = v16[e];
        }
        tc_fence_before();
#pragma unroll
        for (int h = 0; h < G; ++h)
          o[h] = fmaf(fmaf(fmaf(v[3 * H + h], 0.0625f, v[2 * H + h]), 0.0625f, v[H + h]), 0.0625f,
                      v[h]);
      }
      const int64_t hq0 = (pg.pair / a.hkv) * a.hq + (pg.pair % a.hkv) * G;
#pragma unroll
      for (int h = 0; h < G; ++h) {
        const float l = (red[0][h] + red[1][h]) + (red[2][h] + red[3][h]);
        // O is in units of 2^M, l of 2^m (no value with a scale: M = -inf)
        const float f = pM[h] == -INFINITY ? 0.f : hw_exp2(pM[h] - pm[h]);
        const float ov = f > 0.f ? o[h] * f : 0.f;
        if (a.chunks_per_pair == 1) {
          if (r < a.d) a.out[(hq0 + h) * a.d + r] = l != 0.f ? ov / l : 0.f;
          if (r == h) a.lse[hq0 + h] = l != 0.f ? (pm[h] + log2f(l)) * kLn2 : -INFINITY;
        } else {
          float* part = a.partials + (hq0 + h) * hstride + int64_t(pg.seg) * (a.d + 2);
          if (r < a.d) part[r] = ov;
          if (r == h) {
            // (a row of NaN, whose maximum may be -inf: with a finite one the
            // merge cannot drop it)
            part[a.d] = isnan(l) ? 0.f : pm[h];
            part[a.d + 1] = l;
          }
        }
      }
      named_bar(1, kSoftThreads);   // red is read before it is written again
      return true;
    };

    for (uint32_t ci = 0; ok; ++ci) {
      const int64_t c = next_chunk(ci);
      // all four warps go on, or none
      if (named_bar_or(1, kSoftThreads, c < 0)) {
        ok = false;
        break;
      }
      if (c >= a.n_chunks) break;
      const Chunk g = chunk_of(c, a);
      const int64_t b = g.pair / a.hkv;
      if (g.bad && g.seg == 0 && r == 0) report(a.status, COBS_ERR_DEVICE);
      const int64_t len_b = kMode == 0 ? a.seq_len
                                       : sequence_length(a.seq_lens, a.seq_len, b, a.status,
                                                         g.seg == 0 && r == 0);
      const int64_t blocks_b = kMode == 0 ? seq_blocks : (len_b + kBlock - 1) / kBlock;
      const int32_t* row = a.idx + g.pair * a.idx_stride + g.s0;
      const int T = (g.nb + 1) >> 1, buf = n & 1;
      float m[G], M[G], l[G], qf[G];
#pragma unroll
      for (int h = 0; h < G; ++h) {
        m[h] = M[h] = -INFINITY;
        l[h] = 0.f;
      }
      const uint32_t v_item0 = 2u * gt + 1u;   // ring item of V_0
      for (int t = 0; t < T; ++t, ++gt) {
        const uint32_t sb = gt & 1, slot = gt % kPSlots, sl = gt % kScaleSlots;
        // this thread's key
        const int blk = 2 * t + half;
        bool valid = false, zero_row = false;
        if (blk < g.nb) {
          const int j = __ldg(row + blk);
          if (j >= 0 && j < blocks_b) {
            valid = int64_t(j) * kBlock + kk < len_b;
            zero_row = kMode != 0 && !valid;
            if constexpr (kMode == 2) {
              // a block without a page (the producer reports it) has no keys
              const int32_t page = __ldg(a.block_table + b * a.table_stride + j);
              if (page < 0 || page >= a.n_pages) valid = zero_row = false;
            }
          } else if (kk == 0) {
            report(a.status, COBS_ERR_DEVICE);
          }
        }
        bool fail = !warp_wait(&s_full[sb], (gt >> 1) & 1, a.status, &abort_s);
        fail = fail || !warp_wait(&sc_full[sl], (gt / kScaleSlots) & 1, a.status, &abort_s);
        fail = fail || (gt >= uint32_t(kPSlots) &&
                        !warp_wait(&p_free[slot], ((gt / kPSlots) - 1) & 1, a.status, &abort_s));
        if (t == 0) {
          fail = fail || !warp_wait(&q_full[n % kQRing], (n / kQRing) & 1, a.status, &abort_s);
#pragma unroll
          for (int h = 0; h < G; ++h) qf[h] = q_inv[n % kQRing][h] * a.scale_log2;
        }
        float s2[G], te[G], mant = 0.f;
        bool raise = false;
        if (!fail) {
          tc_fence_after();
          uint32_t sv[32];
          if constexpr (N == 32) {
            float v[32];
            tmem_ld32(tmem + lane_base + uint32_t(N) * sb, v);
#pragma unroll
            for (int e = 0; e < 32; ++e) sv[e] = __float_as_uint(v[e]);
          } else {
            uint32_t v[16];
            tmem_ld16_nowait(tmem + lane_base + uint32_t(N) * sb, v);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 16; ++e) sv[e] = v[e];
          }
          tc_fence_before();
          const float ksc = valid ? scales[sl][0][r] : 0.f;
          const float vsc = valid ? scales[sl][1][r] : 0.f;
          // vs = mant 2^ev; a row of zeros (scale 0) never moves O's maximum
          const int eb = int(__float_as_uint(vsc) >> 23);
          mant = vsc > 0.f ? __uint_as_float((__float_as_uint(vsc) & 0x7fffffu) | 0x3f800000u) : 0.f;
          const float ev = vsc > 0.f ? float(eb - 127) : -INFINITY;
#pragma unroll
          for (int h = 0; h < G; ++h) {
            const float dot = fmaf(fmaf(__uint_as_float(sv[2 * H + h]), 0.0625f,
                                        __uint_as_float(sv[H + h])),
                                   0.0625f, __uint_as_float(sv[h]));
            s2[h] = valid ? dot * ksc * qf[h] : -INFINITY;
            te[h] = s2[h] + ev;
            raise = raise || s2[h] > m[h] + kRaiseM || te[h] > M[h] + kRaiseO;
          }
        }
        // every warp has its scores in registers
        __syncwarp();
        if (lane == 0) mbar_arrive(&s_free[sb]);
        if (named_bar_or(1, kSoftThreads, raise || fail)) {
          if (named_bar_or(1, kSoftThreads, fail)) {
            ok = false;
            break;
          }
          // the tile's largest per head, then l and O in the new units
#pragma unroll
          for (int h = 0; h < G; ++h) {
            const float x = warp_max(s2[h]), y = warp_max(te[h]);
            if (lane == 0) {
              red[warp][h] = x;
              red[warp][8 + h] = y;
            }
          }
          named_bar(1, kSoftThreads);
          float alpha[G];
#pragma unroll
          for (int h = 0; h < G; ++h) {
            const float x = fmaxf(fmaxf(red[0][h], red[1][h]), fmaxf(red[2][h], red[3][h]));
            const float y = fmaxf(fmaxf(red[0][8 + h], red[1][8 + h]),
                                  fmaxf(red[2][8 + h], red[3][8 + h]));
            const float mn = fmaxf(m[h], x), Mn = fmaxf(M[h], y - kBelowO);
            l[h] *= m[h] == -INFINITY ? 0.f : hw_exp2(m[h] - mn);
            alpha[h] = M[h] == -INFINITY ? 0.f : hw_exp2(M[h] - Mn);
            m[h] = mn;
            M[h] = Mn;
          }
          if (t > 0) {
            // the products of the tiles before must be complete
            const uint32_t pp = gt - 1;
            fail = !warp_wait(&p_free[pp % kPSlots], (pp / kPSlots) & 1, a.status, &abort_s);
            if (named_bar_or(1, kSoftThreads, fail)) {   // also: red has been read
              ok = false;
              break;
            }
            tc_fence_after();
            const uint32_t addr = o_col + lane_base + uint32_t(N) * buf;
#pragma unroll
            for (int p = 0; p < N; p += 16) {
              float v[16];
              tmem_ld16(addr + p, v);
#pragma unroll
              for (int e = 0; e < 16; ++e) {
                const int h = (p + e) % H;
                v[e] *= h < G ? alpha[h] : 0.f;
              }
              tmem_st16(addr + p, reinterpret_cast<const uint32_t*>(v));
            }
            tmem_wait_st();
            tc_fence_before();
          } else {
            named_bar(1, kSoftThreads);   // red is read before it is written again
          }
        }
        // ---- the weights' parts into the P ring ----
        if (blk < g.nb) {   // rows of a missing second block are never read
          uint8_t* op = base + S::kOffP + slot * S::kOpBytes;
#pragma unroll
          for (int h = 0; h < G; h += 2) {
            float w[2] = {0.f, 0.f};
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              if (h + x < G) {
                const float mh = m[h + x < G ? h + x : h], Mh = M[h + x < G ? h + x : h];
                l[h + x < G ? h + x : h] += valid ? hw_exp2(s2[h + x < G ? h + x : h] - mh) : 0.f;
                w[x] = mant > 0.f ? hw_exp2(te[h + x < G ? h + x : h] - Mh) * mant : 0.f;
              }
            }
            uint32_t code[4];
            split2<4>(w[0], w[1], code);
#pragma unroll
            for (int p = 0; p < 4; ++p) {
              op[op_offset(p * H + h, r)] = uint8_t(code[p]);
              if (h + 1 < G) op[op_offset(p * H + h + 1, r)] = uint8_t(code[p] >> 8);
            }
          }
        }
        if (kMode != 0 && named_bar_or(1, kSoftThreads, zero_row)) {
          // rows past the sequence in its last block: zero before P.V
          const uint32_t vi = v_item0 + 2u * uint32_t(t);
          fail = !warp_wait(&full[vi % kStages], (vi / kStages) & 1, a.status, &abort_s);
          if (named_bar_or(1, kSoftThreads, fail)) {
            ok = false;
            break;
          }
          if (zero_row) {
            uint8_t* vt = base + (vi % kStages) * kStageBytes + r * kW;
#pragma unroll
            for (int e = 0; e < kW / 16; ++e)
              reinterpret_cast<uint4*>(vt)[e] = make_uint4(0u, 0u, 0u, 0u);
          }
        }
        fence_proxy_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[slot]);
      }
      if (!ok) break;
      if (pend && !output()) {
        ok = false;
        break;
      }
      pend = true;
      pg = g;
      p_buf = buf;
      p_use = n >> 1;
      if (T > 0) ++n;
#pragma unroll
      for (int h = 0; h < G; ++h) {
        pm[h] = m[h];
        pM[h] = M[h];
        pl[h] = l[h];
      }
    }
    if (ok && pend) (void)output();
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 0) tmem_dealloc(tmem, S::kTmemCols);
}

// Partial rows of a split pair, merged: one CTA per query head, thread r for
// output dimension r, the loads of 8 chunks at a time:
//   M = max m_s, w_s = 2^(m_s - M), out = sum w_s o_s / sum w_s l_s.
template <int D>
__global__ void __launch_bounds__(D) merge_rows_kernel(const DecodeArgs a) {
  constexpr int kB = 8;
  pdl_wait();
  pdl_launch_dependents();
  const int r = threadIdx.x;
  const int64_t hq = blockIdx.x;
  const float* rows = a.partials + hq * (int64_t(a.part_stride) * (D + 2));
  float M = -INFINITY, L = 0.f, O = 0.f;
  for (int s0 = 0; s0 < a.chunks_per_pair; s0 += kB) {
    float m[kB], l[kB], o[kB], top = M;
#pragma unroll
    for (int u = 0; u < kB; ++u) {
      const bool in = s0 + u < a.chunks_per_pair;
      const float* p = rows + int64_t(in ? s0 + u : 0) * (D + 2);
      m[u] = in ? __ldcg(p + D) : -INFINITY;
      l[u] = __ldcg(p + D + 1);
      o[u] = __ldcg(p + r);
      top = fmaxf(top, m[u]);
    }
    if (top == -INFINITY) continue;
    const float f = hw_exp2(M - top);   // 0 while M is -inf
    L *= f;
    O *= f;
    M = top;
#pragma unroll
    for (int u = 0; u < kB; ++u) {
      const float w = m[u] == -INFINITY ? 0.f : hw_exp2(m[u] - M);
      L = fmaf(w, l[u], L);
      O = w > 0.f ? fmaf(w, o[u], O) : O;
    }
  }
  a.out[hq * D + r] = L != 0.f ? O / L : 0.f;   // (not L > 0: NaN stays)
  if (r == 0) a.lse[hq] = L != 0.f ? (M + log2f(L)) * kLn2 : -INFINITY;
}

template <int G>
cudaError_t launch_g(DecodeArgs a, const float* ks, const float* vs, cudaStream_t stream) {
  using S = Shape<G>;
  const bool paged = a.block_table != nullptr;
  const uint64_t rows = paged ? uint64_t(kBlock) : uint64_t(a.seq_len);
  const uint64_t depth = paged ? uint64_t(a.n_pages) * a.hkv : uint64_t(a.batch) * a.hkv;
  const uint64_t depth_bytes = (paged ? uint64_t(kBlock) : uint64_t(a.cap)) * a.d;
  CUtensorMap kmap, vmap;
  cudaError_t e = make_byte_tensor_map_3d_sw128(&kmap, a.k, a.d, rows, depth, depth_bytes, kBlock);
  if (e == cudaSuccess)
    e = make_byte_tensor_map_3d_sw128(&vmap, a.v, a.d, rows, depth, depth_bytes, kBlock);
  if (e != cudaSuccess) return e;
  auto kern = paged ? decode_e4m3_kernel<G, 2>
                    : (a.seq_lens != nullptr ? decode_e4m3_kernel<G, 1> : decode_e4m3_kernel<G, 0>);
  e = set_smem_attrs(kern, S::kDynSmem);
  if (e != cudaSuccess) return e;
  // the bf16 decode's split: a pair is cut only as far as the resident CTAs
  // can still take every chunk in one wave, four blocks a chunk at least (one
  // sequence of 4 pairs: 8.7 us with its lists cut, 256 whole pairs 24.3)
  int sms = device_sm_count();
  if (sms <= 0) sms = 148;
  const int64_t pairs = int64_t(a.batch) * a.hkv;
  const int64_t resident = 2 * int64_t(sms);
  int64_t per_pair = resident / pairs;
  const int64_t most = (a.idx_stride + 3) / 4;
  per_pair = per_pair > most ? most : per_pair;
  per_pair = per_pair < 1 ? 1 : per_pair;
  a.chunk_slots = int32_t((a.idx_stride + per_pair - 1) / per_pair);
  a.chunks_per_pair = (a.idx_stride + a.chunk_slots - 1) / a.chunk_slots;
  a.n_chunks = int32_t(pairs * a.chunks_per_pair);
  a.n_ctas = int32_t(a.n_chunks < resident ? a.n_chunks : resident);
  e = launch_pdl(kern, dim3(a.n_ctas), dim3(kThreads), S::kDynSmem, stream, kmap, vmap, a, ks, vs);
  if (e != cudaSuccess || a.chunks_per_pair == 1) return e;
  return launch_pdl(a.d == 128 ? merge_rows_kernel<128> : merge_rows_kernel<64>,
                    dim3(unsigned(int64_t(a.batch) * a.hq)), dim3(a.d), 0, stream, a);
}

}  // namespace

cudaError_t launch_decode_e4m3(const DecodeArgs& a, const float* ks, const float* vs,
                               cudaStream_t stream) {
  switch (a.hq / a.hkv) {
    case 1: return launch_g<1>(a, ks, vs, stream);
    case 2: return launch_g<2>(a, ks, vs, stream);
    case 4: return launch_g<4>(a, ks, vs, stream);
    case 8: return launch_g<8>(a, ks, vs, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace cobs
