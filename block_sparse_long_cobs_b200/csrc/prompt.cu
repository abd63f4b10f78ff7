// Causal attention of packed new tokens over the bf16 cache
// (include/cobs_cache.h, cobs_prompt_attention) on the 5th-generation tensor
// cores.
//
//   out_r = sum_{j <= p_r} e^(s_rj - m_r) v_j / sum_j e^(s_rj - m_r),
//   s_rj = softmax_scale q_r . k_j,
// in one pass over the keys with a running maximum m and sum l per row.
//
// Tiles.  The G query heads of a kv-head share its keys, so a tile's 128 rows
// are 128 / G tokens x G heads; a unit of work is two such tiles (consecutive
// tokens of one sequence and kv-head) against all keys up to the unit's last
// position, 128 keys per iteration.  Per iteration and tile the tensor cores
// form S = Q K^T (M = 128 rows, N = 128 keys) and O += P V (P read from
// tensor memory, half a tile as soon as its weights are there).  The two tiles
// alternate: while one tile's P is formed the tensor cores work for the other.
// A unit of one tile (few rows) gives its even iterations to one softmax
// warpgroup and its odd ones to the other, each with its own S, O, m and l,
// joined at the end.
//   warps 0-3, 4-7  softmax of tile (or stream) 0, 1: one row per thread.  p =
//                   2^(s - m) with m raised only when a row's logit exceeds it
//                   by more than 2^8 (the warp then rescales its rows of O in
//                   tensor memory; the products that wrote them were issued
//                   before the ones that made S, so they are complete).  P
//                   overwrites S as bf16.  No barrier among warps: a row
//                   belongs to one thread from the scores to the output.
//   warp 8          schedule and TMA: Q once per unit, K_i, V_i through a ring
//   warp 9          issues the products
//
// What bounds it: an iteration of two tiles costs the tensor cores 2 x (512 +
// 512) cycles at their peak rate, 256 KB of shared-memory traffic (both
// operands of Q K^T, V, and the tiles coming in), 2048 cycles as well, and 2 x
// 128 x 128 exponentials at 16 a cycle, 2048 too; the kernel takes about 3500.
// Long prompts run into the 1000 W power cap (0.99 to 1.05 PFLOP/s at 1.5 GHz
// for 4096 tokens over 28k, 1.2 PFLOP/s before the clock drops), short ones
// into what starting and ending a unit costs, a few tokens over a long context
// and single tokens into HBM (4.9 to 5.2 and 5.1 to 5.5 TB/s).  Tried
// and slower: half a row per thread with sixteen softmax warps (2.05 against
// 1.97 ms), a quarter or half of the exponentials as a polynomial on the
// multiply-add pipe (2.03, 2.19 ms).
//
// Work split.  The iterations of all units, laid end to end, are cut into
// equal shares, one per CTA (one CTA per SM), so that ragged lengths, causal
// triangles and a few rows over a long context all fill the GPU evenly.  A
// unit that a cut goes through leaves partial rows (o, m, l) in the workspace
// (at most two per CTA), which prompt_merge_kernel joins.  With sequences of
// at most kWholeTokens tokens the shares are whole units instead: cutting them
// costs more than it evens out (one prompt of 1000 tokens 24 us whole, 31 in
// equal shares, 32 single tokens at 1000 tokens 31 and 40, eight prompts 122 and
// 113; at 2000 tokens one prompt 68 and 59, four 215 and 169, 32 single tokens 52
// and 60).
//
// Rows of the last block past a sequence's end are zeroed in the V tile after
// it lands (a zero weight times a NaN is not zero); scores of keys past a
// row's position are masked whatever the key holds.  Every wait is bounded;
// a CTA that gives up records COBS_ERR_TIMEOUT, lets its copies and products
// finish, frees its tensor memory and returns.
#include "cache_device.cuh"
#include "tcgen05_issue.cuh"

namespace cobs {
namespace {

constexpr int kThreads = 384;            // two softmax warpgroups, one for the rest
constexpr int kSoftWarps = 8;
constexpr int kProducerWarp = 8, kMmaWarp = 9;
// Registers: 384 x 168 at launch, of which the softmax threads (a row of 128
// scores each) take 208 and the others keep 80.
constexpr int kSoftRegs = 208, kOtherRegs = 80;
static_assert(32 * kSoftWarps * kSoftRegs + 128 * kOtherRegs <= kThreads * 168, "register split");
constexpr int kTileRows = 128;
constexpr int kKeyShift = 7;
constexpr int kKeys = 1 << kKeyShift;    // keys per iteration
constexpr int kUnitRows = 2 * kTileRows;
constexpr int kMaxCtas = 148;            // one per SM
constexpr int64_t kWholeTokens = 1024;   // longest sequence whose units are never cut
// What starting and ending a unit costs, in iterations.  us with 1, 2, 3 and 4,
// six ragged prompts of up to 4099 tokens:
//   d 128: 32 + 8 heads 391, 347, 353, 358; 64 + 8 762, 719, 704, 735; 8 + 8 123,
//          122, 122, 122
//   d 64:  16 + 16 heads 181, 182, 178, 178; 32 + 4 294, 287, 291, 301
// 1500 tokens over 500 57.2, 56.9, 56.4, 55.2; four of 300 over 3000 62.3, 61.8,
// 62.2, 62.7; twenty of 700 over 1500 (16 + 4) 121, 119, 119, 120.
constexpr int kUnitCost = 2;
// Iterations of a share, at least: 16 tokens at 2000 took 14.2, 15.8 and 19.0 us
// with 2, 4 and 8, two single tokens at 4000 18.6, 18.2 and 20.4.
constexpr int kMinShare = 4;
constexpr int kSegQ = 2;                 // segments handed from the producer to the others
constexpr float kRescaleLog2 = 8.f;
constexpr uint32_t kTmemCols = 512;      // S0, S1 (P over them), O0, O1
constexpr float kLn2 = 0.69314718055994530942f;

template <int D>
struct Tile {
  static constexpr int kSlabs = D / 64;
  static constexpr int kSlabBytes = 128 * 128;          // 128 rows x 64 columns bf16
  static constexpr int kBytes = kSlabs * kSlabBytes;
  static constexpr int kStages = D == 128 ? 5 : 8;
  static constexpr int kOffQ = kStages * kBytes;
  static constexpr int kDynSmem = kOffQ + 2 * kBytes + 1024;
};

// How a segment covers its unit.
enum SegType : int32_t { kNone = 0, kWhole = 1, kBegin = 2, kMiddle = 3, kEnd = 4 };

struct Segment {
  int64_t tok0;    // first packed row
  int64_t pos0;    // its position
  int64_t len;     // tokens of the sequence
  int32_t b, h;    // sequence, kv-head
  int32_t ntok;    // tokens of the unit
  int32_t it0, it1;
  int32_t type;
};

// What a CTA leaves in the workspace beside its partial rows: slot 0 its
// first segment when that does not begin its unit, slot 1 its last when that
// begins one without ending it.
struct SlotNote {
  int64_t tok0;
  int32_t ntok, h;
  int32_t type, pad;
};

// Units of one sequence and kv-head: count rows at positions [len - count,
// len), 2^ks tokens per unit (2^ks = 256 / G).  A unit's iterations cover the
// keys up to its last position, one iteration at least (rows before the
// sequence's start have no key and still need their outputs).
struct SeqUnits {
  int64_t c, count, len;   // c = len - count
  int64_t first;           // first packed row
  int32_t ks;
  __host__ __device__ int64_t units() const { return (count + (int64_t(1) << ks) - 1) >> ks; }
  __host__ __device__ int64_t iters(int64_t u) const {
    const int64_t e = c + ((u + 1) << ks), end = e < len ? e : len;
    const int64_t n = (end + kKeys - 1) >> kKeyShift;
    return n > 1 ? n : 1;
  }
  // Iterations of the first n units.  For a full unit j = u + 1 they are
  // max(1, ceil((c + k j) / 128)), k = 2^ks; with k = 128 / m this is
  // ceil((c' + j) / m), c' = ceil(c / k), and with k = 128 s it is
  // ceil(c / 128) + s j.
  __host__ __device__ int64_t before(int64_t n) const {
    int64_t extra = 0;
    if (n > 0 && n == units()) {   // the last unit may be short
      --n;
      extra = iters(n);
    }
    if (n <= 0) return extra;
    if (ks < kKeyShift) {
      const int ms = kKeyShift - ks;
      const int64_t cp = (c + (int64_t(1) << ks) - 1) >> ks;
      const int64_t n0 = -cp < 0 ? 0 : (-cp > n ? n : -cp);   // units with no key: 1 each
      auto f = [ms](int64_t x) {   // sum of ceil(y / m) over y = 1 .. x
        const int64_t q = x >> ms, r = x - (q << ms);
        return ((q * (q + 1) >> 1) << ms) + r * (q + 1);
      };
      if (n0 == n) return extra + n;
      return extra + n0 + f(cp + n) - f(cp > 0 ? cp : 0);
    }
    const int ss = ks - kKeyShift;
    const int64_t cp = (c + kKeys - 1) >> kKeyShift;
    int64_t n0 = -cp >> ss;
    n0 = n0 < 0 ? 0 : (n0 > n ? n : n0);
    return extra + n0 + (n - n0) * cp + ((n * (n + 1) - n0 * (n0 + 1)) >> 1 << ss);
  }
  // Shares are counted in units (whole) or in iterations, with kUnitCost more
  // for the end of each unit.
  __host__ __device__ int64_t cost(int64_t n) const { return before(n) + kUnitCost * n; }
  __host__ __device__ int64_t weight(bool whole) const { return whole ? units() : cost(units()); }
};

__device__ __forceinline__ SeqUnits seq_units(const PromptArgs& a, int64_t b, int ks,
                                              bool reporter) {
  SeqUnits s;
  s.ks = ks;
  s.first = b;
  s.count = 1;
  if (a.cu != nullptr) {
    // rows outside [0, n_tokens) are nobody's, whatever cu_tokens says
    const int64_t c0 = __ldg(a.cu + b), c1 = __ldg(a.cu + b + 1);
    s.first = c0 < 0 ? 0 : (c0 > a.n_tokens ? a.n_tokens : c0);
    const int64_t end = c1 > a.n_tokens ? a.n_tokens : c1;
    s.count = end > s.first ? end - s.first : 0;
    if (reporter && (c0 != s.first || c1 != s.first + s.count)) report(a.status, COBS_ERR_DEVICE);
  }
  s.len = __ldg(a.seq_lens + b);
  if (s.len < 0 || s.len > a.max_seq_len) {
    if (reporter && s.count > 0) report(a.status, COBS_ERR_DEVICE);
    s.len = s.len < 0 ? 0 : a.max_seq_len;
  }
  s.c = s.len - s.count;
  return s;
}

__device__ __forceinline__ int64_t warp_sum64(int64_t v) {
#pragma unroll
  for (int m = 16; m > 0; m >>= 1) v += __shfl_xor_sync(0xffffffffu, v, m);
  return v;
}

// 16-byte units x (first) and y (second) of a pair: lanes with `bit` clear keep
// x and give y for the partner's x, lanes with it set the other way round.
__device__ __forceinline__ void swap_units(uint4& x, uint4& y, int lane, int bit) {
  const bool up = (lane & bit) != 0;
  uint4 s = up ? x : y;
  s.x = __shfl_xor_sync(0xffffffffu, s.x, bit);
  s.y = __shfl_xor_sync(0xffffffffu, s.y, bit);
  s.z = __shfl_xor_sync(0xffffffffu, s.z, bit);
  s.w = __shfl_xor_sync(0xffffffffu, s.w, bit);
  if (up) x = s;
  else y = s;
}

// A CTA's share of the work: where it starts and how much it is (units when
// `whole`, else iterations).
struct Share {
  int64_t left;
  int32_t b, h, u, it;
};

// The share of CTA blockIdx.x; whole warp.
__device__ __forceinline__ Share find_share(const PromptArgs& a, int lane) {
  const bool whole = a.max_seq_len <= kWholeTokens;
  const int hkv = a.c.hkv;
  const int ks = 8 - __ffs(a.hq / hkv) + 1;
  int64_t total = 0;
  for (int64_t b = lane; b < a.batch; b += 32)
    total += seq_units(a, b, ks, blockIdx.x == 0).weight(whole);
  total = warp_sum64(total) * hkv;
  int64_t n = whole ? total : total / kMinShare;
  n = n < 1 ? 1 : (n > int64_t(gridDim.x) ? int64_t(gridDim.x) : n);
  Share s{};
  if (int64_t(blockIdx.x) >= n) return s;
  const int64_t t0 = total * int64_t(blockIdx.x) / n;
  s.left = total * (int64_t(blockIdx.x) + 1) / n - t0;
  int64_t skipped = 0, w_b = 0;
  for (int64_t b0 = 0; b0 < a.batch && s.left > 0; b0 += 32) {
    const int64_t mine = b0 + lane < a.batch ? b0 + lane : a.batch - 1;
    const int64_t wgt =
        b0 + lane < a.batch ? seq_units(a, mine, ks, false).weight(whole) * hkv : 0;
    int64_t inc = wgt;
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
      const int64_t up = __shfl_up_sync(0xffffffffu, inc, m);
      if (lane >= m) inc += up;
    }
    const uint32_t past = __ballot_sync(0xffffffffu, skipped + inc > t0);
    if (past != 0) {
      const int l = __ffs(past) - 1;
      s.b = int32_t(b0 + l);
      w_b = __shfl_sync(0xffffffffu, wgt, l);
      skipped += __shfl_sync(0xffffffffu, inc - wgt, l);
      break;
    }
    skipped += __shfl_sync(0xffffffffu, inc, 31);
  }
  if (s.left > 0) {
    const SeqUnits su = seq_units(a, s.b, ks, false);
    const int64_t w_h = w_b / hkv;
    s.h = int32_t((t0 - skipped) / w_h);
    const int64_t rest = (t0 - skipped) % w_h;
    if (whole) {
      s.u = int32_t(rest);
    } else {
      int64_t lo = 0, hi = su.units() - 1;   // the last u with cost(u) <= rest
      while (lo < hi) {
        const int64_t mid = (lo + hi + 1) / 2;
        if (su.cost(mid) <= rest) lo = mid;
        else hi = mid - 1;
      }
      s.u = int32_t(lo);
      s.it = int32_t(rest - su.cost(lo));
    }
  }
  return s;
}

// D[tmem] (+)= A[tmem] B: A is bf16, two per column.
__device__ __forceinline__ void umma_bf16_ta_if(uint32_t elected, uint32_t tmem_d,
                                                uint32_t tmem_a, uint64_t bdesc, uint32_t idesc,
                                                uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "setp.ne.b32 e, %5, 0;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(tmem_d),
      "r"(tmem_a), "l"(bdesc), "r"(idesc), "r"(accumulate), "r"(elected)
      : "memory");
}

__device__ __forceinline__ void tmem_ld32_nowait(uint32_t taddr, float* v) {
  uint32_t* r = reinterpret_cast<uint32_t*>(v);
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,"
      "%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]),
        "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]),
        "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]),
        "=r"(r[31])
      : "r"(taddr));
}




__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

template <int I>
struct Index {
  static constexpr int value = I;
};


constexpr size_t slot_floats(int d) { return size_t(kUnitRows) * (d + 2); }

// Partial rows of a slot: o as [D / 4][256 rows][4], then m [256], l [256],
// so that a warp's 32 rows write and read whole lines.
__device__ __forceinline__ float* slot_rows(const PromptArgs& a, int d, int64_t slot) {
  return a.partials + kMaxCtas * 2 * (sizeof(SlotNote) / 4) + slot * slot_floats(d);
}
__device__ __forceinline__ SlotNote* slot_note(const PromptArgs& a, int64_t slot) {
  return reinterpret_cast<SlotNote*>(a.partials) + slot;
}


template <int D, bool kPaged>
__global__ void __launch_bounds__(kThreads, 1)
prompt_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
              const __grid_constant__ CUtensorMap qmap, const __grid_constant__ PromptArgs a) {
  using T = Tile<D>;
  constexpr int kStages = T::kStages;
  extern __shared__ uint8_t dyn_smem[];
  uint8_t* base = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(dyn_smem) + 1023) & ~uintptr_t(1023));
  __shared__ __align__(8) uint64_t full[kStages];
  __shared__ __align__(8) uint64_t empty[kStages];
  __shared__ __align__(8) uint64_t q_full, q_empty, v_tail, drain;
  __shared__ __align__(8) uint64_t s_full[2], p_full[2][2], o_full[2];   // p: halves of the keys
  __shared__ __align__(8) uint64_t ml_full, ml_free;   // one tile: the second stream's sums
  __shared__ __align__(8) uint64_t seg_full[kSegQ], seg_empty[kSegQ];
  __shared__ Segment seg_q[kSegQ];
  __shared__ uint32_t tmem_slot;
  __shared__ volatile int abort_s;
  __shared__ Share share;
  __shared__ float other_ml[2][kTileRows];   // one tile: the second stream's maxima, sums

  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);   // the same in every lane
  const int group = a.hq / a.c.hkv;        // 1, 2, 4 or 8
  const int gs = __ffs(group) - 1;
  const int tt = kTileRows >> gs;          // tokens of a tile

  if (tid == 0) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&kmap)) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&vmap)) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&qmap)) : "memory");
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    mbar_init(&q_full, 1);
    mbar_init(&q_empty, 1);
    mbar_init(&v_tail, 1);
    mbar_init(&drain, 1);
    mbar_init(&ml_full, 4);
    mbar_init(&ml_free, 4);
    for (int w = 0; w < 2; ++w) {
      mbar_init(&s_full[w], 1);
      mbar_init(&p_full[w][0], 4);
      mbar_init(&p_full[w][1], 4);
      mbar_init(&o_full[w], 1);
    }
    for (int s = 0; s < kSegQ; ++s) {
      mbar_init(&seg_full[s], 1);
      mbar_init(&seg_empty[s], kSoftWarps + 1);
    }
    fence_barrier_init();
    abort_s = 0;
  }
  if (warp == 0) tmem_alloc(&tmem_slot, kTmemCols);
  pdl_wait();
  if (warp == kProducerWarp) {
    const Share s = find_share(a, lane);
    if (lane == 0) share = s;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  pdl_launch_dependents();
  const uint32_t tmem = tmem_slot;

  if (warp >= kProducerWarp) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
  if (warp == kProducerWarp) {
    // ==================== schedule and TMA (whole warp) ====================
    const bool whole = a.max_seq_len <= kWholeTokens;
    const int ks = 8 - __ffs(group) + 1;      // tokens of a unit: 256 / G = 2^ks
    const int k_unit = 2 * tt;
    const int hkv = a.c.hkv;
    int64_t left = share.left;
    int32_t b = share.b, h = share.h, u = share.u, it = share.it;
    SeqUnits su = seq_units(a, b, ks, false);
    uint32_t item = 0;       // ring items issued
    uint32_t tails = 0;      // uses of v_tail
    uint32_t nseg = 0;
    SlotNote note[2] = {};
    bool ok = true;
    auto next_unit = [&]() {
      it = 0;
      if (++u < su.units()) return;
      u = 0;
      if (++h < hkv) return;
      h = 0;
      do {
        ++b;
        if (b < a.batch) su = seq_units(a, b, ks, false);
      } while (b < a.batch && su.count == 0);
      if (b >= a.batch) left = 0;
    };
    while (left > 0 && ok) {
      const int64_t n_it = su.iters(u);
      if (it >= n_it) {   // the share starts in what the unit's end costs
        left -= n_it + kUnitCost - it;
        next_unit();
        continue;
      }
      Segment g;
      g.b = b;
      g.h = h;
      g.tok0 = su.first + int64_t(u) * k_unit;
      g.pos0 = su.c + int64_t(u) * k_unit;
      g.len = su.len;
      const int64_t rest = su.count - int64_t(u) * k_unit;
      g.ntok = int32_t(rest < k_unit ? rest : k_unit);
      g.it0 = it;
      g.it1 = int32_t(whole || n_it - it <= left ? n_it : it + left);
      const bool first = g.it0 == 0, last = g.it1 == n_it;
      g.type = first ? (last ? kWhole : kBegin) : (last ? kEnd : kMiddle);
      if (g.type != kWhole) {
        SlotNote& nt = note[g.type == kBegin ? 1 : 0];
        nt.tok0 = g.tok0;
        nt.ntok = g.ntok;
        nt.h = g.h;
        nt.type = g.type;
      }
      left -= whole ? 1 : (last ? n_it + kUnitCost - it : g.it1 - it);
      // ---- hand the segment over ----
      const int qs = nseg % kSegQ;
      if (nseg >= kSegQ &&
          !warp_wait(&seg_empty[qs], ((nseg / kSegQ) - 1) & 1, a.status, &abort_s))
        break;
      if (lane == 0) {
        seg_q[qs] = g;
        mbar_arrive(&seg_full[qs]);
      }
      // ---- the unit's queries ----
      if (nseg > 0 && !warp_wait(&q_empty, (nseg - 1) & 1, a.status, &abort_s)) break;
      ++nseg;
      const int tiles = g.ntok > tt ? 2 : 1;
      if (lane == 0) {
        mbar_arrive_expect_tx(&q_full, uint32_t(tiles * T::kBytes));
        for (int w = 0; w < tiles; ++w)
          for (int s = 0; s < T::kSlabs; ++s)
            tma_load_3d(base + T::kOffQ + w * T::kBytes + s * T::kSlabBytes, &qmap, 64 * s,
                        g.h * group, int(g.tok0 + w * tt), &q_full);
      }
      // ---- keys and values ----
      const int64_t blocks = (g.len + kBlock - 1) / kBlock;
      const int64_t rows_bound = (a.max_seq_len + kBlock - 1) / kBlock * kBlock;
      int32_t page = -1;     // page of block pg0 + lane
      int64_t pg0 = -64;
      for (int i = g.it0; i < g.it1 && ok; ++i) {
        int y[2], z[2];
#pragma unroll
        for (int h2 = 0; h2 < 2; ++h2) {
          const int64_t j = 2 * int64_t(i) + h2;
          bool in = j < blocks;
          if constexpr (kPaged) {
            if (j >= pg0 + 32 || j < pg0) {
              pg0 = j;
              const int64_t jj = j + lane;
              page = jj < blocks ? __ldg(a.c.table + int64_t(b) * a.c.table_stride + jj) : -1;
            }
            const int32_t p = __shfl_sync(0xffffffffu, page, int(j - pg0));
            const bool good = p >= 0 && p < a.c.n_pages;
            if (in && !good && lane == 0) report(a.status, COBS_ERR_DEVICE);
            in = in && good;
            y[h2] = in ? 0 : kBlock;       // past the map's rows: reads as zero
            z[h2] = in ? int(int64_t(p) * hkv + g.h) : 0;
          } else {
            y[h2] = in ? int(j * kBlock) : int(rows_bound);
            z[h2] = int(g.b * hkv + g.h);
          }
        }
        // rows of the sequence's last block past its end hold anything
        const int64_t tail_j = g.len % kBlock != 0 ? blocks - 1 : -1;
        const bool tail = tail_j >= 0 && (tail_j == 2 * int64_t(i) || tail_j == 2 * int64_t(i) + 1);
        for (int kv = 0; kv < 2; ++kv, ++item) {
          const int st = item % kStages;
          if (item >= kStages &&
              !warp_wait(&empty[st], ((item / kStages) - 1) & 1, a.status, &abort_s)) {
            ok = false;
            break;
          }
          uint64_t* bar = kv == 1 && tail ? &v_tail : &full[st];
          uint8_t* dst = base + st * T::kBytes;
          if (lane == 0) {
            const CUtensorMap* map = kv ? &vmap : &kmap;
            mbar_arrive_expect_tx(bar, uint32_t(T::kBytes));
            for (int h2 = 0; h2 < 2; ++h2)
              for (int s = 0; s < T::kSlabs; ++s)
                tma_load_3d(dst + s * T::kSlabBytes + h2 * 8192, map, 64 * s, y[h2], z[h2], bar);
          }
          if (kv == 1 && tail) {
            if (!warp_wait(&v_tail, tails & 1, a.status, &abort_s)) {
              (void)mbar_wait_bounded(&v_tail, tails & 1, a.status);   // let it land
              ok = false;
              ++item;
              break;
            }
            ++tails;
            const int r0 = int(tail_j - 2 * int64_t(i)) * 64 + int(g.len % kBlock);
            const int r1 = int(tail_j - 2 * int64_t(i)) * 64 + 64;
            for (int e = lane; e < (r1 - r0) * 8; e += 32) {
#pragma unroll
              for (int s = 0; s < T::kSlabs; ++s)
                *reinterpret_cast<uint4*>(dst + s * T::kSlabBytes + r0 * 128 + e * 16) =
                    make_uint4(0u, 0u, 0u, 0u);
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&full[st]);
          }
        }
      }
      if (!ok) break;
      if (last) next_unit();
    }
    // the end of the work: an empty segment
    if (ok) {
      const int qs = nseg % kSegQ;
      if (nseg < kSegQ || warp_wait(&seg_empty[qs], ((nseg / kSegQ) - 1) & 1, a.status, &abort_s)) {
        if (lane == 0) {
          seg_q[qs].type = kNone;
          mbar_arrive(&seg_full[qs]);
        }
      }
    }
    if (!whole && lane < 2) *slot_note(a, 2 * int64_t(blockIdx.x) + lane) = note[lane];
    __syncwarp();
    if (abort_s) {
      // copies that were issued and that nobody may have waited for
      if (nseg > 0) (void)mbar_wait_bounded(&q_full, (nseg - 1) & 1, a.status);
    }
    for (uint32_t x = item > uint32_t(kStages) ? item - kStages : 0u; x < item; ++x)
      (void)mbar_wait_bounded(&full[x % kStages], (x / kStages) & 1, a.status);
  } else if (warp == kMmaWarp) {
    // ============================= products ================================
    constexpr uint32_t idesc_qk = umma_idesc_bf16(128, kKeys);
    constexpr uint32_t idesc_pv = umma_idesc_bf16(128, D) | (1u << 16);   // B is MN-major
    const uint32_t elected = elect_one();
    const uint32_t ring0 = smem_addr(base), q0 = ring0 + T::kOffQ;
    uint32_t item = 0, nseg = 0;
    uint32_t np0 = 0, np1 = 0;   // P tiles consumed
    bool ok = true, issued = false;
    auto wait = [&](uint64_t* bar, uint32_t parity) {
      return warp_wait(bar, parity, a.status, &abort_s);
    };
    // S of stream wc = Q of tile qt times the keys in ring slot st.  (A
    // descriptor's address field counts 16 bytes; shared memory ends below
    // 2^18, so adding to it never carries out of its 14 bits.)
    auto qk = [&](auto wc, int qt, uint32_t st) {
      constexpr int w = decltype(wc)::value;
      const uint64_t qd = umma_desc_sw128(q0 + qt * T::kBytes);
      const uint64_t kd = umma_desc_sw128(ring0 + st * T::kBytes);
#pragma unroll
      for (int ks = 0; ks < D / 16; ++ks) {
        const uint32_t off = ((ks >> 2) * T::kSlabBytes + (ks & 3) * 32) >> 4;
        umma_bf16_if(elected, tmem + 128u * w, qd + off, kd + off, idesc_qk, ks > 0 ? 1u : 0u);
      }
      umma_commit_if(elected, &s_full[w]);
      issued = true;
    };
    // O += P V over one tile's keys, a half as soon as its weights are there
    auto pv = [&](auto wc, uint32_t st, uint32_t accumulate, uint32_t parity) {
      constexpr int w = decltype(wc)::value;
      const uint64_t vd = umma_desc_sw128_mn(ring0 + st * T::kBytes, T::kSlabBytes);
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        if (!wait(&p_full[w][half], parity)) return false;
        tc_fence_after();
#pragma unroll
        for (int ks = 4 * half; ks < 4 * half + 4; ++ks)
          umma_bf16_ta_if(elected, tmem + 256u + uint32_t(D) * w, tmem + 128u * w + 8u * ks,
                          vd + ks * (2048 >> 4), idesc_pv, ks > 0 ? 1u : accumulate);
      }
      return true;
    };
    const Index<0> tile0;
    const Index<1> tile1;
    while (ok) {
      const int qs = nseg % kSegQ;
      if (!wait(&seg_full[qs], (nseg / kSegQ) & 1)) break;
      const int type = __shfl_sync(0xffffffffu, seg_q[qs].type, 0);
      const int ntok = __shfl_sync(0xffffffffu, seg_q[qs].ntok, 0);
      const int n_it = __shfl_sync(0xffffffffu, seg_q[qs].it1 - seg_q[qs].it0, 0);
      if (lane == 0) mbar_arrive(&seg_empty[qs]);
      __syncwarp();
      if (type == kNone) break;
      const bool two = ntok > tt;
      const uint32_t item0 = item;       // K_i is ring item item0 + 2 i, V_i the next
      auto slot_of = [&](uint32_t x) { return x % kStages; };
      auto wait_item = [&](uint32_t x) {
        const bool r = wait(&full[x % kStages], (x / kStages) & 1);
        if (r) tc_fence_after();
        return r;
      };
      if (!wait(&q_full, nseg & 1) || !wait_item(item0)) break;
      ++nseg;
      qk(tile0, 0, slot_of(item0));
      if (two) qk(tile1, 1, slot_of(item0));
      umma_commit_if(elected, &empty[slot_of(item0)]);
      if (n_it == 1) umma_commit_if(elected, &q_empty);
      item += 2u * uint32_t(n_it);
      if (two) {
        // both tiles, every iteration
        for (int i = 0; i < n_it; ++i) {
          const uint32_t vi = item0 + 2u * i + 1u, ki = vi + 1u;
          const bool more = i + 1 < n_it;
          ok = wait_item(vi) && pv(tile0, slot_of(vi), i > 0 ? 1u : 0u, np0 & 1);
          if (!ok) break;
          ++np0;
          if (more) {
            ok = wait_item(ki);
            if (!ok) break;
            qk(tile0, 0, slot_of(ki));
          } else {
            umma_commit_if(elected, &o_full[0]);
          }
          ok = pv(tile1, slot_of(vi), i > 0 ? 1u : 0u, np1 & 1);
          if (!ok) break;
          ++np1;
          umma_commit_if(elected, &empty[slot_of(vi)]);
          if (more) {
            qk(tile1, 1, slot_of(ki));
            umma_commit_if(elected, &empty[slot_of(ki)]);
            if (i + 2 == n_it) umma_commit_if(elected, &q_empty);
          } else {
            umma_commit_if(elected, &o_full[1]);
          }
        }
      } else {
        // one tile: stream 0 takes its even iterations, stream 1 the odd ones
        if (n_it > 1) {
          ok = wait_item(item0 + 2u);
          if (!ok) break;
          qk(tile1, 0, slot_of(item0 + 2u));
          umma_commit_if(elected, &empty[slot_of(item0 + 2u)]);
          if (n_it == 2) umma_commit_if(elected, &q_empty);
        }
        auto step = [&](auto wc, int i, uint32_t& np) {
          constexpr int w = decltype(wc)::value;
          const uint32_t vi = item0 + 2u * i + 1u, ki = vi + 3u;   // V_i, K_{i + 2}
          if (!wait_item(vi) || !pv(wc, slot_of(vi), i > 1 ? 1u : 0u, np & 1)) return false;
          ++np;
          umma_commit_if(elected, &empty[slot_of(vi)]);
          if (i + 2 < n_it) {
            if (!wait_item(ki)) return false;
            qk(wc, 0, slot_of(ki));
            umma_commit_if(elected, &empty[slot_of(ki)]);
            if (i + 3 == n_it) umma_commit_if(elected, &q_empty);
          } else {
            umma_commit_if(elected, &o_full[w]);
          }
          return true;
        };
        for (int i = 0; i < n_it && ok; i += 2) {
          ok = step(tile0, i, np0);
          if (ok && i + 1 < n_it) ok = step(tile1, i + 1, np1);
        }
      }
    }
    if (issued) {   // every product must be complete before TMEM is freed
      umma_commit_if(elected, &drain);
      (void)mbar_wait_bounded(&drain, 0, a.status);
    }
    __syncwarp();
  }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftRegs));
    // ======================= softmax and output ===========================
    const int w = warp >> 2;
    const int row = (warp & 3) * 32 + lane;         // of the tile
    const uint32_t lane_base = uint32_t((warp & 3) * 32) << 16;
    const uint32_t s_addr = tmem + lane_base + 128u * w;   // weights over the first 64 columns
    const uint32_t o_addr = tmem + lane_base + 256u + uint32_t(D) * w;
    const uint64_t scale2 = pack2(make_float2(a.scale_log2, a.scale_log2));
    uint32_t nseg = 0, ns = 0, no = 0, joins = 0;
    bool ok = true;
    for (; ok; ++nseg) {
      const int qs = nseg % kSegQ;
      if (!warp_wait(&seg_full[qs], (nseg / kSegQ) & 1, a.status, &abort_s)) break;
      if (seg_q[qs].type == kNone) break;
      // two tiles: each warpgroup has one; one tile: both have its rows, and
      // every second iteration
      const bool two = seg_q[qs].ntok > tt;
      const int tok = (two ? w * tt : 0) + (row >> gs);   // token of the unit
      const int tok_w = (two ? w * tt : 0) + ((warp & 3) * 32 >> gs);   // the warp's first
      const bool busy = tok_w < seg_q[qs].ntok;   // a row of the warp is a token's
      const int it0 = seg_q[qs].it0, it1 = seg_q[qs].it1;
      const int pos = int(seg_q[qs].pos0) + tok;
      const int blocks = int((seg_q[qs].len + kBlock - 1) / kBlock);
      const int32_t* table =
          kPaged ? a.c.table + int64_t(seg_q[qs].b) * a.c.table_stride : nullptr;
      float m = -INFINITY, l = 0.f;
      const int first = two ? it0 : it0 + w, step = two ? 1 : 2;
      for (int i = first; i < it1; i += step, ++ns) {
        // (paged) blocks without a page: their keys are not there
        uint32_t gone = 0;
        if constexpr (kPaged) {
          bool bad = false;
          if (busy && lane < 2 && 2 * i + lane < blocks) {
            const int32_t p = __ldg(table + 2 * i + lane);
            bad = p < 0 || p >= a.c.n_pages;
          }
          gone = __ballot_sync(0xffffffffu, bad);
        }
        if (!warp_wait(&s_full[w], ns & 1, a.status, &abort_s)) {
          ok = false;
          break;
        }
        if (busy) {
          tc_fence_after();
          float s[kKeys];
#pragma unroll
          for (int c = 0; c < kKeys; c += 32) tmem_ld32_nowait(s_addr + c, s + c);
          tmem_wait_ld();
          const int lim = pos - i * kKeys;   // the last key that this row sees
          if (__any_sync(0xffffffffu, lim < kKeys - 1) || (kPaged && gone != 0)) {
#pragma unroll
            for (int c = 0; c < kKeys; ++c)
              if (c > lim || (kPaged && ((gone >> (c >> 6)) & 1u))) s[c] = -INFINITY;
          }
          auto row_max = [&]() {
            float m0 = fmaxf(s[0], s[1]), m1 = fmaxf(s[2], s[3]);
#pragma unroll
            for (int c = 4; c < kKeys; c += 4) {
              m0 = max3(m0, s[c], s[c + 1]);
              m1 = max3(m1, s[c + 2], s[c + 3]);
            }
            return fmaxf(m0, m1) * a.scale_log2;
          };
          // weights 2^(s - m) of 64 keys into tensor memory; returns their sum
          auto weights = [&](int c0) {
            const float neg_m = m == -INFINITY ? 0.f : -m;
            const uint64_t neg_m2 = pack2(make_float2(neg_m, neg_m));
            uint64_t sum_a = 0, sum_b = 0;
#pragma unroll
            for (int c = c0; c < c0 + 64; c += 32) {
              uint32_t p[16];
#pragma unroll
              for (int e = 0; e < 16; ++e) {
                float2 pe = unpack2(
                    fma2(pack2(make_float2(s[c + 2 * e], s[c + 2 * e + 1])), scale2, neg_m2));
                pe = make_float2(hw_exp2(pe.x), hw_exp2(pe.y));
                if (e & 1) sum_b = add2(sum_b, pack2(pe));
                else sum_a = add2(sum_a, pack2(pe));
                p[e] = bf16x2_bits(pe.x, pe.y);
              }
              tmem_st16(s_addr + uint32_t(c / 2), p);
            }
            const float2 t = unpack2(add2(sum_a, sum_b));
            return t.x + t.y;
          };
          auto release = [&](int half) {
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&p_full[w][half]);
          };
          // The first half with the maximum as it was: it moves so rarely that
          // the weights are formed while the new one is still being found, and
          // again in the case that it did move.  (One copy of the code for
          // every case: what runs once a unit comes from a cold instruction
          // cache.)
          float sum;
          bool sure = i == first;
          if (sure) m = row_max();
          for (;;) {
            sum = weights(0);
            if (sure) break;
            const float mx = row_max();
            const bool raise = mx > m + kRescaleLog2;
            sure = __any_sync(0xffffffffu, raise);
            if (!sure) break;
            // the weights that were stored with the old maximum are in place
            // before the new ones go to the same columns (two stores are not
            // ordered by themselves)
            tmem_wait_st();
            const float mn = raise ? mx : m;
            const float alpha = raise ? hw_exp2(m - mn) : 1.f;   // 0 while m is -inf
            m = mn;
            l *= alpha;
#pragma unroll 1
            for (int c = 0; c < D; c += 16) {   // narrow: 128 scores are live
              float o[16];
              tmem_ld16(o_addr + c, o);
#pragma unroll
              for (int e = 0; e < 16; ++e) o[e] *= alpha;
              tmem_st16(o_addr + c, reinterpret_cast<const uint32_t*>(o));
            }
          }
          release(0);
          l += sum + weights(64);
          release(1);
        } else if (lane == 0) {
          mbar_arrive(&p_full[w][0]);
          mbar_arrive(&p_full[w][1]);
        }
        __syncwarp();
      }
      if (!ok) break;
      // ---- the unit's rows (or this segment's part of them) ----
      if (first < it1) {
        if (!warp_wait(&o_full[w], no & 1, a.status, &abort_s)) break;
        ++no;
      }
      float m1 = -INFINITY, l1 = 0.f;    // one tile: the other stream's part of the row
      if (!two && w == 1) {
        // handed to the first warpgroup, which also reads this stream's O
        other_ml[0][row] = m;
        other_ml[1][row] = l;
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&ml_full);
        if (!warp_wait(&ml_free, joins & 1, a.status, &abort_s)) break;
      } else if (!two) {
        if (!warp_wait(&ml_full, joins & 1, a.status, &abort_s)) break;
        m1 = other_ml[0][row];
        l1 = other_ml[1][row];
      }
      // (read again: nothing but the loop's own state stays in registers; given
      // back before the stores, which an arrival would wait for)
      const int type = seg_q[qs].type;
      const int64_t tok0 = seg_q[qs].tok0;
      const int ntok = seg_q[qs].ntok, head0 = seg_q[qs].h * group;
      __syncwarp();
      if (lane == 0) mbar_arrive(&seg_empty[qs]);
      if (busy && (two || w == 0)) {
        tc_fence_after();
        const bool mine = tok < ntok;
        const float mm = fmaxf(m, m1);
        const float w0 = m != -INFINITY ? hw_exp2(m - mm) : 0.f;
        const float w1 = m1 != -INFINITY ? hw_exp2(m1 - mm) : 0.f;
        const float ll = l * w0 + l1 * w1;
        // whether the row has a key is asked of the sum: a NaN among its scores
        // leaves the maximum alone (it may still be -inf), and must come out
        const bool some = ll != 0.f;
        const float inv = type == kWhole ? (some ? 1.f / ll : 0.f) : 1.f;
        const float f0 = w0 * inv, f1 = w1 * inv;
        const int64_t r = (tok0 + tok) * a.hq + head0 + (row & (group - 1));
        float* part = slot_rows(a, D, 2 * int64_t(blockIdx.x) + (type == kBegin ? 1 : 0));
        const int pr = (two ? w * kTileRows : 0) + row;
        // (not from f1 alone: rows of nobody may hold NaN, and the second tile
        // has no columns after its own)
        const bool both = !two && __any_sync(0xffffffffu, m1 != -INFINITY);
        // (not unrolled: four copies of this, run once a unit from a cold
        // instruction cache, took 9000 cycles)
#pragma unroll 1
        for (int c = 0; c < D; c += 32) {
          float o[32];
          __syncwarp();   // rows of nobody skip the stores: together again for the load
          tmem_ld32(o_addr + c, o);
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = f0 != 0.f ? o[e] * f0 : 0.f;
          if (both) {
            float o1[32];
            tmem_ld32(o_addr + uint32_t(D) + c, o1);
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = f1 != 0.f ? fmaf(o1[e], f1, o[e]) : o[e];
          }
          if (type == kWhole) {
            // 32 columns of 4 rows in 4 lanes, transposed in units of 16
            // bytes: each store then covers 64 bytes of 8 rows instead of 16
            // bytes of 32
            uint4 p[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
              p[e] = make_uint4(bf16x2_bits(o[8 * e], o[8 * e + 1]),
                                bf16x2_bits(o[8 * e + 2], o[8 * e + 3]),
                                bf16x2_bits(o[8 * e + 4], o[8 * e + 5]),
                                bf16x2_bits(o[8 * e + 6], o[8 * e + 7]));
            swap_units(p[0], p[1], lane, 1);
            swap_units(p[2], p[3], lane, 1);
            swap_units(p[0], p[2], lane, 2);
            swap_units(p[1], p[3], lane, 2);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int rr = (row & ~3) + e;     // the row of p[e] now
              const int tr = (two ? w * tt : 0) + (rr >> gs);
              if (tr < ntok)
                *reinterpret_cast<uint4*>(
                    a.out + ((tok0 + tr) * a.hq + head0 + (rr & (group - 1))) * D + c + 8 * (lane & 3)) =
                    p[e];
            }
          } else if (mine) {
#pragma unroll
            for (int e = 0; e < 8; ++e)
              reinterpret_cast<float4*>(part)[(c / 4 + e) * kUnitRows + pr] =
                  make_float4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
          }
        }
        if (mine && type == kWhole) {
          if (a.lse != nullptr) a.lse[r] = some ? (mm + log2f(ll)) * kLn2 : -INFINITY;
        } else if (mine) {
          // (a row of NaN: with a finite maximum the merge cannot drop it)
          part[kUnitRows * D + pr] = isnan(ll) ? 0.f : mm;
          part[kUnitRows * (D + 1) + pr] = ll;
        }
        tc_fence_before();
      }
      __syncwarp();
      if (!two && w == 0 && lane == 0) mbar_arrive(&ml_free);
      joins += two ? 0u : 1u;
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 0) tmem_dealloc(tmem, kTmemCols);
}

// Units that were cut, joined: the CTA whose last segment begins a unit
// (slot 1) and the following CTAs' first segments (slot 0) up to the one that
// ends it.  Block (c, y) joins 8 dimensions of the unit that begins in CTA c,
// one row per thread, the loads of 4 segments at a time:
//   M = max m_s, L = sum 2^(m_s - M) l_s, out = sum 2^(m_s - M) o_s / L.
// (One segment after the other it took 28 us for 19 segments of 128 rows.)
constexpr int kMergeDims = 8;
constexpr int kMergeBatch = 4;
template <int D>
__global__ void __launch_bounds__(kUnitRows) prompt_merge_kernel(const PromptArgs a, int n_ctas) {
  __shared__ int n_follow;
  pdl_wait();
  pdl_launch_dependents();
  const int c = blockIdx.x;
  const SlotNote g = *slot_note(a, 2 * int64_t(c) + 1);
  if (g.type != kBegin) return;
  const int r = threadIdx.x;
  // segments that follow the first: up to the first one that ends a unit
  if (r == 0) n_follow = n_ctas - 1 - c;
  __syncthreads();
  if (c + 1 + r < n_ctas && slot_note(a, 2 * int64_t(c + 1 + r))->type == kEnd)
    atomicMin(&n_follow, r + 1);
  __syncthreads();
  const int n_seg = 1 + n_follow;
  const int group = a.hq / a.c.hkv;
  const int tt = kTileRows / group;
  const int tok = r / kTileRows * tt + r % kTileRows / group;
  if (tok >= g.ntok) return;
  const int d0 = blockIdx.y * kMergeDims;
  float M = -INFINITY, L = 0.f, o[kMergeDims] = {};
  for (int s0 = 0; s0 < n_seg; s0 += kMergeBatch) {
    float m[kMergeBatch], l[kMergeBatch], top = M;
    float4 v[kMergeBatch][kMergeDims / 4];
#pragma unroll
    for (int i = 0; i < kMergeBatch; ++i) {
      const int s = s0 + i;
      m[i] = -INFINITY;
      l[i] = 0.f;
#pragma unroll
      for (int e = 0; e < kMergeDims / 4; ++e) v[i][e] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (s < n_seg) {
        const float* part = slot_rows(a, D, 2 * int64_t(c + s) + (s == 0 ? 1 : 0));
        m[i] = __ldcg(part + kUnitRows * D + r);
        l[i] = __ldcg(part + kUnitRows * (D + 1) + r);
#pragma unroll
        for (int e = 0; e < kMergeDims / 4; ++e)
          v[i][e] = __ldcg(reinterpret_cast<const float4*>(part) + (d0 / 4 + e) * kUnitRows + r);
      }
      top = fmaxf(top, m[i]);
    }
    if (top == -INFINITY) continue;
    const float f = hw_exp2(M - top);   // 2^-inf = 0
    M = top;
    L *= f;
#pragma unroll
    for (int e = 0; e < kMergeDims; ++e) o[e] *= f;
#pragma unroll
    for (int i = 0; i < kMergeBatch; ++i) {
      if (m[i] == -INFINITY) continue;
      const float w = hw_exp2(m[i] - M);
      L = fmaf(w, l[i], L);
#pragma unroll
      for (int e = 0; e < kMergeDims / 4; ++e) {
        o[4 * e] = fmaf(w, v[i][e].x, o[4 * e]);
        o[4 * e + 1] = fmaf(w, v[i][e].y, o[4 * e + 1]);
        o[4 * e + 2] = fmaf(w, v[i][e].z, o[4 * e + 2]);
        o[4 * e + 3] = fmaf(w, v[i][e].w, o[4 * e + 3]);
      }
    }
  }
  const int64_t row = (g.tok0 + tok) * a.hq + g.h * group + r % group;
  const float inv = M != -INFINITY ? 1.f / L : 0.f;
  *reinterpret_cast<uint4*>(a.out + row * D + d0) =
      make_uint4(bf16x2_bits(o[0] * inv, o[1] * inv), bf16x2_bits(o[2] * inv, o[3] * inv),
                 bf16x2_bits(o[4] * inv, o[5] * inv), bf16x2_bits(o[6] * inv, o[7] * inv));
  if (blockIdx.y == 0 && a.lse != nullptr)
    a.lse[row] = M != -INFINITY ? (M + log2f(L)) * kLn2 : -INFINITY;
}

// CTAs of a launch: no more than there can be shares.
int prompt_ctas(int64_t n_tokens, int batch, int hkv, int group, int64_t max_seq_len) {
  const int64_t k = 2 * kTileRows / group;
  const int64_t units = (n_tokens / k + (batch < n_tokens ? batch : n_tokens)) * hkv;
  const int64_t shares =
      max_seq_len <= kWholeTokens ? units : units * ((max_seq_len + kKeys - 1) / kKeys);
  return int(shares < kMaxCtas ? shares : kMaxCtas);
}

template <int D>
cudaError_t launch_d(const PromptArgs& a, cudaStream_t stream) {
  using T = Tile<D>;
  const int group = a.hq / a.c.hkv;
  CUtensorMap kmap, vmap, qmap;
  const bool paged = a.c.table != nullptr;
  const uint64_t rows = paged ? uint64_t(kBlock) : uint64_t(a.max_seq_len);
  const uint64_t depth = paged ? uint64_t(a.c.n_pages) * a.c.hkv : uint64_t(a.batch) * a.c.hkv;
  const uint64_t depth_bytes = (paged ? uint64_t(kBlock) : uint64_t(a.c.cap)) * D * 2;
  cudaError_t e = make_bf16_tensor_map_3d_sw128(&kmap, a.c.k, D, rows, depth, depth_bytes, kBlock);
  if (e == cudaSuccess)
    e = make_bf16_tensor_map_3d_sw128(&vmap, a.c.v, D, rows, depth, depth_bytes, kBlock);
  if (e == cudaSuccess)
    e = make_bf16_tensor_map_3d_sw128_box(&qmap, a.q, D, uint64_t(a.hq), uint64_t(a.n_tokens),
                                          uint64_t(D) * 2, uint64_t(a.hq) * D * 2, group,
                                          kTileRows / group);
  if (e != cudaSuccess) return e;
  auto kern = paged ? prompt_kernel<D, true> : prompt_kernel<D, false>;
  e = set_smem_attrs(kern, T::kDynSmem);
  if (e != cudaSuccess) return e;
  const int ctas = prompt_ctas(a.n_tokens, a.batch, a.c.hkv, group, a.max_seq_len);
  e = launch_pdl(kern, dim3(ctas), dim3(kThreads), T::kDynSmem, stream, kmap, vmap, qmap, a);
  if (e != cudaSuccess || a.max_seq_len <= kWholeTokens) return e;
  return launch_pdl(prompt_merge_kernel<D>, dim3(ctas, D / kMergeDims), dim3(kUnitRows), 0,
                    stream, a, ctas);
}

}  // namespace

size_t prompt_partial_bytes(const cobs_dims* d, int64_t n_tokens, int64_t max_seq_len) {
  if (n_tokens == 0 || max_seq_len <= kWholeTokens) return 0;
  const int ctas = prompt_ctas(n_tokens, d->batch, d->num_kv_heads,
                               d->num_q_heads / d->num_kv_heads, max_seq_len);
  return kMaxCtas * 2 * sizeof(SlotNote) + size_t(ctas) * 2 * slot_floats(d->head_dim) * 4;
}

cudaError_t launch_prompt(const PromptArgs& a, cudaStream_t stream) {
  return a.d == 128 ? launch_d<128>(a, stream) : launch_d<64>(a, stream);
}

}  // namespace cobs
