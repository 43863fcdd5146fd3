// pkv_weigh_tc.cu -- accumulated attention weights of many rows (query chunks,
// windows, whole prompts) on the 5th-generation tensor cores.
//
// The formulas are pkv_weigh.cu's.  Scores of many rows do not fit anywhere
// (rows x keys), so both passes compute them, from one kernel:
//  * sums (pass 1): S = Q K^T, 128 query rows (128 / G tokens x the G heads of a
//    kv head) as M, 128 keys as N; a thread has a row's scores and keeps its
//    running maximum and sum.
//  * weights (pass 2): S^T = K Q^T, 128 keys as M, 128 query rows as N; a thread
//    has a key's scores and adds exp2(s - lse) over rows in a register: no sum
//    crosses threads, and none goes through atomics.
// Of either pass two tiles of the M side stay in shared memory (double-buffered:
// the next item's pair lands while this one's rows stream past) and tiles of
// the N side stream through a ring, each used for both: what the tensor cores
// read from L2 is halved.  S goes to TMEM, two buffers for each M tile (all 512
// columns), and from there to the registers of the four warps that own the
// tile's lanes; the buffer is free again as soon as it is read.
//
// Work: a unit is a tile of the N side under a pair of the M side; units in the
// order (sequence, kv head, pair) are cut into equal shares, one a CTA, one CTA
// an SM.  A pair cut between CTAs leaves records (its item + the CTA: unique, as
// one of them grows from piece to piece), joined in CTA order by small kernels:
// pkv_weigh_join_kernel makes the rows' log-sums, pkv_weigh_write_kernel the new
// scores.  A row tile is left out where causality hides the whole key pair.
//
// What bounds it: of a unit of two 128 x 128 x 128 products, 1024 cycles of the
// tensor pipe, operand reads and copies take shared memory about 1300; measured are
// 1700 (pass 1) to 2000, no unit is full, and what the epilogue's chain (score tile
// to registers, maxima, 32 exponentials a thread) takes of the rest has not been
// measured alone.  All rows of a 4095-token prompt, 32
// + 8 heads: 139 us between others in a graph, passes of 67 and 80 under ncu; the
// last 32 rows of eight prompts of 4096 to 8192 tokens 59, K twice from HBM.
//
// E4M3 pages: TMA lands a tile's codes and scale bytes in a staging area, four
// warps widen them to bf16, scale included: exact but for codes without an exponent
// under scale bytes 1 and 2, whose last bits fall below bf16's smallest number
// (2^-133).  What they and the epilogue issue together is what bounds it.
#include <cuda.h>

#include <algorithm>
#include <atomic>
#include <type_traits>

#include "pkv_tcgen05.cuh"
#include "pkv_weigh.cuh"

namespace pkv {
namespace {

constexpr int kTile = 128;            // rows or keys of a tile
constexpr int kPair = 2 * kTile;      // of the M side's pair
constexpr int kTilePages = kTile / kPage;
constexpr uint32_t kHalf = kTile * 128;      // 128 rows of 64 bf16, 128-byte swizzle
constexpr uint32_t kTileBytes = 2 * kHalf;
constexpr uint32_t kColumns = 512;

// Warps: 16 of the epilogue (four for the lanes of the M tiles, four times for
// quarters of their columns; a warp takes first one tile's 32 columns, then the
// other's, so that in pass 2 both use the log-sums that it has read), one each
// for the pairs, the stream, the MMAs and the log-sums, four that widen E4M3
// tiles.
constexpr int kEpilogueWarps = 16;
constexpr int kPairWarp = kEpilogueWarps, kStreamWarp = kPairWarp + 1, kMmaWarp = kPairWarp + 2;
constexpr int kLseWarp = kPairWarp + 3;  // pass 2: log-sums of the row tiles
constexpr int kWidenWarp = kPairWarp + 4, kWidenWarps = 4;
template <bool F8>
constexpr int kTcThreads = 32 * (F8 ? kWidenWarp + kWidenWarps : kWidenWarp);
template <bool F8>
constexpr int kRing = F8 ? 2 : 3;     // tiles of the N side in flight
constexpr int kLseRing = 3;

// Shared memory, from a 1024-byte boundary.
constexpr uint32_t kStagePage = kPage * kHeadDim;
constexpr uint32_t kStageTile = kTilePages * (kStagePage + kScaleBytes);  // codes, then scale bytes
template <bool F8>
struct Smem {
  static constexpr uint32_t pair = 0;                                 // [2][2 tiles]
  static constexpr uint32_t ring = pair + 4 * kTileBytes;
  static constexpr uint32_t stage = ring + kRing<F8> * kTileBytes;    // [2]: codes of both, then scales of both
  static constexpr uint32_t lse = stage + (F8 ? 2 * kStageTile : 0);  // [kLseRing][128], pass 2
  static constexpr uint32_t bars = lse + kLseRing * kTile * 4;
  static constexpr uint32_t total = bars + 256 + 1024;
  static_assert(total <= 232448, "above the 227 KiB of shared memory a CTA can have");
};

// An item's pieces and, in pass 2, its place.
struct Item {
  int32_t b, g, pair, first, last;  // first and last CTA with a piece of it
};

struct TcParams {
  WeighArgs a;
  int32_t small_rows;          // rows x heads that are the few-rows kernels'; 0: they are not launched
  int64_t max_items1, max_items2;
  int64_t* totals;             // [2]: items of pass 1, of pass 2
  Item *items1, *items2;
  float2* records1;            // [items1 + CTAs][4][256]: (maximum, sum) of a row, log2 domain, by column quarter
  float* lse;                  // [items1][256]: -log2 of the rows' sums
  float* records2;             // [items2 + CTAs][4][256]: weight of a key
  int32_t* damaged;            // [num_seqs]: 1 where a page of the sequence is not the pool's
};

// ---- counting units ----------------------------------------------------------

// Sum over i < x of floor(i / 2^k).
__device__ __forceinline__ int64_t floor_sum(int x, int k) {
  const int64_t q = x >> k;
  return ((q * (q - 1) / 2) << k) + q * (x - (q << k));
}

// A sequence as a pass sees it.  A row tile has 2^log_tokens query tokens (8 to
// 128); every size here is a power of two, so that there are no divisions.
template <int PASS>
struct Shape {
  int n, L, context, log_tokens;
  __device__ __forceinline__ int row_tiles() const { return ((n - 1) >> log_tokens) + 1; }
  __device__ __forceinline__ int row_pairs() const { return ((n - 1) >> (log_tokens + 1)) + 1; }
  __device__ __forceinline__ int items() const { return PASS == 1 ? row_pairs() : (L - 1) / kPair + 1; }
  // Pass 2: first row tile that sees a key of the pair.
  __device__ __forceinline__ int first_row_tile(int pair) const {
    return max(0, pair * kPair - context) >> log_tokens;
  }
  // Tiles of the N side for one pair of the M side.
  __device__ __forceinline__ int units(int pair) const {
    if constexpr (PASS == 1)
      return (context + int(min(int64_t(n), (int64_t(pair) + 1) << (log_tokens + 1))) - 1) / kTile + 1;
    else
      return row_tiles() - first_row_tile(pair);
  }
  // Units of the pairs before `pair` (pass 1: not the last one's, which may be short).
  __device__ __forceinline__ int64_t before(int pair) const {
    if constexpr (PASS == 1) {
      // floor((a + i 2^t) / 128) + 1 of pair i, with 2^t tokens a pair
      const int t = log_tokens + 1, a = context + (1 << t) - 1;
      const int64_t triangle = int64_t(pair) * (pair - 1) / 2;
      const int64_t sum = t >= 7 ? int64_t(pair) * (a >> 7) + (triangle << (t - 7))
                                 : floor_sum((a >> t) + pair, 7 - t) - floor_sum(a >> t, 7 - t);
      return sum + pair;
    } else {
      // hidden row tiles of pair i: max(0, i 2^d - e)
      const int d = 8 - log_tokens, e = (context + (1 << log_tokens) - 1) >> log_tokens;
      const int64_t i0 = (e >> d) + 1, x = pair;
      int64_t hidden = 0;
      if (x > i0) hidden = ((x * (x - 1) / 2 - i0 * (i0 - 1) / 2) << d) - e * (x - i0);
      return x * row_tiles() - hidden;
    }
  }
  __device__ __forceinline__ int64_t all() const {
    const int last = items() - 1;
    return before(last) + units(last);
  }
};

// A place in the order of units, and the walk from piece to piece: forward in pass
// 1, backward in pass 2, whose first pairs then are the last keys that pass 1
// read, of which L2 still holds a part.
template <int PASS>
struct Walk {
  Shape<PASS> s;
  int b, q0, g, pair;
  int at;               // pass 1: the piece's first unit in the pair; pass 2: the one behind its last
  int64_t item, item1;  // of this pass; of pass 1 at the sequence's start

  __device__ __forceinline__ bool load(const TcParams& p) {
    WeighSequence x;
    const int G = p.a.desc.num_q_heads / p.a.desc.num_kv_heads;
    if (!weigh_sequence(p.a, b, x) || x.n == 0 || int64_t(x.n) * G <= p.small_rows) return false;
    s = {x.n, x.L, x.L - x.n, __ffs(kTile / G) - 1};
    q0 = x.q0;
    return true;
  }
  // Units of this piece when `left` remain in the CTA's share, and its first.
  __device__ __forceinline__ int count(int64_t left) const {
    return int(min(left, int64_t(PASS == 1 ? s.units(pair) - at : at)));
  }
  __device__ __forceinline__ int first(int count) const { return PASS == 1 ? at : at - count; }
  __device__ __forceinline__ void next(const TcParams& p, int64_t left) {
    const int Hkv = p.a.desc.num_kv_heads;
    if constexpr (PASS == 1) {
      at = 0;
      ++item;
      if (++pair < s.items()) return;
      pair = 0;
      if (++g < Hkv) return;
      g = 0;
      item1 += int64_t(s.row_pairs()) * Hkv;
      ++b;
      if (left > 0)
        while (b < p.a.num_seqs && !load(p)) ++b;
    } else {
      --item;
      if (--pair < 0) {
        if (--g < 0) {
          g = Hkv - 1;
          --b;
          if (left <= 0) return;
          while (b >= 0 && !load(p)) --b;
          item1 -= int64_t(s.row_pairs()) * Hkv;
        }
        pair = s.items() - 1;
      }
      at = s.units(pair);
    }
  }
};

// This CTA's share of units, and its first place, the same in every thread.
// Sequences beyond the workspace are left out and flagged.  `scratch`: 3 x
// (kMaxSeqs + 1) + 3 x warps + 1 int64 in shared memory.
template <int PASS, int kThreads>
__device__ __forceinline__ void plan_shares(const TcParams& p, int64_t* scratch, Walk<PASS>& w, int64_t& share,
                                            bool& idle) {
  const int B = p.a.num_seqs, Hkv = p.a.desc.num_kv_heads, lane = threadIdx.x & 31;
  int64_t *units = scratch, *items1 = scratch + kMaxSeqs + 1, *items2 = items1 + kMaxSeqs + 1;
  auto* warp_sums = reinterpret_cast<int64_t (*)[3]>(items2 + kMaxSeqs + 1);
  auto* limit = reinterpret_cast<unsigned long long*>(warp_sums + kThreads / 32);
  const int per = (B + kThreads - 1) / kThreads;
  const int b0 = min(B, int(threadIdx.x) * per), b1 = min(B, b0 + per);
  int64_t sum[3] = {0, 0, 0}, total[3];  // units, items of pass 1, of pass 2
  bool bad = false;
  for (int b = b0; b < b1; ++b) {
    WeighSequence x;
    bad = !weigh_sequence(p.a, b, x) || bad;
    Walk<PASS> v;
    v.b = b;
    int64_t u = 0, i1 = 0, i2 = 0;
    if (v.load(p)) {
      u = v.s.all() * Hkv;
      i1 = int64_t(v.s.row_pairs()) * Hkv;
      i2 = int64_t((v.s.L - 1) / kPair + 1) * Hkv;
    }
    units[b] = u;
    items1[b] = i1;
    items2[b] = i2;
    sum[0] += u;
    sum[1] += i1;
    sum[2] += i2;
  }
  if (threadIdx.x == 0) limit[0] = B;
  block_scan<kThreads, 3>(sum, total, warp_sums);
  for (int b = b0; b < b1; ++b) {
    const int64_t u = units[b], i1 = items1[b], i2 = items2[b];
    if (i1 > 0 && (sum[1] + i1 > p.max_items1 || sum[2] + i2 > p.max_items2)) {
      atomicMin(limit, static_cast<unsigned long long>(b));
      bad = true;
    }
    units[b] = sum[0];
    items1[b] = sum[1];
    items2[b] = sum[2];
    sum[0] += u;
    sum[1] += i1;
    sum[2] += i2;
  }
  if (threadIdx.x == 0) {
    units[B] = total[0];
    items1[B] = total[1];
    items2[B] = total[2];
  }
  if (PASS == 1 && bad && blockIdx.x == 0) flag_status(p.a.status, PKV_STATUS_BAD_QUERY);
  __syncthreads();
  const int end = int(limit[0]);  // sequences that count
  if (blockIdx.x == 0 && threadIdx.x == 0) p.totals[PASS - 1] = PASS == 1 ? items1[end] : items2[end];
  const int64_t U = units[end], ctas = min(int64_t(gridDim.x), U);
  idle = int64_t(blockIdx.x) >= ctas;
  if (!idle) {
    int64_t rest;
    const int64_t u0 = divide(int64_t(blockIdx.x) * U, ctas, rest);
    const int64_t u1 = divide((int64_t(blockIdx.x) + 1) * U, ctas, rest);
    share = u1 - u0;
    const int64_t from = PASS == 1 ? u0 : u1 - 1;
    int lo = 0, hi = end;  // last sequence with units[b] <= from: it has units
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (units[mid] <= from) lo = mid;
      else hi = mid;
    }
    w.b = lo;
    w.load(p);
    int64_t rem;
    w.g = int(divide(from - units[lo], w.s.all(), rem));
    // last pair with before(pair) <= rem, a warp's lanes trying 32 places at a time
    int first = 0, span = w.s.items();
    while (span > 1) {
      const int step = (span + 31) >> 5;
      const int mid = first + lane * step;
      const uint32_t below = __ballot_sync(0xffffffffu, lane * step < span && w.s.before(mid) <= rem);
      const int last = 31 - __clz(below);  // lane 0's holds always
      first += last * step;
      span = min(step, span - last * step);
    }
    w.pair = first;
    w.at = int(rem - w.s.before(first)) + (PASS == 1 ? 0 : 1);
    w.item1 = items1[lo];
    w.item = (PASS == 1 ? items1[lo] : items2[lo]) + int64_t(w.g) * w.s.items() + first;
  }
  __syncthreads();  // scratch is free
}

// S of one tile pair: all 128 dims, eight MMAs (operands K-major: 32 bytes apart
// in a half's rows, then the other half), and the commit to `bar`.  One block,
// so that a lane is elected once and descriptors are a constant apart: issued
// one by one, with descriptors made anew, they took the warp longer than the
// tensor cores.
__device__ __forceinline__ void umma_tile(uint32_t tmem_d, uint64_t a, uint64_t b, uint32_t idesc, uint64_t* bar) {
  static_assert(kHalf / 16 == 1024, "the block below steps by it");
  asm volatile(
      "{\n\t.reg .pred e, f, t;\n\t.reg .b32 l;\n\t.reg .b64 x, y;\n\t"
      "elect.sync l|e, 0xffffffff;\n\t"
      "setp.ne.b32 f, 0, 0;\n\tsetp.eq.b32 t, 0, 0;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, f;\n\t"
      "add.s64 x, %1, 2;\n\tadd.s64 y, %2, 2;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, t;\n\t"
      "add.s64 x, %1, 4;\n\tadd.s64 y, %2, 4;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, t;\n\t"
      "add.s64 x, %1, 6;\n\tadd.s64 y, %2, 6;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, t;\n\t"
      "add.s64 x, %1, 1024;\n\tadd.s64 y, %2, 1024;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, t;\n\t"
      "add.s64 x, %1, 1026;\n\tadd.s64 y, %2, 1026;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, t;\n\t"
      "add.s64 x, %1, 1028;\n\tadd.s64 y, %2, 1028;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, t;\n\t"
      "add.s64 x, %1, 1030;\n\tadd.s64 y, %2, 1030;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, t;\n\t"
      "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%4];\n\t}" ::"r"(tmem_d),
      "l"(a), "l"(b), "r"(idesc), "r"(smem_u32(bar))
      : "memory");
}

// ---- E4M3 tiles ------------------------------------------------------------------

// Two codes in the high bytes of w's halves, as bf16 times 2^120: the exponent
// field is the code's, so codes without one are bf16 without one.
__device__ __forceinline__ uint32_t as_bf16(uint32_t w) { return ((w >> 4) & 0x07F007F0u) | (w & 0x80008000u); }

__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// Half a row of a staged page, dims 64h .. 64h + 63 of row r times 2^(scale - 127),
// as bf16 into row `out` of the half-h block of a tile (both 128-byte swizzled):
// codes to exponent fields by shifts, one product by a power of two (exact above
// bf16's smallest number, also for codes without an exponent).  The upper half's
// lanes start two pieces on, so that a quarter-warp's stores are on banks of their
// own.
__device__ __forceinline__ void widen_half(const uint8_t* page, uint32_t scale, uint8_t* out, int r, int h) {
  // 2^(scale - 127 + 120), in two steps where that is beyond bf16 (scales above 134)
  const uint32_t s1 = min(scale, 134u), more = scale - s1;
  const uint32_t m1 = ((s1 + 120u) << 7) * 0x00010001u, m2 = ((more + 127u) << 7) * 0x00010001u;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int i = k ^ (2 * h);
    const uint4 v = *reinterpret_cast<const uint4*>(page + r * 128 + (((4 * h + i) ^ (r & 7)) << 4));
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    uint32_t o[8];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      o[2 * j] = mul_bf16x2(as_bf16(__byte_perm(w[j], 0u, 0x1404u)), m1);
      o[2 * j + 1] = mul_bf16x2(as_bf16(__byte_perm(w[j], 0u, 0x3424u)), m1);
    }
    if (more) {
#pragma unroll
      for (int j = 0; j < 8; ++j) o[j] = mul_bf16x2(o[j], m2);
    }
    *reinterpret_cast<uint4*>(out + (((2 * i) ^ (r & 7)) << 4)) = make_uint4(o[0], o[1], o[2], o[3]);
    *reinterpret_cast<uint4*>(out + (((2 * i + 1) ^ (r & 7)) << 4)) = make_uint4(o[4], o[5], o[6], o[7]);
  }
}

// ---- the two passes ------------------------------------------------------------

template <int PASS, bool F8>
__global__ void __launch_bounds__(kTcThreads<F8>, 1)
    pkv_weigh_tc_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
                        const TcParams p) {
  extern __shared__ uint8_t smem_raw[];
  if (threadIdx.x == 0) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&map_q)) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&map_k)) : "memory");
  }
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  using S = Smem<F8>;
  constexpr int kN = kRing<F8>;
  // Planned while the kernel before still runs, where that is one of this call's:
  // it has itself waited for what came before the call, and writes none of the
  // arrays read here; no kernel before reads this pass's total any more.
  if (PASS == 1 && p.small_rows == 0) griddep_wait();
  Walk<PASS> w;
  int64_t left = 0;
  bool idle;
  plan_shares<PASS, kTcThreads<F8>>(p, reinterpret_cast<int64_t*>(sm), w, left, idle);
  if (idle) {
    griddep_wait();
    return;
  }

  uint64_t* bars = reinterpret_cast<uint64_t*>(sm + S::bars);
  uint64_t* pair_full = bars;             // [2]
  uint64_t* pair_free = bars + 2;         // [2]
  uint64_t* ring_full = bars + 4;         // [kN]
  uint64_t* ring_free = ring_full + kN;   // [kN]
  uint64_t* s_full = ring_free + kN;      // [2 tiles][2 buffers]
  uint64_t* s_free = s_full + 4;          // [2][2]
  uint64_t* stage_full = s_free + 4;      // [2], E4M3
  uint64_t* stage_free = stage_full + 2;  // [2]
  uint64_t* lse_full = stage_free + 2;    // [kLseRing], pass 2
  uint64_t* lse_free = lse_full + kLseRing;
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(sm + S::bars + 248);
  static_assert((4 + 2 * 3 + 8 + 4 + 2 * kLseRing) * 8 <= 248, "barriers and the TMEM address share 256 bytes");
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      // K tiles on E4M3 pages are complete by the widening warps' arrivals
      mbar_init(pair_full + i, F8 && PASS == 2 ? 2 * kWidenWarps : 1);
      mbar_init(pair_free + i, 1);
      mbar_init(stage_full + i, 1);
      mbar_init(stage_free + i, kWidenWarps);
    }
    for (int i = 0; i < kN; ++i) {
      mbar_init(ring_full + i, F8 && PASS == 1 ? kWidenWarps : 1);
      mbar_init(ring_free + i, 1);
    }
    for (int i = 0; i < kLseRing; ++i) {
      mbar_init(lse_full + i, 1);
      mbar_init(lse_free + i, kEpilogueWarps);
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(s_full + i, 1);
      mbar_init(s_free + i, kEpilogueWarps);
    }
    fence_mbar_init();
  }
  if (warp == kMmaWarp) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(s_tmem)),
                 "r"(kColumns));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  fence_proxy_async_smem();  // the plan's shared memory is written by copies next
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *s_tmem;
  griddep_wait();

  const WeighArgs& a = p.a;
  const int Hkv = a.desc.num_kv_heads, G = a.desc.num_q_heads / Hkv;
  const int shift = 31 - __clz(G);
  // Tiles of the M side that the pair has.
  auto tiles_of = [&](const Walk<PASS>& x) {
    return (PASS == 1 ? (x.s.n - 1) >> x.s.log_tokens : (x.s.L - 1) / kTile) > 2 * x.pair ? 2 : 1;
  };
  // The table entry of this lane's page (lane < 8) of a key tile, -1 behind the
  // sequence; nothing here waits for it.
  struct Entry {
    int id;
    bool live;
  };
  auto entry_of = [&](const Walk<PASS>& x, int tile) {
    const int page = tile * kTilePages + lane;
    const bool live = lane < kTilePages && page < (x.s.L + kPage - 1) / kPage;
    return Entry{live ? __ldg(a.block_tables + int64_t(x.b) * a.desc.max_blocks_per_seq + page) : -1, live};
  };
  // Its page id; one outside the pool is flagged and page 0 read in its place, and
  // pass 2, which meets every page, marks the sequence: its scores are left alone.
  auto page_id = [&](const Walk<PASS>& x, const Entry& e) {
    if (!e.live || (e.id >= 0 && e.id < a.desc.num_blocks)) return e.id;
    flag_status(a.status, PKV_STATUS_BAD_BLOCK);
    if (PASS == 2) p.damaged[x.b] = 1;
    return 0;
  };
  // A lane's page of a key tile into the tile's buffer, bytes announced before.
  auto copy_page = [&](uint8_t* tile, int id, int g, uint64_t* bar) {
    if (id < 0) return;
    const int row = (id * Hkv + g) * kPage;
    tma_load_2d(tile + lane * 2048, &map_k, 0, row, bar);
    tma_load_2d(tile + kHalf + lane * 2048, &map_k, 64, row, bar);
  };
  auto stage_page = [&](int slot, int id, int g) {
    if (id < 0) return;
    uint8_t* codes = sm + S::stage + slot * kTilePages * kStagePage;
    uint8_t* scales = sm + S::stage + 2 * kTilePages * kStagePage + slot * kTilePages * kScaleBytes;
    const int64_t page = int64_t(id) * Hkv + g;
    tma_load_2d(codes + lane * kStagePage, &map_k, 0, int(page) * kPage, stage_full + slot);
    bulk_copy(scales + lane * kScaleBytes, a.k_scale + page * kScaleBytes, kScaleBytes, stage_full + slot);
  };
  auto copy_rows = [&](uint8_t* tile, const Walk<PASS>& x, int token, uint64_t* bar) {
    for (int h = 0; h < 2; ++h) tma_load_3d(tile + h * kHalf, &map_q, h * 64, x.g * G, x.q0 + token, bar);
  };
  // All lanes wait; a warp goes on only if all saw the phase.
  auto wait_all = [&](uint64_t* bar, uint32_t parity) { return __all_sync(0xffffffffu, mbar_wait(bar, parity)); };
  bool ok = true;

  if (warp == kPairWarp) {
    // ===== the M side's pairs =====
    int staged = 0, i = 0;
    for (; left > 0 && ok; ++i) {
      const int count = w.count(left), tiles = tiles_of(w), slot = i & 1;
      uint8_t* dst = sm + S::pair + slot * 2 * kTileBytes;
      int ids[2];
      if constexpr (PASS == 2) {
        const Entry e0 = entry_of(w, 2 * w.pair), e1 = entry_of(w, 2 * w.pair + 1);
        ids[0] = page_id(w, e0);
        ids[1] = page_id(w, e1);
      }
      if constexpr (PASS == 2 && F8) {
        for (int u = 0; u < tiles && ok; ++u, ++staged) {
          const int st = staged & 1;
          if (staged >= 2 && !(ok = wait_all(stage_free + st, ((staged >> 1) - 1) & 1))) break;
          const int valid = __popc(__ballot_sync(0xffffffffu, ids[u] >= 0));
          if (lane == 0) mbar_arrive_expect_tx(stage_full + st, uint32_t(valid) * (kStagePage + kScaleBytes));
          __syncwarp();
          if (!(kDropFirstCopy && staged == 0)) stage_page(st, ids[u], w.g);
        }
      } else {
        if (i >= 2 && !(ok = wait_all(pair_free + slot, ((i >> 1) - 1) & 1))) break;
        if constexpr (PASS == 1) {
          if (lane == 0) {
            mbar_arrive_expect_tx(pair_full + slot, uint32_t(tiles) * kTileBytes);
            for (int u = 0; u < (kDropFirstCopy && i == 0 ? 0 : tiles); ++u)
              copy_rows(dst + u * kTileBytes, w, (2 * w.pair + u) << w.s.log_tokens, pair_full + slot);
          }
        } else {
          const int valid = __popc(__ballot_sync(0xffffffffu, ids[0] >= 0)) +
                            __popc(__ballot_sync(0xffffffffu, ids[1] >= 0));
          if (lane == 0) mbar_arrive_expect_tx(pair_full + slot, uint32_t(valid) * 4096);
          __syncwarp();
          if (!(kDropFirstCopy && i == 0)) {
            copy_page(dst, ids[0], w.g, pair_full + slot);
            copy_page(dst + kTileBytes, ids[1], w.g, pair_full + slot);
          }
        }
      }
      left -= count;
      w.next(p, left);
    }
    // copies land before the CTA's shared memory is released
    if constexpr (PASS == 2 && F8) {
      for (int k = max(0, staged - 2); k < staged; ++k)
        ok = mbar_wait(stage_full + (k & 1), (k >> 1) & 1, ok ? kLandLimitNs : kDrainLimitNs) && ok;
    } else {
      for (int k = max(0, i - 2); k < i; ++k)
        ok = mbar_wait(pair_full + (k & 1), (k >> 1) & 1, ok ? kLandLimitNs : kDrainLimitNs) && ok;
    }
    if (!ok && lane == 0) flag_status(a.status, PKV_STATUS_TIMEOUT);
  } else if (warp == kStreamWarp) {
    // ===== the N side's tiles =====
    int j = 0;
    while (left > 0 && ok) {
      const int count = w.count(left);
      const int at = w.first(count);
      Entry next{-1, false};
      if constexpr (PASS == 1) next = entry_of(w, at);
      for (int u = 0; u < count; ++u, ++j) {
        if constexpr (PASS == 1) {
          const int now = page_id(w, next);
          if (u + 1 < count) next = entry_of(w, at + u + 1);  // read a tile ahead
          const int valid = __popc(__ballot_sync(0xffffffffu, now >= 0));
          if constexpr (F8) {
            const int st = j & 1;
            if (j >= 2 && !(ok = wait_all(stage_free + st, ((j >> 1) - 1) & 1))) break;
            if (lane == 0) mbar_arrive_expect_tx(stage_full + st, uint32_t(valid) * (kStagePage + kScaleBytes));
            __syncwarp();
            stage_page(st, now, w.g);
          } else {
            const int slot = j % kN;
            if (j >= kN && !(ok = wait_all(ring_free + slot, (j / kN - 1) & 1))) break;
            if (lane == 0) mbar_arrive_expect_tx(ring_full + slot, uint32_t(valid) * 4096);
            __syncwarp();
            copy_page(sm + S::ring + slot * kTileBytes, now, w.g, ring_full + slot);
          }
        } else {
          const int slot = j % kN;
          if (j >= kN && !(ok = wait_all(ring_free + slot, (j / kN - 1) & 1))) break;
          if (lane == 0) {
            const int tile = w.s.first_row_tile(w.pair) + at + u;
            mbar_arrive_expect_tx(ring_full + slot, kTileBytes);
            copy_rows(sm + S::ring + slot * kTileBytes, w, tile << w.s.log_tokens, ring_full + slot);
          }
        }
      }
      left -= count;
      w.next(p, left);
    }
    if constexpr (PASS == 1 && F8) {
      for (int k = max(0, j - 2); k < j; ++k)
        ok = mbar_wait(stage_full + (k & 1), (k >> 1) & 1, ok ? kLandLimitNs : kDrainLimitNs) && ok;
    } else {
      for (int k = max(0, j - kN); k < j; ++k)
        ok = mbar_wait(ring_full + k % kN, (k / kN) & 1, ok ? kLandLimitNs : kDrainLimitNs) && ok;
    }
    if (!ok && lane == 0) flag_status(a.status, PKV_STATUS_TIMEOUT);
  } else if (PASS == 2 && warp == kLseWarp) {
    // ===== log-sums of the row tiles, as many tiles ahead as the ring holds =====
    int j = 0;
    while (left > 0 && ok) {
      const int count = w.count(left);
      const float* src = p.lse + (w.item1 + int64_t(w.g) * w.s.row_pairs()) * kPair +
                         int64_t(w.s.first_row_tile(w.pair) + w.first(count)) * kTile;
      for (int u = 0; u < count; ++u, ++j) {
        const int slot = j % kLseRing;
        if (j >= kLseRing && !(ok = wait_all(lse_free + slot, (j / kLseRing - 1) & 1))) break;
        if (lane == 0) {
          mbar_arrive_expect_tx(lse_full + slot, kTile * 4);
          bulk_copy(sm + S::lse + slot * kTile * 4, src + int64_t(u) * kTile, kTile * 4, lse_full + slot);
        }
      }
      left -= count;
      w.next(p, left);
    }
    for (int k = max(0, j - kLseRing); k < j; ++k)
      ok = mbar_wait(lse_full + k % kLseRing, (k / kLseRing) & 1, ok ? kLandLimitNs : kDrainLimitNs) && ok;
    if (!ok && lane == 0) flag_status(a.status, PKV_STATUS_TIMEOUT);
  } else if (warp == kMmaWarp) {
    // ===== MMAs: the warp runs the loop, one elected lane issues =====
    const uint32_t idesc = idesc_bf16(kTile, kTile, false);
    const uint64_t pair_desc = smem_desc(smem_u32(sm + S::pair), 16, 1024);
    const uint64_t ring_desc = smem_desc(smem_u32(sm + S::ring), 16, 1024);
    int i = 0, j = 0, done[2] = {0, 0}, last_tile = 0;
    for (; left > 0 && ok; ++i) {
      const int count = w.count(left), tiles = tiles_of(w), slot = i & 1;
      if (!(ok = wait_all(pair_full + slot, (i >> 1) & 1))) break;
      for (int u = 0; u < count; ++u, ++j) {
        const int r = j % kN;
        if (!(ok = wait_all(ring_full + r, (j / kN) & 1))) break;
        for (int x = 0; x < tiles; ++x) {
          const int buf = done[x] & 1;
          if (done[x] >= 2 && !(ok = wait_all(s_free + 2 * x + buf, ((done[x] >> 1) - 1) & 1))) break;
          tc_fence_after();
          umma_tile(tmem + x * 256 + buf * 128, pair_desc + ((slot * 2 + x) * kTileBytes >> 4),
                    ring_desc + (r * kTileBytes >> 4), idesc, s_full + 2 * x + buf);
          ++done[x];
          last_tile = x;
        }
        if (!ok) break;
        umma_commit(ring_free + r);
      }
      if (!ok) break;
      umma_commit(pair_free + slot);
      left -= count;
      w.next(p, left);
    }
    // the newest commits arrive before shared memory and TMEM are released
    if (ok) {
      ok = mbar_wait(pair_free + ((i - 1) & 1), ((i - 1) >> 1) & 1, kLandLimitNs) &&
           mbar_wait(ring_free + (j - 1) % kN, ((j - 1) / kN) & 1, kLandLimitNs);
    } else {
      if (done[last_tile] > 0) {
        const int k = done[last_tile] - 1;
        mbar_wait(s_full + 2 * last_tile + (k & 1), (k >> 1) & 1, kDrainLimitNs);
      }
      if (j > 0) mbar_wait(ring_free + (j - 1) % kN, ((j - 1) / kN) & 1, kDrainLimitNs);
      if (i > 0) mbar_wait(pair_free + ((i - 1) & 1), ((i - 1) >> 1) & 1, kDrainLimitNs);
    }
    if (!ok && lane == 0) flag_status(a.status, PKV_STATUS_TIMEOUT);
    __syncwarp();
  } else if (F8 && warp >= kWidenWarp) {
    // ===== E4M3 key tiles to bf16, two pages a warp =====
    if constexpr (F8) {
      const int mine = warp - kWidenWarp;
      int staged = 0, i = 0, j = 0;
      auto widen = [&](uint8_t* tile, const Walk<PASS>& x, int key_tile) {
        const int st = staged & 1;
        if (!wait_all(stage_full + st, (staged >> 1) & 1)) return false;
        const uint8_t* codes = sm + S::stage + st * kTilePages * kStagePage;
        const uint8_t* scales = sm + S::stage + 2 * kTilePages * kStagePage + st * kTilePages * kScaleBytes;
        const int pages = (x.s.L + kPage - 1) / kPage;
        const int r = lane >> 1, h = lane & 1;
#pragma unroll 1
        for (int k = mine; k < kTilePages; k += kWidenWarps)
          if (key_tile * kTilePages + k < pages)
            widen_half(codes + k * kStagePage, scales[k * kScaleBytes + r],
                       tile + h * kHalf + (k * kPage + r) * 128, r, h);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(stage_free + st);
        ++staged;
        return true;
      };
      while (left > 0 && ok) {
        const int count = w.count(left);
        if constexpr (PASS == 1) {
          for (int u = 0; u < count; ++u, ++j) {
            const int slot = j % kN;
            if (j >= kN && !(ok = wait_all(ring_free + slot, (j / kN - 1) & 1))) break;
            if (!(ok = widen(sm + S::ring + slot * kTileBytes, w, w.first(count) + u))) break;
            if (lane == 0) mbar_arrive(ring_full + slot);
          }
        } else {
          const int slot = i & 1, tiles = tiles_of(w);
          if (i >= 2 && !(ok = wait_all(pair_free + slot, ((i >> 1) - 1) & 1))) break;
          for (int u = 0; u < 2; ++u) {
            if (u < tiles && !(ok = widen(sm + S::pair + (slot * 2 + u) * kTileBytes, w, 2 * w.pair + u))) break;
            if (lane == 0) mbar_arrive(pair_full + slot);
          }
          ++i;
        }
        left -= count;
        w.next(p, left);
      }
      if (!ok && lane == 0) flag_status(a.status, PKV_STATUS_TIMEOUT);
    }
  } else if (warp < kEpilogueWarps) {
    // ===== scores to sums or weights =====
    const int quarter = warp >> 2;
    const int r = (warp & 3) * 32 + lane;  // TMEM lane: row or key of a tile
    const uint32_t columns = tmem + quarter * 32 + (uint32_t((warp & 3) * 32) << 16);
    const uint64_t qs2 = f2(a.qscale, a.qscale);
    // A piece's sums and, of its first and its last piece, the item's place.
    auto leave = [&](int count, int at, int tiles, const float (&m)[2], const float (&sum)[2]) {
      const int64_t record = ((w.item + blockIdx.x) * 4 + quarter) * kPair + r;
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        if (x >= tiles) break;
        if constexpr (PASS == 1) p.records1[record + x * kTile] = make_float2(m[x], sum[x]);
        else p.records2[record + x * kTile] = sum[x];
      }
      if (tid == 0) {
        Item& item = (PASS == 1 ? p.items1 : p.items2)[w.item];
        if (at == 0) {
          item.b = w.b;
          item.g = w.g;
          item.pair = w.pair;
          item.first = int(blockIdx.x);
        }
        if (at + count == w.s.units(w.pair)) item.last = int(blockIdx.x);
      }
      left -= count;
      w.next(p, left);
    };
    int j = 0, done[2] = {0, 0};
    while (left > 0 && ok) {
      const int count = w.count(left), at = w.first(count), tiles = tiles_of(w);
      float m[2] = {kWeighNoScore, kWeighNoScore}, sum[2] = {0.f, 0.f};
      // Pass 1: keys up to the row's last one, from the piece's first tile and
      // this quarter on.  Pass 2: the token, from the piece's first row tile on,
      // whose rows are the first to see the thread's key, and the first behind
      // the sequence.  (Of tile 1: the next tokens, the 128th key from there.)
      int seen[2], end = 0;
      if constexpr (PASS == 1) {
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const int token = ((2 * w.pair + x) << w.s.log_tokens) + (r >> shift);
          seen[x] = (token < w.s.n ? w.s.context + token + 1 : INT32_MAX) - at * kTile - quarter * 32;
        }
      } else {
        const int token = (w.s.first_row_tile(w.pair) + at) << w.s.log_tokens;
        seen[0] = w.pair * kPair + r - w.s.context - token;
        seen[1] = seen[0] + kTile;
        end = w.s.n - token;
      }
      for (int u = 0; u < count; ++u, ++j) {
        // (E4M3 blocks have registers for one tile's scores only: read for each)
        constexpr bool kHold = PASS == 2 && !F8;
        uint64_t lse[kHold ? 16 : 1];
        const ulonglong2* sums = nullptr;
        if constexpr (PASS == 2) {
          if (!(ok = wait_all(lse_full + j % kLseRing, (j / kLseRing) & 1))) break;
          sums = reinterpret_cast<const ulonglong2*>(sm + S::lse + ((j % kLseRing) * kTile + quarter * 32) * 4);
          if constexpr (kHold) {
#pragma unroll
            for (int c = 0; c < 8; ++c) {
              const ulonglong2 x = sums[c];
              lse[2 * c] = x.x;
              lse[2 * c + 1] = x.y;
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(lse_free + j % kLseRing);
          }
        }
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          if (x >= tiles) break;
          const int buf = done[x] & 1;
          // Columns [from, to) of the quarter count for this thread.
          int from = 0, to;
          if constexpr (PASS == 1) {
            to = seen[x];
            seen[x] -= kTile;
          } else {
            from = (min(kTile, max(0, seen[x])) << shift) - quarter * 32;
            to = (min(kTile, end) << shift) - quarter * 32;
            seen[x] -= 1 << w.s.log_tokens;
          }
          const bool full = __all_sync(0xffffffffu, from <= 0 && to >= 32);
          const bool none = __all_sync(0xffffffffu, to <= max(0, from) || from >= 32);
          if (!(ok = wait_all(s_full + 2 * x + buf, (done[x] >> 1) & 1))) break;
          ++done[x];
          tc_fence_after();
          uint32_t v[32];
          tmem_ld32(columns + x * 256 + buf * 128, v);
          tmem_wait_ld();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(s_free + 2 * x + buf);
          // MASKED: some columns do not count, their weight is 0 whatever the
          // score or (rows behind the sequence have none) the log-sum is.
          auto add = [&](auto masked_t) {
            constexpr bool MASKED = decltype(masked_t)::value;
            uint32_t which = ~0u;  // bit c: column c counts
            if constexpr (MASKED)
              which = (to <= 0 ? 0u : to >= 32 ? ~0u : (1u << to) - 1u) & (from >= 32 ? 0u : ~0u << max(0, from));
            auto counts = [&](int c) { return (which >> c & 1u) != 0; };
            uint64_t acc[2] = {0ull, 0ull};
            if constexpr (PASS == 1) {
              if constexpr (MASKED) {
#pragma unroll
                for (int c = 0; c < 32; ++c)
                  if (!counts(c)) v[c] = 0xFF800000u;  // -infinity
              }
              // (the maximum times the scale: kept before the product, one that no key
              // has raised would leave fp32's range where scales are large)
              float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
              for (int c = 0; c < 32; c += 4) {
                top[0] = max3(top[0], __uint_as_float(v[c]), __uint_as_float(v[c + 1]));
                top[1] = max3(top[1], __uint_as_float(v[c + 2]), __uint_as_float(v[c + 3]));
              }
              const float mn = fmaxf(m[x], fmaxf(top[0], top[1]) * a.qscale);
              sum[x] *= ex2(m[x] - mn);
              m[x] = mn;
              const uint64_t by = f2(-mn, -mn);
#pragma unroll
              for (int c = 0; c < 32; c += 2) {
                float e0, e1;
                f2_split(f2_fma(f2(__uint_as_float(v[c]), __uint_as_float(v[c + 1])), qs2, by), e0, e1);
                acc[(c >> 1) & 1] = f2_add(acc[(c >> 1) & 1], f2(ex2(e0), ex2(e1)));
              }
            } else {
#pragma unroll
              for (int c = 0; c < 32; c += 2) {
                uint64_t n;
                if constexpr (kHold) n = lse[c >> 1];
                else n = reinterpret_cast<const uint64_t*>(sums)[c >> 1];
                float e0, e1;
                f2_split(f2_fma(f2(__uint_as_float(v[c]), __uint_as_float(v[c + 1])), qs2, n), e0, e1);
                if constexpr (MASKED) {
                  if (!counts(c)) e0 = -INFINITY;
                  if (!counts(c + 1)) e1 = -INFINITY;
                }
                acc[(c >> 1) & 1] = f2_add(acc[(c >> 1) & 1], f2(ex2(e0), ex2(e1)));
              }
            }
            float s0, s1, s2, s3;
            f2_split(acc[0], s0, s1);
            f2_split(acc[1], s2, s3);
            sum[x] += (s0 + s1) + (s2 + s3);
          };
          if (full) add(std::false_type{});
          else if (!none) add(std::true_type{});
        }
        if (!ok) break;
        if constexpr (PASS == 2) {
          end -= 1 << w.s.log_tokens;
          if constexpr (!kHold) {
            __syncwarp();
            if (lane == 0) mbar_arrive(lse_free + j % kLseRing);
          }
        }
      }
      if (!ok) break;
      leave(count, at, tiles, m, sum);
    }
    // Once a wait has run out the sums of its piece and of those behind it are not
    // numbers; their records and items are written all the same: the joining
    // kernels go by what stands there, in a workspace that nobody initialised.
    const float lost[2] = {__uint_as_float(0x7FC00000u), __uint_as_float(0x7FC00000u)}, none[2] = {0.f, 0.f};
#pragma unroll 1
    while (left > 0) {
      const int count = w.count(left);
      leave(count, w.first(count), tiles_of(w), none, lost);
    }
    if (!ok && lane == 0) flag_status(a.status, PKV_STATUS_TIMEOUT);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kColumns));
  }
}

// ---- joining pieces ---------------------------------------------------------------

// A row pair's pieces, in CTA order -> -log2 of its rows' sums.
__global__ void __launch_bounds__(kPair) pkv_weigh_join_kernel(const TcParams p) {
  griddep_launch_dependents();  // pass 2 of the same call, which waits before it reads or writes pools
  griddep_wait();
  if (blockIdx.x == 0)
    for (int b = threadIdx.x; b < p.a.num_seqs; b += kPair) p.damaged[b] = 0;
  const int64_t items = p.totals[0];
  for (int64_t i = blockIdx.x; i < items; i += gridDim.x) {
    const int first = p.items1[i].first, last = p.items1[i].last;
    float m = kWeighNoScore, l = 0.f;
    for (int c = 4 * first; c < 4 * last + 4; ++c) {
      const float2 x = __ldcg(p.records1 + (4 * i + c) * kPair + threadIdx.x);
      const float mn = fmaxf(m, x.x);
      l = l * ex2(m - mn) + x.y * ex2(x.x - mn);
      m = mn;
    }
    p.lse[i * kPair + threadIdx.x] = -(m + __log2f(l));
  }
}

// A key pair's pieces, in CTA order -> its paged scores.
__global__ void __launch_bounds__(kPair) pkv_weigh_write_kernel(const TcParams p) {
  griddep_wait();
  const WeighArgs& a = p.a;
  const int64_t items = p.totals[1];
  for (int64_t i = blockIdx.x; i < items; i += gridDim.x) {
    const Item item = p.items2[i];
    const int damaged = p.damaged[item.b];
    WeighSequence s;
    weigh_sequence(a, item.b, s);
    const int64_t key = int64_t(item.pair) * kPair + threadIdx.x;
    const int from = a.first ? __ldg(a.first + item.b) : 0;
    if (key >= s.L || key < from || damaged) continue;
    const int scored = a.decay == 0.f ? 0 : a.scored ? __ldg(a.scored + item.b) : s.L - s.n;
    const int id = __ldg(a.block_tables + int64_t(item.b) * a.desc.max_blocks_per_seq + key / kPage);
    if (id < 0 || id >= a.desc.num_blocks) continue;  // flagged where its keys were read
    const int64_t at = (int64_t(id) * a.desc.num_kv_heads + item.g) * kPage + key % kPage;
    float sum = 0.f;
    for (int c = 4 * item.first; c < 4 * item.last + 4; ++c)
      sum += __ldcg(p.records2 + (4 * i + c) * kPair + threadIdx.x);
    const float old = key < scored ? __ldcg(a.scores + at) : 0.f;
    a.scores[at] = fmaf(a.decay, old, sum);
  }
  __syncthreads();
  griddep_launch_dependents();
}

// ---- host side ------------------------------------------------------------------

int tile_tokens(const pkv_desc& d) { return kTile / (d.num_q_heads / d.num_kv_heads); }

// Every sequence may end in a part of a pair.
int64_t most_items1(const pkv_desc& d, int32_t num_seqs, int32_t num_tokens) {
  return (int64_t(num_tokens) / (2 * tile_tokens(d)) + std::min(num_seqs, num_tokens)) * d.num_kv_heads;
}
int64_t most_items2(const pkv_desc& d, int32_t num_seqs, int32_t num_tokens, int64_t num_keys) {
  return (num_keys / kPair + std::min(num_seqs, num_tokens)) * d.num_kv_heads;
}

struct TcLayout {
  size_t totals, items1, items2, records1, lse, records2, damaged, total;
};

TcLayout tc_layout(const DeviceInfo& dev, const pkv_desc& d, int32_t num_seqs, int32_t num_tokens, int64_t num_keys) {
  const size_t i1 = size_t(most_items1(d, num_seqs, num_tokens));
  const size_t i2 = size_t(most_items2(d, num_seqs, num_tokens, num_keys));
  TcLayout w{};
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t at = off;
    off = align_up(off + bytes, 256);
    return at;
  };
  w.totals = take(2 * sizeof(int64_t));
  w.items1 = take(i1 * sizeof(Item));
  w.items2 = take(i2 * sizeof(Item));
  w.records1 = take((i1 + dev.sm_count) * 4 * kPair * sizeof(float2));
  w.lse = take(i1 * kPair * sizeof(float));
  w.records2 = take((i2 + dev.sm_count) * 4 * kPair * sizeof(float));
  w.damaged = take(size_t(num_seqs) * sizeof(int32_t));
  w.total = off;
  return w;
}

template <int PASS, bool F8>
int ensure_attr(int device) {
  static std::atomic<bool> done[64] = {};
  if (device < 0 || device >= 64) return PKV_ERR_DEVICE;
  if (!done[device].load(std::memory_order_acquire)) {
    if (cudaFuncSetAttribute(pkv_weigh_tc_kernel<PASS, F8>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             int(Smem<F8>::total)) != cudaSuccess) {
      cudaGetLastError();
      return PKV_ERR_LAUNCH;
    }
    done[device].store(true, std::memory_order_release);
  }
  return PKV_OK;
}

template <class... Params, class... Args>
int launch(const LaunchCtx& ctx, void (*kernel)(Params...), int grid, int threads, size_t smem, const Args&... args) {
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(grid));
  cfg.blockDim = dim3(unsigned(threads));
  cfg.dynamicSmemBytes = smem;
  cfg.stream = ctx.stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  TraceScope ts(ctx.stream, PKV_K_WEIGH);
  cudaLaunchKernelEx(&cfg, kernel, args...);
  return ts.done();
}

template <bool F8>
int run(const LaunchCtx& ctx, const CUtensorMap& q, const CUtensorMap& k, const TcParams& p) {
  if (int e = ensure_attr<1, F8>(ctx.dev->device)) return e;
  if (int e = ensure_attr<2, F8>(ctx.dev->device)) return e;
  const int sms = ctx.dev->sm_count;
  auto blocks = [&](int64_t items) { return int(std::max<int64_t>(1, std::min<int64_t>(items, int64_t(sms) * 8))); };
  if (int e = launch(ctx, pkv_weigh_tc_kernel<1, F8>, sms, kTcThreads<F8>, Smem<F8>::total, q, k, p)) return e;
  if (int e = launch(ctx, pkv_weigh_join_kernel, blocks(p.max_items1), kPair, 0, p)) return e;
  if (int e = launch(ctx, pkv_weigh_tc_kernel<2, F8>, sms, kTcThreads<F8>, Smem<F8>::total, q, k, p)) return e;
  return launch(ctx, pkv_weigh_write_kernel, blocks(p.max_items2), kPair, 0, p);
}

}  // namespace

size_t weigh_tc_workspace_bytes(const DeviceInfo& dev, const pkv_desc& d, int32_t num_seqs, int32_t num_tokens,
                                int64_t num_keys) {
  return tc_layout(dev, d, num_seqs, num_tokens, num_keys).total;
}

int launch_weigh_tc(const LaunchCtx& ctx, const WeighArgs& a, bool fp8, int32_t small_rows, uint8_t* workspace) {
  const pkv_desc& d = a.desc;
  const TcLayout w = tc_layout(*ctx.dev, d, a.num_seqs, a.num_tokens, a.num_keys);
  CUtensorMap q, k;
  {
    const cuuint64_t dims[3] = {cuuint64_t(kHeadDim), cuuint64_t(d.num_q_heads), cuuint64_t(a.num_tokens)};
    const cuuint64_t strides[2] = {cuuint64_t(kHeadDim) * 2, cuuint64_t(d.num_q_heads) * kHeadDim * 2};
    const cuuint32_t box[3] = {64, cuuint32_t(d.num_q_heads / d.num_kv_heads), cuuint32_t(tile_tokens(d))};
    if (!encode_tensor_map(&q, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, a.q, 3, dims, strides, box)) return PKV_ERR_LAUNCH;
  }
  {
    const cuuint64_t dims[2] = {cuuint64_t(kHeadDim), cuuint64_t(d.num_blocks) * d.num_kv_heads * kPage};
    const cuuint64_t strides[1] = {cuuint64_t(kHeadDim) * (fp8 ? 1 : 2)};
    const cuuint32_t box[2] = {cuuint32_t(fp8 ? kHeadDim : kHeadDim / 2), cuuint32_t(kPage)};
    if (!encode_tensor_map(&k, fp8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, a.k_cache, 2,
                           dims, strides, box))
      return PKV_ERR_LAUNCH;
  }
  const TcParams p{a,
                   small_rows,
                   most_items1(d, a.num_seqs, a.num_tokens),
                   most_items2(d, a.num_seqs, a.num_tokens, a.num_keys),
                   reinterpret_cast<int64_t*>(workspace + w.totals),
                   reinterpret_cast<Item*>(workspace + w.items1),
                   reinterpret_cast<Item*>(workspace + w.items2),
                   reinterpret_cast<float2*>(workspace + w.records1),
                   reinterpret_cast<float*>(workspace + w.lse),
                   reinterpret_cast<float*>(workspace + w.records2),
                   reinterpret_cast<int32_t*>(workspace + w.damaged)};
  return fp8 ? run<true>(ctx, q, k, p) : run<false>(ctx, q, k, p);
}

}  // namespace pkv
