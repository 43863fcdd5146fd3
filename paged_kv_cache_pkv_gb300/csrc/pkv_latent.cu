// pkv_latent.cu -- attention over latent pages in the absorbed form: one
// vector of 576 values a cached token is the key of every query head, and its
// first 512 values are the value of every head.
//
//   s[r][k] = scale * q[r] . row[k]            r a (query token, head) pair
//   o[r]    = sum_k softmax_k(s[r][k]) row[k][0:512],  keys k visible to r
//
// What bounds it: a key's 1152 bytes serve H rows of 2 * (576 + 512) FLOPs
// each, so one query token a sequence at 128 heads is just below the ridge
// of this GPU (242 FLOP a byte) and fewer heads are bound by HBM; several
// query tokens a sequence are bound by the tensor cores.
//
// Design:
//  * Rows of a sequence (token-major, then head: contiguous in q and out) are
//    cut into tiles of N = 16, 32, 48 or 64 rows, so any head count fits.  A
//    tile needs 512 x N fp32 of accumulators and one SM's TMEM holds
//    512 x 128, all of it: N = 64 leaves room for two score tiles.  Sequences
//    of more than 64 rows go to pairs of CTAs (pkv_latent_pair.cu) unless they
//    are short.
//  * The products are computed transposed, with the cache tile as the A
//    operand of both, straight from shared memory as TMA landed it:
//      S^T [64 keys x N] = K Q^T      9 x 4 tcgen05.mma, M = 64, K-major A
//      O^T [512 x N]    += V^T P^T    4 blocks of M = 128 dims, MN-major A
//    Few rows then cost little (N is the short side), where rows as M would
//    pad them to 64 or 128, and one copy of the tile serves both products.
//    At N = 64 a tile takes 2500 cycles of shared-memory reads by the two
//    products, which bounds it; 64 sequences of 512-4096 tokens take 36, 44
//    and 53 us at 16, 32 and 64 heads, and their bytes 23, 26 and 27.
//  * A cache tile is 64 keys = 4 pages.  One TMA box a page, from the pool
//    viewed as [groups of 8 rows][9 chunks of 64 dims][8 rows][64 dims], so
//    that each (group, chunk) lands as one 128-byte-swizzled 1 KiB atom and
//    atoms follow each other at one stride along keys (9 KiB) and along dims
//    (1 KiB), as both products' descriptors need.  (Five smaller boxes a page,
//    which would let the scores start earlier, were slower: TMA spends 56-70
//    cycles a box.)  Two tiles are in flight, let go of and refilled page by
//    page as P V gets through them, and the pages of the next tile are asked
//    into L2 meanwhile (long tail 239 us without that, 219 with it; two or
//    three tiles ahead it was slower again).
//  * P of a tile overwrites the tile's rotated chunk, which only the scores
//    read: it needs no buffer of its own and never waits for the P V before.
//  * Softmax without a row maximum a tile.  In S^T a row's scores lie across
//    lanes and warps, where a maximum costs shuffles; but P needs only some
//    reference m near the row's maximum: p = 2^(s - m) has the same relative
//    precision in bf16 whatever its size.  m is the score of the piece's first
//    key, and is raised (and O^T rescaled) only where a later score exceeds it
//    by more than 2^kLtTau; otherwise a tile needs one vote.
//    Row sums add the rounded p in fp32, a partial sum a thread, joined once
//    at the end of a tile of rows.
//  * P is one bf16 term: rounding it (2^-9 a value, independent from key to
//    key) adds as much error as rounding the output to bf16 does, and a
//    second term would double the larger product's cost.
//  * Two warpgroups run the softmax, each for half of the rows; a thread has
//    one key and N/4 rows (16x32bx2 loads: lanes 0-15 and 16-31 read the
//    same keys' two column halves).  One warp loads, one issues the scores'
//    MMAs and one the values': in one warp P V stood behind scores that waited
//    for copies that waited for P V.
//  * Work split (stream-K): tiles of rows laid end to end, each weighing its
//    keys plus a constant, are cut into equal shares, one a CTA; a share may
//    start or end inside a tile.  (Few tiles are split each by itself, see
//    lt_plan.)  Pieces of a cut tile leave fp32 partials (m, l, O) in the
//    workspace that a merge kernel joins; whole tiles are written at once.  A
//    CTA cuts at most two tiles, so the partials do not grow with the batch,
//    and the joining order is fixed.
//  * Every mbarrier wait is bounded; on expiry the role flags
//    PKV_STATUS_TIMEOUT, what is in flight lands, TMEM is freed.
#include <algorithm>
#include <mutex>

#include "pkv_internal.h"
#include "pkv_latent.cuh"
#include "pkv_latent_merge.cuh"

namespace pkv {
namespace {

constexpr int kLtKeys = 64;                        // keys a cache tile
constexpr int kLtPages = kLtKeys / kPage;          // 4
constexpr int kLtSoftmaxThreads = 256;
constexpr int kLtThreads = kLtSoftmaxThreads + 96;  // + loader, score and value warps
constexpr uint32_t kLtGroupBytes = kLtChunks * 1024;         // 8 rows
constexpr uint32_t kLtPageBytes = 2 * kLtGroupBytes;         // 18 KiB
constexpr uint32_t kLtTileBytes = kLtPages * kLtPageBytes;   // 72 KiB
constexpr int kLtStages = 2;
// P of a tile overwrites the tile's rotated chunk, which only the scores read:
// 64 keys of 128 bytes, at the same strides, so P needs no memory of its own
// and never waits for the P V before it.
constexpr uint32_t kLtChunkP = (kLtChunks - 1) * 1024;
constexpr int kLtPairTokens = 2048;  // table width in tokens from which pairs of CTAs take over (a quarter over context)
constexpr float kLtTau = 20.0f;  // log2 of how far a score may exceed the reference

// Shared memory (offsets from a 1024-byte aligned base).
template <int N>
struct LtSmem {
  static constexpr uint32_t kv = 0;
  static constexpr uint32_t q = kv + kLtStages * kLtTileBytes;  // [9][N rows][128 B]
  static constexpr uint32_t misc = q + kLtChunks * N * 128;
  // misc: barriers, TMEM address, plan, per-row reductions
  static constexpr uint32_t bars = misc;           // 16 x 8
  static constexpr uint32_t tmem = misc + 128;
  static constexpr uint32_t plan = misc + 144;     // LtPlan
  static constexpr uint32_t wsum = misc + 272;     // [2][11] x 16, plan scans
  static constexpr uint32_t red = misc + 624;      // [4 quadrants][N] floats
  static constexpr uint32_t alpha = red + 16 * N;  // [N] floats
  static constexpr uint32_t end = alpha + 4 * N;
  static constexpr uint32_t bytes = end + 1024;    // + alignment slack
};
static_assert(LtSmem<64>::bytes <= 232448, "latent attention shared memory above the 227 KiB limit");


// tcgen05.ld of X columns: lanes 0-15 read theirs from taddr on, lanes 16-31
// the same TMEM lanes' columns SPLIT further on.
#define PKV_LD_SPLIT(SPLIT)                                                                       \
  if constexpr (X == 4)                                                                           \
    asm volatile("tcgen05.ld.sync.aligned.16x32bx2.x4.b32 {%0, %1, %2, %3}, [%4], " #SPLIT ";"    \
                 : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3])                                 \
                 : "r"(taddr));                                                                   \
  else if constexpr (X == 8)                                                                      \
    asm volatile(                                                                                 \
        "tcgen05.ld.sync.aligned.16x32bx2.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8], " #SPLIT \
        ";"                                                                                       \
        : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]),     \
          "=f"(r[7])                                                                              \
        : "r"(taddr));                                                                            \
  else                                                                                            \
    asm volatile(                                                                                 \
        "tcgen05.ld.sync.aligned.16x32bx2.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, " \
        "%11, %12, %13, %14, %15}, [%16], " #SPLIT ";"                                            \
        : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]),     \
          "=f"(r[7]), "=f"(r[8]), "=f"(r[9]), "=f"(r[10]), "=f"(r[11]), "=f"(r[12]),              \
          "=f"(r[13]), "=f"(r[14]), "=f"(r[15])                                                   \
        : "r"(taddr));

// N/4 score columns a thread: columns c0.. for lanes 0-15, c0 + N/4.. for 16-31.
template <int N>
__device__ __forceinline__ void lt_load_scores(uint32_t taddr, float (&s)[N / 4]) {
  float* r = s;
  if constexpr (N == 16) {
    constexpr int X = 4;
    PKV_LD_SPLIT(4)
  } else if constexpr (N == 32) {
    constexpr int X = 8;
    PKV_LD_SPLIT(8)
  } else if constexpr (N == 48) {
    {
      constexpr int X = 8;
      PKV_LD_SPLIT(12)
    }
    r += 8;
    taddr += 8;
    {
      constexpr int X = 4;
      PKV_LD_SPLIT(12)
    }
  } else {
    constexpr int X = 16;
    PKV_LD_SPLIT(16)
  }
}
#undef PKV_LD_SPLIT

__device__ __forceinline__ void tmem_ld8(uint32_t taddr, float* r) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]),
                 "=f"(r[7])
               : "r"(taddr));
}
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const float* r) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr),
               "f"(r[0]), "f"(r[1]), "f"(r[2]), "f"(r[3]), "f"(r[4]), "f"(r[5]), "f"(r[6]), "f"(r[7]));
}
// X columns (a multiple of 8) of this warp's 32 lanes.
template <int X>
__device__ __forceinline__ void tmem_ld_cols(uint32_t taddr, float (&r)[X]) {
#pragma unroll
  for (int i = 0; i < X; i += 8) tmem_ld8(taddr + i, r + i);
}

__device__ __forceinline__ void tma_load_4d(void* dst, const CUtensorMap* map, int c0, int c1, int c2, int c3,
                                            uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, "
      "{%2, %3, %4, %5}], [%6];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(smem_u32(bar))
      : "memory");
}

// Bytes that a phase of the barrier waits for, beside its arrivals.
__device__ __forceinline__ void mbar_expect_tx(uint64_t* bar, uint32_t bytes) {
  asm volatile("mbarrier.expect_tx.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(smem_u32(bar)), "r"(bytes) : "memory");
}

template <int N>
__global__ void __launch_bounds__(kLtThreads, 1)
    pkv_latent_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_kv,
                      const LatentParams p) {
  using S = LtSmem<N>;
  constexpr int NC = N / 4;  // score columns a thread
  constexpr int NW = N / 2;  // rows a softmax warpgroup
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(sm + S::bars);
  uint64_t* bar_q = bars;            // a tile's queries landed
  uint64_t* bar_qfree = bars + 1;    // its score MMAs are done
  uint64_t* bar_kv = bars + 2;       // [2] cache tile landed
  uint64_t* bar_kvfree = bars + 4;   // [2][4] the MMAs that read a page of it are done
  uint64_t* bar_s = bars + 12;       // [2] scores written
  uint64_t* bar_p = bars + 14;       // [2] P written (256 arrivals)
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(sm + S::tmem);
  LtPlan* plan = reinterpret_cast<LtPlan*>(sm + S::plan);
  longlong2* s_wsum = reinterpret_cast<longlong2*>(sm + S::wsum);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

  if (tid == 0) {
    for (int i = 0; i < 16; ++i) mbar_init(bars + i, bars + i == bar_p || bars + i == bar_p + 1 ? kLtSoftmaxThreads : 1);
    fence_mbar_init();
  }
  if (warp == 9) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(s_tmem)),
                 "r"(512u));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  if (warp == 8 && lane == 0) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tm_kv)) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tm_q)) : "memory");
  }
  if (warp == 10) {
    // The block tables into L2, shared among the CTAs: the first page ids
    // then come 2500 cycles sooner.  (A hint: what the stream does before may
    // still write them.)
    const char* tables = reinterpret_cast<const char*>(p.block_tables);
    const int64_t bytes = int64_t(p.B) * p.max_blocks * 4;
    for (int64_t i = (int64_t(blockIdx.x) * 32 + lane) * 128; i < bytes; i += int64_t(gridDim.x) * 32 * 128)
      asm volatile("prefetch.global.L2 [%0];" ::"l"(tables + i));
  }
  // The lengths, query starts and tables are not what the call right before
  // this one writes, so the plan need not wait for it.
  lt_plan<N, kLtKeys, kLtThreads>(p, int(blockIdx.x), int(gridDim.x), s_wsum, plan);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *s_tmem;
  const LtPos begin = plan->begin, end = plan->end;
  const LtWalk first{begin, end, lt_seq<N>(p, begin.b, plan->q0, plan->q1, plan->L)};
  // The merge kernel may be scheduled; it waits for this grid.  A kernel that
  // is not this library's may write before it waits, to memory that the caller
  // has back once this call is behind it on the stream: what follows the call
  // is let in no sooner than the call has read everything.
  if (p.joins) griddep_launch_dependents();
  auto tmem_s = [&](int g) { return tmem + 256u + uint32_t(g & 1) * 64u; };

  // every lane waits; the warp goes on only if all of them saw the phase
  auto wait_all = [&](uint64_t* bar, uint32_t parity) {
    return __all_sync(0xffffffffu, mbar_wait(bar, parity));
  };

  if (warp == 8) {
    // ===== loader: queries and cache tiles, in the order they are used =====
    LtWalk walk = first;
    LtPiece x;
    int g = 0, pieces = 0;  // cache tiles and tiles of rows so far
    int landing = 0;        // cache tiles whose copies were issued
    bool ok = true;
    while (ok && lt_next<N, kLtKeys>(p, walk, x)) {
      const int32_t* table = p.block_tables + int64_t(x.b) * p.max_blocks;
      const int pages = (x.L + kPage - 1) / kPage;
      // lane l: page l of a group of eight cache tiles, read a group ahead.
      // -1 past the sequence (no copy); an id that is no page of the pool is
      // flagged and page 0 is read in its place.
      auto group_id = [&](int k) {
        const int i = k * kLtPages + lane;
        if (i >= x.k1 * kLtPages || i >= pages) return -1;
        int id = __ldg(table + i);
        if (id < 0 || id >= p.num_blocks) {
          flag_status(p.status, PKV_STATUS_BAD_BLOCK);
          id = 0;
        }
        return id;
      };
      // (before the wait below: the reads take longer than what is left of the
      // piece before)
      int ids = group_id(x.k0), next = group_id(x.k0 + 8);
      if (pieces == 0) {
        // the first tile's pages into L2 (a hint), then what the stream did
        // before: the queries, this step's rows
        if (lane < kLtPages && ids >= 0)
          prefetch_l2(p.cache + size_t(ids) * (kPage * kLatentRow), kLtPageBytes);
        griddep_wait();
      }
      if (lane == 0) {
        if (pieces > 0) ok = mbar_wait(bar_qfree, (pieces - 1) & 1);
        if (ok) {
          mbar_arrive_expect_tx(bar_q, kLtChunks * N * 128);
          if (!(kDropFirstCopy && pieces == 0)) tma_load_3d(sm + S::q, &tm_q, 0, x.row0, 0, bar_q);
        }
      }
      ok = __shfl_sync(0xffffffffu, int(ok), 0) != 0;
      ++pieces;
      for (int k = x.k0; ok && k < x.k1; ++k, ++g) {
        const int in_group = (k - x.k0) & 7;
        if (k > x.k0 && in_group == 0) {
          ids = next;
          next = group_id(k + 8);
        }
        int id[kLtPages];
        int valid = 0;
#pragma unroll
        for (int i = 0; i < kLtPages; ++i) {
          id[i] = __shfl_sync(0xffffffffu, ids, in_group * kLtPages + i);
          valid += id[i] >= 0;
        }
        const int st = g % kLtStages;
        if (lane == 0) {
          // page by page, as P V of the tile two before lets go of them.  The
          // arrival comes behind the last page's wait, also where that page
          // is not loaded: what follows it writes P over all four, and zeros
          // behind the sequence's end.
          int sent = 0;
#pragma unroll
          for (int i = 0; i < kLtPages; ++i) {
            if (g >= kLtStages && ok) ok = mbar_wait(bar_kvfree + st * kLtPages + i, (g / kLtStages - 1) & 1);
            if (!ok) break;
            if (i == 0) mbar_expect_tx(bar_kv + st, uint32_t(valid) * kLtPageBytes);
            if (id[i] >= 0) {
              tma_load_4d(sm + S::kv + st * kLtTileBytes + i * kLtPageBytes, &tm_kv, 0, 0, 0, 2 * id[i], bar_kv + st);
              ++sent;
            }
          }
          // a tile given up half way: let its phase end with what was sent
          if (!ok && sent > 0)
            asm volatile("mbarrier.complete_tx.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(smem_u32(bar_kv + st)),
                         "r"(uint32_t(valid - sent) * kLtPageBytes)
                         : "memory");
          if (sent > 0) {  // (a tile's first page is always loaded)
            mbar_arrive(bar_kv + st);
            landing = g + 1;
          }
        }
        ok = __shfl_sync(0xffffffffu, int(ok), 0) != 0;
        if (!ok) break;
        // the next tile's pages into L2, a lane a page (the second tile's own
        // copies follow at once)
        const int id_next = __shfl_sync(0xffffffffu, in_group < 7 ? ids : next,
                                        ((in_group + 1) & 7) * kLtPages + (lane & (kLtPages - 1)));
        if (g > 0 && lane < kLtPages && id_next >= 0)
          prefetch_l2(p.cache + size_t(id_next) * (kPage * kLatentRow), kLtPageBytes);
      }
    }
    if (lane == 0) {
      // copies land before the CTA's shared memory is released
      const uint64_t limit = ok ? kLandLimitNs : kDrainLimitNs;
      for (int i = landing > kLtStages ? landing - kLtStages : 0; i < landing; ++i)
        mbar_wait(bar_kv + i % kLtStages, (i / kLtStages) & 1, limit);
      if (pieces > 0) mbar_wait(bar_q, (pieces - 1) & 1, limit);
      if (!ok) flag_status(p.status, PKV_STATUS_TIMEOUT);
      // Where nothing is joined a share is one whole tile at most, and with its
      // copies landed this CTA has read all that it reads: a kernel let in now
      // waits for what is left (four short sequences behind one another 10.7 us
      // a call without this, 8.7 with it).
      if (ok && pieces > 0 && !p.joins) griddep_launch_dependents();
    }
    __syncwarp();
  } else if (warp == 9) {
    // ===== scores: S^T of tile after tile, each once it has landed and the
    // softmax has taken the scores two tiles before from its buffer =====
    constexpr uint32_t idesc = idesc_bf16(64, N, false);
    const uint32_t aq = smem_u32(sm + S::q);
    LtWalk walk = first;
    LtPiece x;
    int g = 0, pieces = 0;
    bool ok = true;
    while (ok && lt_next<N, kLtKeys>(p, walk, x)) {
      ok = wait_all(bar_q, pieces & 1);
      for (int k = x.k0; ok && k < x.k1; ++k, ++g) {
        if (g >= 2) ok = wait_all(bar_p + (g & 1), ((g >> 1) - 1) & 1);
        if (ok) ok = wait_all(bar_kv + g % kLtStages, (g / kLtStages) & 1);
        if (!ok) break;
        const uint32_t kv = smem_u32(sm + S::kv) + uint32_t(g % kLtStages) * kLtTileBytes;
        tc_fence_after();
#pragma unroll 3
        for (int c = 0; c < kLtChunks; ++c)
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            umma(tmem_s(g), smem_desc(kv + c * 1024 + kk * 32, 16, kLtGroupBytes),
                 smem_desc(aq + c * (N * 128) + kk * 32, 16, 1024), idesc, c + kk > 0);
        umma_commit(bar_s + (g & 1));
        if (k + 1 == x.k1) umma_commit(bar_qfree);
      }
      ++pieces;
    }
    if (!ok && lane == 0) flag_status(p.status, PKV_STATUS_TIMEOUT);
    // what was issued lands before TMEM is released
    if (g > 0) mbar_wait(bar_s + ((g - 1) & 1), ((g - 1) >> 1) & 1, kLandLimitNs);
    __syncwarp();
  } else if (warp == 10) {
    // ===== values: O^T += V^T P^T of tile after tile, once its P is written.
    // A warp of its own: behind the scores of the next tile, in one warp, P V
    // waited for that tile's copies, and they for the buffer that P V frees
    // (5000 cycles a tile against 3100). =====
    constexpr uint32_t idesc = idesc_bf16(128, N, true, true);
    LtWalk walk = first;
    LtPiece x;
    int g = 0;
    bool ok = true;
    while (ok && lt_next<N, kLtKeys>(p, walk, x)) {
      for (int k = x.k0; k < x.k1; ++k, ++g) {
        if (!(ok = wait_all(bar_p + (g & 1), (g >> 1) & 1))) break;
        const uint32_t kv = smem_u32(sm + S::kv) + uint32_t(g % kLtStages) * kLtTileBytes;
        tc_fence_after();
#pragma unroll
        for (int ks = 0; ks < kLtPages; ++ks) {
#pragma unroll
          for (int d = 0; d < 4; ++d)
            umma(tmem + uint32_t(d) * N, smem_desc(kv + ks * kLtPageBytes + d * 2048, 1024, kLtGroupBytes),
                 smem_desc(kv + ks * kLtPageBytes + kLtChunkP, 1024, kLtGroupBytes), idesc,
                 (k > x.k0 || ks > 0) ? 1u : 0u);
          umma_commit(bar_kvfree + (g % kLtStages) * kLtPages + ks);
        }
      }
    }
    if (!ok && lane == 0) flag_status(p.status, PKV_STATUS_TIMEOUT);
    if (g > 0)
      mbar_wait(bar_kvfree + ((g - 1) % kLtStages) * kLtPages + kLtPages - 1, ((g - 1) / kLtStages) & 1, kLandLimitNs);
    __syncwarp();
  } else {
    // ===== softmax and results: warpgroup w has rows [w * NW, (w + 1) * NW) =====
    const int wg = warp >> 2, quad = warp & 3, half = lane >> 4;
    const int key = quad * 16 + (lane & 15);      // this thread's key of a tile
    const int col0 = wg * NW + half * NC;         // its first row
    const uint32_t lane_off = uint32_t(quad * 32) << 16;
    float* s_red = reinterpret_cast<float*>(sm + S::red);      // [4][N]
    float* s_alpha = reinterpret_cast<float*>(sm + S::alpha);  // [N]
    const int bar_id = 1 + wg;
    griddep_wait();  // an earlier call may still read the workspace and write to out
    // (here, in the time that the first copies take)
    if (tid == 0 && p.joins) p.joins[blockIdx.x] = lt_join<N>(p, *plan, int(blockIdx.x), int(gridDim.x));
    LtWalk walk = first;
    LtPiece x;
    int g = 0;
    // A warp whose wait ran out waits no more, but goes through the rest of
    // its share all the same (writing no result), so that the warpgroup's
    // barriers keep all their threads.
    bool ok = true;
    auto wait = [&](uint64_t* bar, uint32_t parity) {
      if (ok) ok = __all_sync(0xffffffffu, mbar_wait(bar, parity));
    };
    // O^T up to date with tile t, the last one whose P this warp gave away:
    // P V's last page is let go of.  (A wait names a phase by its parity, so it
    // must not be able to be a whole phase late: the next phase of that barrier
    // is tile t + 2's, whose P this warp has yet to write.  For the same reason
    // even and odd tiles have a barrier each for P and for the scores.)
    auto wait_o = [&](int t) {
      wait(bar_kvfree + (t % kLtStages) * kLtPages + kLtPages - 1, (t / kLtStages) & 1);
    };
    while (lt_next<N, kLtKeys>(p, walk, x)) {
      float m[NC];       // reference of each row
      uint64_t l2[NC / 2];  // row sums of this thread's keys, two rows a word
      int lim[NC];  // last key that the row sees
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        m[c] = 0.f;
        l2[c / 2] = 0;
        lim[c] = x.L - x.n + min(x.n - 1, lt_token(p, x.local_row + col0 + c));
      }
      const int first_lim = x.L - x.n + lt_token(p, x.local_row);  // the tile's first row's
      for (int k = x.k0; k < x.k1; ++k, ++g) {
        wait(bar_s + (g & 1), (g >> 1) & 1);
        tc_fence_after();
        float s[NC];
        lt_load_scores<N>(tmem_s(g) + uint32_t(wg * NW) + lane_off, s);
        tmem_wait_ld();
        const int pos = k * kLtKeys + key;
        const bool masked = k * kLtKeys + kLtKeys - 1 > first_lim;
        // x = scaled score - reference, two rows an instruction
        float xs[NC];
        auto relative = [&]() {
          const uint64_t q2 = f2(p.qscale, p.qscale);
#pragma unroll
          for (int c = 0; c < NC; c += 2)
            f2_split(f2_fma(f2(s[c], s[c + 1]), q2, f2(-m[c], -m[c + 1])), xs[c], xs[c + 1]);
          if (masked) {
#pragma unroll
            for (int c = 0; c < NC; ++c)
              if (pos > lim[c]) xs[c] = -INFINITY;
          }
        };
        relative();
        if (k == x.k0) {
          // A piece's first reference is its first key's score.  Rows that do
          // not see that key see nothing of this piece (what a row sees is a
          // prefix) and keep 0.  (Through s_red, whose readers of the piece
          // before are behind a barrier: of s_alpha a slower warp may still
          // read that piece's 1 / row sums.)  Rows behind the tile's last, the
          // next sequence's or what a padded batch holds, take infinity, so
          // that no score of theirs ever moves the tile's references.
          if (key == 0) {
#pragma unroll
            for (int c = 0; c < NC; ++c)
              s_red[col0 + c] = col0 + c >= x.rows ? INFINITY : xs[c] == -INFINITY ? 0.f : xs[c];
          }
          named_sync(bar_id, 128);
#pragma unroll
          for (int c = 0; c < NC; ++c) m[c] = s_red[col0 + c];
          relative();
        }
        float top = xs[0];
#pragma unroll
        for (int c = 0; c < NC; c += 2) top = max3(top, xs[c], xs[c + 1]);
        if (named_sync_or(bar_id, 128, top > kLtTau)) {
          // New references: the maximum over the tile's 64 keys where that is
          // above the old one.
#pragma unroll
          for (int c = 0; c < NC; ++c) {
            float v = xs[c];
#pragma unroll
            for (int o = 8; o >= 1; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
            if ((lane & 15) == 0) s_red[quad * N + col0 + c] = v;
          }
          named_sync(bar_id, 128);
#pragma unroll
          for (int c = 0; c < NC; c += 2) {
            float a[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              float v = s_red[col0 + c + e];
#pragma unroll
              for (int q = 1; q < 4; ++q) v = fmaxf(v, s_red[q * N + col0 + c + e]);
              a[e] = 1.f;
              if (v > 0.f) {
                const float up = m[c + e] + v;
                a[e] = ex2(m[c + e] - up);
                m[c + e] = up;
              }
              if (quad == 0 && (lane & 15) == 0) s_alpha[col0 + c + e] = a[e];
            }
            l2[c / 2] = f2_fma(l2[c / 2], f2(a[0], a[1]), 0);
          }
          relative();
          if (k > x.k0) {
            // O^T of the earlier tiles under the new references
            named_sync(bar_id, 128);
            wait_o(g - 1);
            tc_fence_after();
#pragma unroll 1
            for (int d = 0; d < 4; ++d)
#pragma unroll 1
              for (int c = 0; c < NW; c += 8) {
                const uint32_t ta = tmem + uint32_t(d * N + wg * NW + c) + lane_off;
                float o[8];
                tmem_ld8(ta, o);
                tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 8; ++e) o[e] *= s_alpha[wg * NW + c + e];
                tmem_st8(ta, o);
              }
            tmem_wait_st();
          }
        }
        uint32_t pk[NC / 2];
#pragma unroll
        for (int c = 0; c < NC; c += 2) {
          pk[c / 2] = pack_bf16x2(ex2(xs[c]), ex2(xs[c + 1]));
          l2[c / 2] = f2_add(l2[c / 2], f2(bf_lo(pk[c / 2]), bf_hi(pk[c / 2])));
        }
        if (!ok) continue;
        uint8_t* kv = sm + S::kv + (g % kLtStages) * kLtTileBytes;
        uint8_t* prow = kv + (key >> 3) * kLtGroupBytes + kLtChunkP + (key & 7) * 128;
#pragma unroll
        for (int c = 0; c < NC; c += 4) {
          const uint32_t byte = uint32_t(col0 + c) * 2;
          *reinterpret_cast<uint2*>(prow + (((byte >> 4) ^ (key & 7)) << 4) + (byte & 8)) =
              make_uint2(pk[c / 2], pk[c / 2 + 1]);
        }
        const int valid = x.L - k * kLtKeys;
        if (valid < kLtKeys) {
          // rows past the sequence hold whatever the pages or the buffer
          // held: zero their values, since 0 x NaN is NaN (their scores are
          // masked).  The scores' MMAs are done, this tile's P V not issued.
          for (int i = tid; i < (kLtKeys - valid) * 64; i += kLtSoftmaxThreads) {
            const int r = valid + (i >> 6), ch = (i >> 3) & 7, v = i & 7;
            *reinterpret_cast<uint4*>(kv + (r >> 3) * kLtGroupBytes + ch * 1024 + (r & 7) * 128 + v * 16) =
                make_uint4(0, 0, 0, 0);
          }
        }
        fence_proxy_async_smem();
        tc_fence_before();
        mbar_arrive(bar_p + (g & 1));
      }

      // ---- the piece's result ----
      const bool whole = x.k0 == 0 && x.k1 == x.blocks;
      float l[NC];
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        if (c % 2 == 0) f2_split(l2[c / 2], l[c], l[c + 1]);
#pragma unroll
        for (int o = 8; o >= 1; o >>= 1) l[c] += __shfl_xor_sync(0xffffffffu, l[c], o);
      }
      named_sync(bar_id, 128);  // s_red's last readers are done
#pragma unroll
      for (int c = 0; c < NC; ++c)
        if ((lane & 15) == 0) s_red[quad * N + col0 + c] = l[c];
      float* part = p.partials + (size_t(blockIdx.x) * 2 + (x.k0 == 0 ? 1 : 0)) * kLtPartialFloats;
      if (!whole && quad == 0 && (lane & 15) == 0) {
#pragma unroll
        for (int c = 0; c < NC; ++c) part[N * kLatentDim + col0 + c] = m[c];
      }
      named_sync(bar_id, 128);
      if (quad == 0 && lane < NW) {
        const int r = wg * NW + lane;
        const float sum = (s_red[r] + s_red[N + r]) + (s_red[2 * N + r] + s_red[3 * N + r]);
        if (whole)
          s_alpha[r] = 1.f / sum;
        else
          part[N * kLatentDim + N + r] = sum;
      }
      named_sync(bar_id, 128);
      wait_o(g - 1);
      if (ok) {
        tc_fence_after();
        const int r0 = wg * NW;  // this warpgroup's rows of the tile
        float inv[NW];
        if (whole) {
#pragma unroll
          for (int c = 0; c < NW; c += 4)
            *reinterpret_cast<float4*>(inv + c) = *reinterpret_cast<const float4*>(s_alpha + r0 + c);
        }
#pragma unroll 1
        for (int d = 0; d < 4; ++d) {
          float o[NW];  // lane: dim d * 128 + quad * 32 + lane; column: row
          tmem_ld_cols<NW>(tmem + uint32_t(d * N + r0) + lane_off, o);
          tmem_wait_ld();
          const int dim = d * 128 + quad * 32;
          if (whole) {
            // two rows at a time: even lanes take the first row's pair of
            // dims, odd lanes the second's, so a lane stores two values
            uint32_t* to = reinterpret_cast<uint32_t*>(p.out + size_t(x.row0 + r0 + (lane & 1)) * kLatentDim + dim) +
                           (lane >> 1);
#pragma unroll
            for (int c = 0; c < NW; c += 2) {
              const float a = o[c] * inv[c], b = o[c + 1] * inv[c + 1];
              const float other = __shfl_xor_sync(0xffffffffu, (lane & 1) ? a : b, 1);
              if (r0 + c + (lane & 1) < x.rows)
                to[c * (kLatentDim / 2)] = (lane & 1) ? pack_bf16x2(other, b) : pack_bf16x2(a, other);
            }
          } else {
            float4* to = reinterpret_cast<float4*>(part) + ((d * 4 + quad) * (N / 4) + r0 / 4) * 32 + lane;
#pragma unroll
            for (int c = 0; c < NW; c += 4)
              if (r0 + c < x.rows) to[c * 8] = make_float4(o[c], o[c + 1], o[c + 2], o[c + 3]);
          }
        }
        tc_fence_before();  // read before the next piece's first P V overwrites it
      }
    }
    if (!ok) flag_status(p.status, PKV_STATUS_TIMEOUT);
    // A share that begins and ends at the same block inside a tile is a piece
    // without keys, which the merge skips by its l of 0.
    if (begin.k > 0 && begin.b == end.b && begin.j == end.j && begin.k == end.k && tid < N)
      p.partials[size_t(blockIdx.x) * 2 * kLtPartialFloats + N * kLatentDim + N + tid] = 0.f;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  griddep_launch_dependents();  // behind the barrier: one thread of a CTA speaks for all
  if (warp == 9)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512u));
}

template <int N>
int launch_latent(const LaunchCtx& ctx, const LatentAttendArgs& a, LatentParams lp) {
  static std::mutex mu;
  static bool ready[64] = {};
  const int device = ctx.dev->device;
  {
    std::lock_guard<std::mutex> lk(mu);
    if (!ready[device]) {
      if (cudaFuncSetAttribute(pkv_latent_kernel<N>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                               int(LtSmem<N>::bytes)) != cudaSuccess) {
        cudaGetLastError();
        return PKV_ERR_LAUNCH;
      }
      ready[device] = true;
    }
  }
  const pkv_desc& d = a.desc;
  CUtensorMap tq, tkv;
  {
    const cuuint64_t dims[3] = {64, cuuint64_t(a.num_tokens) * d.num_q_heads, kLtChunks};
    const cuuint64_t strides[2] = {kLatentRow * 2, 128};
    const cuuint32_t box[3] = {64, N, kLtChunks};
    if (!encode_tensor_map(&tq, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, a.q, 3, dims, strides, box)) return PKV_ERR_LAUNCH;
  }
  {
    const cuuint64_t dims[4] = {64, 8, kLtChunks, cuuint64_t(d.num_blocks) * 2};
    const cuuint64_t strides[3] = {kLatentRow * 2, 128, kLatentRow * 16};
    const cuuint32_t box[4] = {64, 8, kLtChunks, 2};
    if (!encode_tensor_map(&tkv, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, a.cache, 4, dims, strides, box))
      return PKV_ERR_LAUNCH;
  }
  // Where the plan cuts no tile there is nothing to join: few tiles (so that
  // each has CTAs of its own, lt_plan) of sequences no longer than two least
  // pieces (four sequences of up to 255 tokens: 11.6 -> 10.4 us).
  const int64_t tiles = int64_t(a.num_tokens) * d.num_q_heads / N + a.num_seqs;
  const bool cut = int64_t(d.max_blocks_per_seq) * kPage > 2 * kLtLeastOwn || 2 * tiles > ctx.dev->sm_count;
  if (!cut) lp.joins = nullptr;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctx.dev->sm_count);
  cfg.blockDim = dim3(kLtThreads);
  cfg.dynamicSmemBytes = LtSmem<N>::bytes;
  cfg.stream = ctx.stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  {
    TraceScope ts(ctx.stream, PKV_K_LATENT);
    cudaLaunchKernelEx(&cfg, pkv_latent_kernel<N>, tq, tkv, lp);
    if (int e = ts.done()) return e;
  }
  if (!cut) return PKV_OK;
  cfg.gridDim = dim3(ctx.dev->sm_count, lt_merge_blocks(N));
  cfg.blockDim = dim3(kLtMergeThreads);
  cfg.dynamicSmemBytes = 0;
  TraceScope ts(ctx.stream, PKV_K_MERGE);
  cudaLaunchKernelEx(&cfg, pkv_latent_merge_kernel<N, false>, lp);
  return ts.done();
}

}  // namespace

// Two partials and one join record a CTA, whatever the batch.
size_t latent_workspace_bytes(const DeviceInfo& dev) {
  return align_up(size_t(dev.sm_count) * 2 * kLtPartialFloats * sizeof(float), 256) +
         align_up(size_t(dev.sm_count) * sizeof(int4), 256);
}

int launch_attend_latent(const LaunchCtx& ctx, const LatentAttendArgs& a) {
  const pkv_desc& d = a.desc;
  if (ctx.dev->sm_count > kLtMergeThreads) return PKV_ERR_LAUNCH;  // the merge holds a piece a thread
  if (a.workspace_bytes < latent_workspace_bytes(*ctx.dev)) return PKV_ERR_WORKSPACE;
  LatentParams lp{};
  lp.block_tables = a.block_tables;
  lp.seq_lens = a.seq_lens;
  lp.qsl = a.query_start_loc;
  lp.out = a.out;
  lp.cache = a.cache;
  uint8_t* ws = static_cast<uint8_t*>(a.workspace);
  lp.partials = reinterpret_cast<float*>(ws);
  lp.joins = reinterpret_cast<int4*>(
      ws + align_up(size_t(ctx.dev->sm_count) * 2 * kLtPartialFloats * sizeof(float), 256));
  lp.status = ctx.status;
  lp.B = a.num_seqs;
  lp.T = a.num_tokens;
  lp.H = d.num_q_heads;
  lp.inv_heads = uint32_t(std::min<uint64_t>((uint64_t(1) << 32) / d.num_q_heads, 0xFFFFFFFFu));
  lp.max_blocks = d.max_blocks_per_seq;
  lp.num_blocks = d.num_blocks;
  lp.qscale = a.scale * 1.4426950408889634f;
  const int64_t most = a.max_query_len > 0 && a.max_query_len < a.num_tokens ? a.max_query_len : a.num_tokens;
  const int64_t rows = most * d.num_q_heads;
  // More than 64 rows a sequence go to pairs of CTAs, which take longer to start
  // and to end a tile but half as long a key: 64 sequences of 128 heads and
  // 512-4096 tokens 61 us against 77, of 512-1023 tokens 38 against 43; two
  // 1023-token chunks over 1536-3584 tokens, 64 heads, 553 against 944; a
  // 512-token chunk over 1500 tokens, 128 heads, 195 against 309.  Not where
  // tiles are short: four sequences of up to 255 tokens 17 against 10, prompts
  // of 400-1500 tokens, whose tiles see half of them, 84-567 against 76-528
  // (2200 tokens: 1021 and 994; 4096 of 16 heads: 342 and 380).  How long
  // sequences are is known here only as the tables' width, and context only as
  // what that leaves beside the longest query.
  const int64_t width = int64_t(d.max_blocks_per_seq) * kPage;
  if (rows > 64 && (width >= kLtPairTokens || (width >= kLtPairTokens / 4 && most <= width / 2)))
    return launch_latent_pair(ctx, a, lp);
  // Rows a tile: the least multiple of 16 that cuts the longest sequence's
  // rows into as few tiles as 64 would.
  const int64_t tiles = (rows + 63) / 64;
  const int64_t per = (rows + tiles - 1) / tiles;
  if (per <= 16) return launch_latent<16>(ctx, a, lp);
  if (per <= 32) return launch_latent<32>(ctx, a, lp);
  if (per <= 48) return launch_latent<48>(ctx, a, lp);
  return launch_latent<64>(ctx, a, lp);
}

}  // namespace pkv
