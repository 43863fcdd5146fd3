// pkv_latent_pair.cu -- attention over latent pages for sequences of more than
// 64 rows (query tokens x heads): tiles of 128 rows on pairs of CTAs.
//
// The one-CTA kernel (pkv_latent.cu) holds O of 64 rows, 512 dims each, in
// TMEM, and both its products are bound by shared memory, whose every operand
// byte feeds 64 rows only: 2500 cycles a 64-key tile of 64 rows.  A pair of
// CTAs with tcgen05's cta_group::2 holds 128 rows, split by dims, and each
// product reads half of its B operand from each CTA:
//   S [128 rows x 128 keys] = Q K^T      M = 128: CTA i has rows 64 i .. and
//                                        keys 64 i .. of the tile, 576 dims
//   O^T [512 dims x 128 rows] += V^T P^T M = 256, twice: CTA i has dims
//                                        256 i .. of all 128 keys, and P of
//                                        its own rows
// so that softmax and P stay within the CTA that has the rows.  A tile costs
// 36 x 32 + 16 x 64 = 2176 cycles of tensor time and about 3000 of shared
// memory (copies in 1090, operands 1920) for 128 keys x 128 rows, which two
// single CTAs have in 5000.
//
//  * K (64 own keys x 576 dims) and V (128 keys x 256 own dims) are copies of
//    their own: the products need their operands at the same place in both
//    CTAs, which a shared copy of the own keys' own dims could not be.  72 +
//    64 KiB, with 72 KiB of queries and 16 KiB of P all that an SM has, so
//    each has one buffer, loaded and let go of in slices (K by three chunks of
//    64 dims, V by 32 keys).
//  * The leader (rank 0) issues all MMAs.  Copies of K and V report to its
//    barriers from both CTAs (a warp that forwards them costs 400 cycles, in
//    the loops of load and use that set the pace), but for a sequence's last
//    tile, whose rows past the end of V the CTA itself has to zero.  Commits go
//    to both CTAs.
//  * In S a row is a lane, so the row's reference is one register.  A score
//    may exceed the reference (the first key's score) by 2^64 without harm to
//    bf16 or fp32; there is no test a tile, only a flag when one does.  Then
//    the pair does its whole share again, each piece with a pass for its
//    maxima first.  (Rescaling O^T would need both CTAs at every such tile.)
//  * Work split, partials and merge are pkv_latent.cu's, with a pair in the
//    place of a CTA.
//
// Measured: two 1023-token chunks over 1536-3584 tokens and 33 decode rows, 64
// heads: 555-565 us, 0.75 of the bf16 burst peak (one CTA a tile: 944).  A tile
// takes 3200 cycles there: with one buffer each, a slice's way from being let
// go of to being here again (2300 cycles, 400 of them for the word to the other
// CTA) and its product follow one another, and neither product has work while
// both wait.  64 decode rows of 128 heads over 512-4096 tokens: 62 us; a share is
// 16 tiles there, and the 13000 cycles from the last P V of one piece to the
// first of the next (result out, 72 KiB of queries and the first K and V in)
// cost as much as four of them.  Of a whole tile's 11000 the result takes 6000,
// through shared memory so that rows leave in one piece; 16 rows at a time with
// half as many barriers a row, by plain or by TMA stores, it was slower (a
// 2200-token prompt of 128 heads 1021 us, 1074 and 1084).
#include <algorithm>
#include <mutex>

#include "pkv_internal.h"
#include "pkv_latent.cuh"
#include "pkv_latent_merge.cuh"

namespace pkv {
namespace {

constexpr int kPrRows = 128;                // rows a tile
constexpr int kPrKeys = 128;                // keys a cache tile
constexpr int kPrOwn = 64;                  // rows, and keys, of one CTA
constexpr int kPrSoftmaxThreads = 256;
constexpr int kPrThreads = kPrSoftmaxThreads + 128;  // + K loader, score, value and V loader warps
constexpr int kPrSlicesK = 3, kPrSlicesV = 4;
constexpr uint32_t kPrSliceK = 4 * 2 * 3 * 1024;  // [4 pages][2 groups][3 chunks][8 rows][128 B]
constexpr uint32_t kPrGroupK = 3 * 1024;
constexpr uint32_t kPrPageV = 2 * 4 * 1024;       // [2 groups][4 chunks][8 rows][128 B]
constexpr uint32_t kPrGroupV = 4 * 1024;
constexpr uint32_t kPrSliceV = 2 * kPrPageV;
constexpr float kPrTau = 64.0f;  // log2 of how far a score may exceed the reference

// Shared memory (offsets from a 1024-byte aligned base), the same in both CTAs.
struct PrSmem {
  static constexpr uint32_t k = 0;
  static constexpr uint32_t v = k + kPrSlicesK * kPrSliceK;
  static constexpr uint32_t q = v + kPrSlicesV * kPrSliceV;  // [9][64 rows][128 B]
  static constexpr uint32_t p = q + kLtChunks * kPrOwn * 128;  // [2 halves][64 rows][64 keys]
  static constexpr uint32_t bars = p + 2 * kPrOwn * 128;       // 33 x 8
  static constexpr uint32_t tmem = bars + 272;
  static constexpr uint32_t flags = tmem + 8;                  // own, the other CTA's
  static constexpr uint32_t plan = tmem + 16;                  // LtPlan
  static constexpr uint32_t inv = plan + 128;                  // [2 whole tiles][64] 1 / row sums of the other CTA's rows
  static constexpr uint32_t red = inv + 512;                   // [4][64] partial sums, maxima; own rows' 1 / row sums
  static constexpr uint32_t wsum = red;                        // plan scans
  static constexpr uint32_t end = red + 1024;
  static constexpr uint32_t bytes = end + 1024;                // + alignment slack
};
static_assert(PrSmem::bytes <= 232448, "paired latent attention: shared memory above the 227 KiB limit");
static_assert(2 * (kPrThreads / 32) * 16 <= 1024, "what the plan borrows");

// ---- two-CTA forms of the tcgen05 and barrier helpers ---------------------------
__device__ __forceinline__ void umma_pair(uint32_t tmem_d, uint64_t a, uint64_t b, uint32_t idesc,
                                          uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\t.reg .b32 l;\n\t"
      "elect.sync l|e, 0xffffffff;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "@e tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(tmem_d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate));
}
// Arrives on the barrier at this place in both CTAs.
__device__ __forceinline__ void umma_pair_commit(uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .pred e;\n\t.reg .b32 l;\n\t"
      "elect.sync l|e, 0xffffffff;\n\t"
      "@e tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;\n\t}" ::"r"(
          smem_u32(bar)),
      "h"(uint16_t(3))
      : "memory");
}
__device__ __forceinline__ uint32_t cluster_addr(const void* p, uint32_t rank) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
  return a;
}
// Arrival on a barrier of either CTA.  What these arrivals tell of is this
// CTA's own shared memory and TMEM, which only the tensor cores read behind
// them and which fence.proxy.async and the tcgen05 fences have ordered; no
// thread of the other CTA reads it.  With .release.cluster, a fence over the
// thread's global stores too, a tile took 6600 cycles against 4100.
__device__ __forceinline__ void arrive_at(uint32_t cluster_bar) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(cluster_bar) : "memory");
}
// The same where the other CTA's threads read what was stored before it, and
// their wait.
__device__ __forceinline__ void arrive_publish(uint32_t cluster_bar) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_bar) : "memory");
}
__device__ __forceinline__ bool try_wait_published(uint64_t* bar, uint32_t parity) {
  uint32_t done;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(done)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return done != 0;
}
__device__ __forceinline__ bool wait_published(uint64_t* bar, uint32_t parity) {
  if (try_wait_published(bar, parity)) return true;
  const uint64_t t0 = global_ns();
  while (!try_wait_published(bar, parity))
    if (global_ns() - t0 > kWaitLimitNs) return false;
  return true;
}
// Both CTAs are here.  (No fence: barriers' initial values have one of their
// own, and nothing else is handed over this way.)
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.relaxed;\n\tbarrier.cluster.wait;" ::: "memory");
}

// A copy into this CTA's shared memory that reports to a barrier of either CTA
// of the pair (its cluster address), and the announcement of its bytes there.
__device__ __forceinline__ void tma_load_4d_pair(void* dst, const CUtensorMap* map, int c0, int c1, int c2, int c3,
                                                 uint32_t cluster_bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes.cta_group::2 [%0], [%1, "
      "{%2, %3, %4, %5}], [%6];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(cluster_bar)
      : "memory");
}
__device__ __forceinline__ void arrive_expect_at(uint32_t cluster_bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cluster.b64 _, [%0], %1;" ::"r"(cluster_bar), "r"(bytes) : "memory");
}
__device__ __forceinline__ void tmem_ld32f(uint32_t taddr, float (&r)[32]) {
  uint32_t u[32];
  tmem_ld32(taddr, u);
  tmem_wait_ld();
#pragma unroll
  for (int i = 0; i < 32; ++i) r[i] = __uint_as_float(u[i]);
}

__global__ void __launch_bounds__(kPrThreads, 1)
    pkv_latent_pair_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                           const __grid_constant__ CUtensorMap tm_v, const LatentParams p) {
  using S = PrSmem;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(sm + S::bars);
  uint64_t* bar_q = bars;                          // own queries landed
  uint64_t* bar_qfree = bars + 1;                  // the piece's scores are done
  uint64_t* bar_k = bars + 2;                      // [3] leader: slice of K landed in both CTAs
  uint64_t* bar_kfree = bars + 5;                  // [3] the scores that read it are done
  uint64_t* bar_v = bars + 8;                      // [4] leader: slice of V landed in both CTAs
  uint64_t* bar_vfree = bars + 12;                 // [4] the P V that reads it is done
  uint64_t* bar_s = bars + 16;                     // [2] scores written
  uint64_t* bar_p = bars + 18;                     // [2 tiles][2 halves] leader: P of 64 keys written (8 warps)
  uint64_t* bar_x = bars + 22;                     // [2][2] leader: scores taken, in a pass for maxima
  uint64_t* bar_inv = bars + 26;                   // row sums of both CTAs here (16 warps)
  uint64_t* bar_q2 = bars + 27;                    // leader: the other CTA's queries landed
  uint64_t* bar_tail = bars + 28;                  // [4] own slice of V landed, of a sequence's last tile
  uint64_t* bar_round = bars + 32;                 // the other CTA's flags are here
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(sm + S::tmem);
  volatile int* s_flags = reinterpret_cast<volatile int*>(sm + S::flags);
  LtPlan* plan = reinterpret_cast<LtPlan*>(sm + S::plan);
  float* s_inv = reinterpret_cast<float*>(sm + S::inv);
  float* s_red = reinterpret_cast<float*>(sm + S::red);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = int(blockIdx.x & 1), pair = int(blockIdx.x >> 1), pairs = int(gridDim.x >> 1);
  enum { kOverflow = 1, kTimeout = 2 };  // of s_flags

  if (tid == 0) {
    for (int i = 0; i < 33; ++i) {
      uint64_t* b = bars + i;
      const bool both = (b >= bar_k && b < bar_k + kPrSlicesK) || (b >= bar_v && b < bar_v + kPrSlicesV);
      mbar_init(b, both ? 2 : b == bar_inv ? 16 : b >= bar_p && b < bar_inv ? 8 : 1);
    }

    fence_mbar_init();
    s_flags[0] = s_flags[1] = 0;
  }
  if (warp == 9) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(s_tmem)),
                 "r"(512u));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
  }
  if (warp == 10) {
    // The block tables into L2, shared among the CTAs.  (A hint: what the
    // stream does before may still write them.)
    const char* tables = reinterpret_cast<const char*>(p.block_tables);
    const int64_t bytes = int64_t(p.B) * p.max_blocks * 4;
    for (int64_t i = (int64_t(blockIdx.x) * 32 + lane) * 128; i < bytes; i += int64_t(gridDim.x) * 32 * 128)
      asm volatile("prefetch.global.L2 [%0];" ::"l"(tables + i));
  }
  // The lengths, query starts and tables are not what the call right before
  // this one writes, so the plan need not wait for it.
  lt_plan<kPrRows, kPrKeys, kPrThreads>(p, pair, pairs, reinterpret_cast<longlong2*>(sm + S::wsum), plan);
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // both CTAs' barriers are initialised, their plans read
  tc_fence_after();
  const uint32_t tmem = *s_tmem;
  const LtPos begin = plan->begin, end = plan->end;
  const LtWalk first{begin, end, lt_seq<kPrRows>(p, begin.b, plan->q0, plan->q1, plan->L)};
  auto next_piece = [&](LtWalk& w, LtPiece& x) { return lt_next<kPrRows, kPrKeys>(p, w, x); };
  const uint32_t tmem_s[2] = {tmem + 256u, tmem + 320u};  // O^T: [0, 128) and [128, 256)
  auto wait_all = [&](uint64_t* bar, uint32_t parity) {
    return __all_sync(0xffffffffu, mbar_wait(bar, parity));
  };
  // Page ids of a piece, 32 at a time, a group ahead.  -1 past the sequence (no
  // copy); an id that is no page of the pool is flagged and page 0 is read in
  // its place.
  auto page_id = [&](const LtPiece& x, int i) {
    if (i >= x.k1 * (kPrKeys / kPage) || i >= (x.L + kPage - 1) / kPage) return -1;
    int id = __ldg(p.block_tables + int64_t(x.b) * p.max_blocks + i);
    if (id < 0 || id >= p.num_blocks) {
      flag_status(p.status, PKV_STATUS_BAD_BLOCK);
      id = 0;
    }
    return id;
  };

  // What each role carries from the first round to a second.  g counts cache
  // tiles, gv those with a P V.  A second round (some score exceeded the
  // reference by too much) walks every piece twice, for maxima first.
  griddep_launch_dependents();  // the merge kernel, which waits for this grid
  if (warp < kPrSoftmaxThreads / 32) griddep_wait();  // an earlier call may still read the workspace and write to out
  if (tid == 0 && rank == 0) p.joins[pair] = lt_join<kPrRows>(p, *plan, pair, pairs);
  int g = 0, gv = 0, pieces = 0, wholes = 0;
  int slices = 0, tails = 0;  // that a loader has sent; slices of last tiles
  int g0 = 0, taken[2] = {-1, -1};  // tiles of passes for maxima; of the tile in each score buffer, count and kind
  bool ok = true;
  for (int round = 0; round < 2; ++round) {
    LtWalk walk = first;
    LtPiece x;
    if (warp == 8) {
      // ===== queries and K =====
      const uint32_t lead_k = cluster_addr(bar_k, 0);
      while (ok && next_piece(walk, x)) {
        for (int pass = round == 0; ok && pass < 2; ++pass) {
          // (before the wait below: the reads take longer than what is left of
          // the piece before)
          int ids = page_id(x, x.k0 * 8 + lane), next = page_id(x, x.k0 * 8 + 32 + lane);
          if (pieces == 0) {
            // the first tile's pages into L2 (a hint), then what the stream did
            // before: the queries, this step's rows
            if (lane >> 2 == rank && ids >= 0)
              prefetch_l2(p.cache + size_t(ids) * (kPage * kLatentRow), kPage * kLatentRow * 2);
            griddep_wait();
          }
          if (lane == 0) {
            if (pieces > 0) ok = mbar_wait(bar_qfree, (pieces - 1) & 1);
            if (ok) {
              mbar_arrive_expect_tx(bar_q, kLtChunks * kPrOwn * 128);
              if (!(kDropFirstCopy && pieces == 0))
                tma_load_3d(sm + S::q, &tm_q, 0, x.row0 + rank * kPrOwn, 0, bar_q);
            }
          }
          ok = __shfl_sync(0xffffffffu, int(ok), 0) != 0;
          ++pieces;
          for (int k = x.k0; ok && k < x.k1; ++k, ++g) {
            const int in_group = (k - x.k0) & 3;
            if (k > x.k0 && in_group == 0) {
              ids = next;
              next = page_id(x, (k + 4) * 8 + lane);
            }
            int id[4], valid = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              id[i] = __shfl_sync(0xffffffffu, ids, in_group * 8 + rank * 4 + i);
              valid += id[i] >= 0;
            }
            if (lane == 0) {
              for (int d = 0; ok && d < kPrSlicesK; ++d) {
                if (g > 0) ok = mbar_wait(bar_kfree + d, (g - 1) & 1);
                if (!ok) break;
                ++slices;
                arrive_expect_at(lead_k + d * 8, uint32_t(valid) * (kPrSliceK / 4));
#pragma unroll
                for (int i = 0; i < 4; ++i)
                  if (id[i] >= 0)
                    tma_load_4d_pair(sm + S::k + d * kPrSliceK + i * (kPrSliceK / 4), &tm_k, 0, 0, d * 3, 2 * id[i],
                                     lead_k + d * 8);
              }
            }
            ok = __shfl_sync(0xffffffffu, int(ok), 0) != 0;
            if (!ok) break;
            // the next tile's pages into L2, a lane a page
            const int id_next = __shfl_sync(0xffffffffu, in_group < 3 ? ids : next,
                                            ((in_group + 1) & 3) * 8 + rank * 4 + (lane & 3));
            if (lane < 4 && id_next >= 0)
              prefetch_l2(p.cache + size_t(id_next) * (kPage * kLatentRow), kPage * kLatentRow * 2);
          }
        }
      }
    } else if (warp == 11) {
      // ===== V: the 128 keys' own dims =====
      const uint32_t lead_v = cluster_addr(bar_v, 0);
      while (ok && next_piece(walk, x)) {
        int ids = page_id(x, x.k0 * 8 + lane), next = page_id(x, x.k0 * 8 + 32 + lane);
        if (gv == 0) griddep_wait();
        for (int k = x.k0; ok && k < x.k1; ++k, ++gv) {
          const int in_group = (k - x.k0) & 3;
          if (k > x.k0 && in_group == 0) {
            ids = next;
            next = page_id(x, (k + 4) * 8 + lane);
          }
          // the sequence's last tile, if it ends short, goes to barriers of
          // this CTA's own: its value warp zeroes the rows behind the end first
          const bool tail = x.L - k * kPrKeys < kPrKeys;
          for (int d = 0; ok && d < kPrSlicesV; ++d) {
            const int id0 = __shfl_sync(0xffffffffu, ids, in_group * 8 + d * 2);
            const int id1 = __shfl_sync(0xffffffffu, ids, in_group * 8 + d * 2 + 1);
            if (lane == 0) {
              if (gv > 0) ok = mbar_wait(bar_vfree + d, (gv - 1) & 1);
              if (ok) {
                const uint32_t bar = tail ? smem_u32(bar_tail + d) : lead_v + d * 8;
                arrive_expect_at(tail ? cluster_addr(bar_tail + d, rank) : bar,
                                 uint32_t((id0 >= 0) + (id1 >= 0)) * kPrPageV);
                uint8_t* dst = sm + S::v + d * kPrSliceV;
                if (id0 >= 0) tma_load_4d_pair(dst, &tm_v, 0, 0, rank * 4, 2 * id0, bar);
                if (id1 >= 0) tma_load_4d_pair(dst + kPrPageV, &tm_v, 0, 0, rank * 4, 2 * id1, bar);
                if (tail)
                  ++tails;
                else
                  ++slices;
              }
            }
            ok = __shfl_sync(0xffffffffu, int(ok), 0) != 0;
          }
        }
      }
    } else if (warp == 9) {
      // ===== scores (leader); the other CTA's warp says when its queries are here =====
      constexpr uint32_t idesc = idesc_bf16(128, kPrKeys, false);
      const uint32_t aq = smem_u32(sm + S::q), ak = smem_u32(sm + S::k);
      // g0: tiles of passes for maxima.  Each kind of pass reports to barriers
      // of its own, so that the value warp, which waits in one kind only,
      // cannot miss a phase.
      while (ok && next_piece(walk, x)) {
        for (int pass = round == 0; ok && pass < 2; ++pass) {
          ok = wait_all(bar_q, pieces & 1);
          if (ok && rank == 0) ok = wait_all(bar_q2, pieces & 1);
          if (ok && rank == 1 && lane == 0) arrive_at(cluster_addr(bar_q2, 0));
          for (int k = x.k0; rank == 0 && ok && k < x.k1; ++k, ++g) {
            // the softmax has taken the scores two tiles before
            if (taken[g & 1] >= 0) {
              const int t = taken[g & 1] >> 1;
              uint64_t* bar = (taken[g & 1] & 1 ? bar_p : bar_x) + (t & 1) * 2;
              ok = wait_all(bar, (t >> 1) & 1) && wait_all(bar + 1, (t >> 1) & 1);
            }
            taken[g & 1] = pass == 1 ? gv++ * 2 + 1 : g0++ * 2;
            for (int d = 0; ok && d < kPrSlicesK; ++d) {
              if (!(ok = wait_all(bar_k + d, g & 1))) break;
              tc_fence_after();
#pragma unroll
              for (int c = 0; c < 3; ++c)
#pragma unroll
                for (int kk = 0; kk < 4; ++kk)
                  umma_pair(tmem_s[g & 1], smem_desc(aq + (d * 3 + c) * (kPrOwn * 128) + kk * 32, 16, 1024),
                            smem_desc(ak + d * kPrSliceK + c * 1024 + kk * 32, 16, kPrGroupK), idesc,
                            (d + c + kk) > 0);
              umma_pair_commit(bar_kfree + d);
            }
            if (!ok) break;
            umma_pair_commit(bar_s + (g & 1));
            if (k + 1 == x.k1) umma_pair_commit(bar_qfree);
          }
          ++pieces;
        }
      }
    } else if (warp == 10) {
      // ===== values (leader); both CTAs' warps zero what lies behind a sequence's end =====
      constexpr uint32_t idesc = idesc_bf16(256, kPrRows, false, true);
      const uint32_t av = smem_u32(sm + S::v), ap = smem_u32(sm + S::p);
      while (ok && next_piece(walk, x)) {
        for (int k = x.k0; ok && k < x.k1; ++k, ++gv) {
          const int valid = x.L - k * kPrKeys;
          if (valid < kPrKeys) {
            // rows past the sequence hold whatever the pages or the buffer
            // held: zero them, since their weight of 0 times NaN is NaN
            for (int d = 0; ok && d < kPrSlicesV; ++d, ++tails) {
              if (!(ok = wait_all(bar_tail + d, (tails / kPrSlicesV) & 1))) break;
              const int first = max(0, valid - d * 32);
              for (int r = first; r < 32; ++r)
                *reinterpret_cast<uint4*>(sm + S::v + d * kPrSliceV + (r >> 3) * kPrGroupV + (lane >> 3) * 1024 +
                                          (r & 7) * 128 + (lane & 7) * 16) = make_uint4(0, 0, 0, 0);
              if (first < 32) fence_proxy_async_smem();
              __syncwarp();
              if (lane == 0) arrive_at(cluster_addr(bar_v + d, 0));
            }
          }
          if (rank == 1) continue;
#pragma unroll 1
          for (int d = 0; ok && d < kPrSlicesV; ++d) {
            if ((d & 1) == 0) ok = wait_all(bar_p + (gv & 1) * 2 + (d >> 1), (gv >> 1) & 1);
            if (ok) ok = wait_all(bar_v + d, gv & 1);
            if (!ok) break;
            tc_fence_after();
#pragma unroll
            for (int ks = 0; ks < 2; ++ks) {
              const int i = d * 2 + ks;  // 16 keys
#pragma unroll
              for (int e = 0; e < 2; ++e)
                umma_pair(tmem + uint32_t(e) * kPrRows,
                          smem_desc(av + i * kPrPageV + e * 2048, 1024, kPrGroupV),
                          smem_desc(ap + (i >> 2) * (kPrOwn * 128) + (i & 3) * 32, 16, 1024), idesc,
                          (k > x.k0 || i > 0) ? 1u : 0u);
            }
            umma_pair_commit(bar_vfree + d);
          }
        }
      }
    } else {
      // ===== softmax and results: a thread has one row and 32 keys of a tile =====
      const int wg = warp >> 2, quad = warp & 3;
      const int row = (quad & 1) * 32 + lane;                     // of this CTA's 64
      const int key0 = (quad >> 1) * 64 + wg * 32;                // its first key of a tile
      const int part_of_row = (quad >> 1) * 2 + wg;               // 0..3
      const uint32_t lane_off = uint32_t(quad * 32) << 16;
      auto wait = [&](uint64_t* bar, uint32_t parity) {
        if (ok) ok = wait_all(bar, parity);
      };
      const int half = quad >> 1;                                 // its keys' half of a tile
      const uint32_t lead_p = cluster_addr(bar_p + half, 0), lead_x = cluster_addr(bar_x + half, 0);  // + 16: odd tiles
      bool over = false;
      while (next_piece(walk, x)) {
        const int lim = x.L - x.n + min(x.n - 1, lt_token(p, x.local_row + rank * kPrOwn + row));  // last key it sees
        const int first_lim = x.L - x.n + lt_token(p, x.local_row);
        float m = 0.f, l = 0.f;
        for (int pass = round == 0; pass < 2; ++pass) {
          float top = -INFINITY;
          for (int k = x.k0; k < x.k1; ++k, ++g) {
            wait(bar_s + (g & 1), (g >> 1) & 1);
            tc_fence_after();
            float s[32];
            tmem_ld32f(tmem_s[g & 1] + uint32_t(wg * 32) + lane_off, s);
            const bool masked = k * kPrKeys + kPrKeys - 1 > first_lim;
            const int seen = lim - (k * kPrKeys + key0);  // columns up to this one are seen
            if (pass == 1 && round == 0 && k == x.k0) {
              // The piece's first reference is its first key's score.  Rows
              // that do not see that key see nothing of this piece (what a row
              // sees is a prefix) and keep 0.
              if (part_of_row == 0) {
                m = s[0] * p.qscale;
                if (seen < 0 || m == -INFINITY) m = 0.f;
                s_red[row] = m;
              }
              named_sync(1, kPrSoftmaxThreads);
              m = s_red[row];
              named_sync(1, kPrSoftmaxThreads);  // before s_red's next use
            }
            {
              const uint64_t q2 = f2(p.qscale, p.qscale), m2 = f2(-m, -m);
#pragma unroll
              for (int c = 0; c < 32; c += 2) f2_split(f2_fma(f2(s[c], s[c + 1]), q2, m2), s[c], s[c + 1]);
            }
            if (masked) {
#pragma unroll
              for (int c = 0; c < 32; ++c)
                if (c > seen) s[c] = -INFINITY;
            }
#pragma unroll
            for (int c = 0; c < 32; c += 2) top = max3(top, s[c], s[c + 1]);
            if (pass == 1) {
              uint32_t pk[16];
              uint64_t sum = 0;
#pragma unroll
              for (int c = 0; c < 32; c += 2) {
                pk[c / 2] = pack_bf16x2(ex2(s[c]), ex2(s[c + 1]));
                sum = f2_add(sum, f2(bf_lo(pk[c / 2]), bf_hi(pk[c / 2])));
              }
              float lo, hi;
              f2_split(sum, lo, hi);
              l += lo + hi;
              // P's half of the buffer is free once the P V before is through
              // with its keys: P V of the next tile starts on the first half
              // while the second is still written
              if (gv > 0) wait(bar_vfree + half * 2 + 1, (gv - 1) & 1);
              ++gv;
              uint8_t* prow = sm + S::p + (key0 >> 6) * (kPrOwn * 128) + row * 128;
#pragma unroll
              for (int j = 0; j < 4; ++j)
                *reinterpret_cast<uint4*>(prow + (((wg * 4 + j) ^ (row & 7)) << 4)) =
                    make_uint4(pk[4 * j], pk[4 * j + 1], pk[4 * j + 2], pk[4 * j + 3]);
              fence_proxy_async_smem();
            }
            tc_fence_before();
            __syncwarp();
            if (ok && lane == 0) arrive_at(pass == 1 ? lead_p + ((gv - 1) & 1) * 16 : lead_x + (g0 & 1) * 16);
            if (pass == 0) ++g0;
          }
          if (pass == 0) {
            // the row's maximum, over its four threads
            s_red[part_of_row * kPrOwn + row] = top;
            named_sync(1, kPrSoftmaxThreads);
            m = fmaxf(fmaxf(s_red[row], s_red[kPrOwn + row]), fmaxf(s_red[2 * kPrOwn + row], s_red[3 * kPrOwn + row]));
            if (m == -INFINITY) m = 0.f;
            named_sync(1, kPrSoftmaxThreads);
          } else if (top > kPrTau && rank * kPrOwn + row < x.rows) {
            over = true;  // (rows behind the tile's last are another sequence's, or padding)
          }
        }

        // ---- the piece's result ----
        const bool whole = x.k0 == 0 && x.k1 == x.blocks;
        s_red[part_of_row * kPrOwn + row] = l;
        named_sync(1, kPrSoftmaxThreads);
        float* part = p.partials + (size_t(blockIdx.x) * 2 + (x.k0 == 0 ? 1 : 0)) * kLtPartialFloats;
        if (part_of_row == 0) {
          const float sum = (s_red[row] + s_red[kPrOwn + row]) + (s_red[2 * kPrOwn + row] + s_red[3 * kPrOwn + row]);
          if (whole) {
            // Into the other CTA by turns: it may still be at the result of
            // the whole tile before, which takes the other buffer.  That one
            // is free: all of its warps have said (bar_inv) that they have
            // this CTA's rows' sums of the tile before, behind their last read
            // of the one before that.  Own rows' go where this thread's
            // partial sums were.
            const float inv = 1.f / sum;
            s_red[row] = inv;
            asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(
                             cluster_addr(s_inv + (wholes & 1) * kPrOwn + row, rank ^ 1)),
                         "f"(inv)
                         : "memory");
          } else {
            part[kPrRows * kLatentDim / 2 + row] = m;
            part[kPrRows * kLatentDim / 2 + kPrOwn + row] = sum;
          }
        }
        named_sync(1, kPrSoftmaxThreads);
        if (whole) {
          // both CTAs need all 128 rows' sums (said before the wait for the last
          // P V, which takes as long as the word to the other CTA)
          __syncwarp();
          if (lane == 0) {
            arrive_publish(cluster_addr(bar_inv, 0));
            arrive_publish(cluster_addr(bar_inv, 1));
          }
        }
        wait(bar_vfree + kPrSlicesV - 1, (gv - 1) & 1);
        const float* s_other = s_inv + (wholes & 1) * kPrOwn;
        if (whole) {
          if (ok) ok = __all_sync(0xffffffffu, wait_published(bar_inv, wholes & 1));
          ++wholes;
        }
        if (ok) {
          tc_fence_after();
          // lane: dim rank * 256 + e * 128 + quad * 32 + lane; column: row
          if (!whole) {
#pragma unroll 1
            for (int i = 0; i < 4; ++i) {
              const int e = i >> 1, r1 = wg * kPrOwn + (i & 1) * 32;
              if (r1 >= x.rows) continue;
              float o[32];
              tmem_ld32f(tmem + uint32_t(e * kPrRows + r1) + lane_off, o);
              float4* to = reinterpret_cast<float4*>(part) + ((e * 4 + quad) * (kPrRows / 4) + r1 / 4) * 32 + lane;
#pragma unroll
              for (int c = 0; c < 32; c += 4)
                if (r1 + c < x.rows) to[c * 8] = make_float4(o[c], o[c + 1], o[c + 2], o[c + 3]);
            }
          }
        }
        if (whole) {
          // 32 rows at a time through P's buffer (the last P V is done with
          // it), so that a row's 512 bytes leave in one piece: 2-byte or
          // paired stores straight from the columns take 6000 cycles a tile.
          uint8_t* stage = sm + S::p;
          const int e = wg;
#pragma unroll 1
          for (int r1 = 0; r1 < x.rows; r1 += 32) {
            const float* s_of = ((r1 >> 6) == rank ? s_red : s_other) + (r1 & (kPrOwn - 1));
            float o[32];
            tmem_ld32f(tmem + uint32_t(e * kPrRows + r1) + lane_off, o);
            // even lanes take the first row's pair of dims, odd lanes the
            // second's; odd rows swap their 64-byte halves, for the banks
            uint8_t* to = stage + (lane & 1) * 512 + ((e * 256 + quad * 64 + (lane >> 1) * 4) ^ ((lane & 1) << 6));
#pragma unroll
            for (int c = 0; c < 32; c += 4) {
              const float4 inv = *reinterpret_cast<const float4*>(s_of + c);
              const float v[4] = {o[c] * inv.x, o[c + 1] * inv.y, o[c + 2] * inv.z, o[c + 3] * inv.w};
#pragma unroll
              for (int h = 0; h < 4; h += 2) {
                const float other = __shfl_xor_sync(0xffffffffu, (lane & 1) ? v[h] : v[h + 1], 1);
                *reinterpret_cast<uint32_t*>(to + (c + h) * 512) =
                    (lane & 1) ? pack_bf16x2(other, v[h + 1]) : pack_bf16x2(v[h], other);
              }
            }
            named_sync(1, kPrSoftmaxThreads);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const int r = j * 8 + warp;
              const uint4 v = *reinterpret_cast<const uint4*>(stage + r * 512 + ((lane * 16) ^ ((r & 1) << 6)));
              if (ok && r1 + r < x.rows)
                *(reinterpret_cast<uint4*>(p.out + size_t(x.row0 + r1 + r) * kLatentDim + rank * 256) + lane) = v;
            }
            named_sync(1, kPrSoftmaxThreads);
          }
        }
        tc_fence_before();  // read before the next piece's first P V overwrites it
      }
      if (over) s_flags[0] = kOverflow;  // (a plain store: every writer's value)
    }
    // Both CTAs agree on whether there is a second round.  (One thread of a
    // warp that stores nothing to global memory tells the other CTA: a release
    // over every thread's stores would wait for the results to be written.)
    const bool failed = __syncthreads_or(!ok) != 0;
    if (warp == 9 && lane == 0) {
      const int mine = failed ? kTimeout : int(s_flags[0]);
      s_flags[0] = mine;
      asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(cluster_addr(const_cast<int*>(s_flags + 1), rank ^ 1)),
                   "r"(mine)
                   : "memory");
      arrive_publish(cluster_addr(bar_round, rank ^ 1));
      if (failed) flag_status(p.status, PKV_STATUS_TIMEOUT);
      if (!wait_published(bar_round, round)) s_flags[0] = kTimeout;
    }
    __syncthreads();
    if ((s_flags[0] | s_flags[1]) != kOverflow) break;
  }

  // What is still under way lands before shared memory and TMEM are let go of:
  // each CTA's copies on its own barriers, and the MMAs' commits.
  if ((warp == 8 || warp == 11) && lane == 0) {
    const uint64_t limit = ok ? kLandLimitNs : kDrainLimitNs;
    const int n = warp == 8 ? kPrSlicesK : kPrSlicesV;
    const int sent = warp == 8 ? slices : slices + tails;  // phases of the leader's barriers
    uint64_t* bar = warp == 8 ? bar_k : bar_v;
    if (rank == 0)  // they count both CTAs' copies
      for (int i = max(0, sent - n); i < sent; ++i) mbar_wait(bar + i % n, (i / n) & 1, limit);
    for (int i = max(0, tails - n); i < tails; ++i) mbar_wait(bar_tail + i % n, (i / n) & 1, limit);
    if (warp == 8 && pieces > 0) {
      mbar_wait(bar_q, (pieces - 1) & 1, limit);
      mbar_wait(bar_qfree, (pieces - 1) & 1, limit);  // (commits that reach this CTA)
      for (int d = 0; d < n; ++d) mbar_wait(bar_kfree + d, (g - 1) & 1, limit);
    }
  }
  if (warp == 9 && rank == 0 && g > 0) mbar_wait(bar_s + ((g - 1) & 1), ((g - 1) >> 1) & 1, kLandLimitNs);
  if (warp == 10 && rank == 0 && gv > 0) mbar_wait(bar_vfree + kPrSlicesV - 1, (gv - 1) & 1, kLandLimitNs);
  __syncwarp();

  // A share that begins and ends at the same block inside a tile is a piece
  // without keys, which the merge skips by its l of 0.
  if (begin.k > 0 && begin.b == end.b && begin.j == end.j && begin.k == end.k && tid < kPrOwn)
    p.partials[size_t(blockIdx.x) * 2 * kLtPartialFloats + kPrRows * kLatentDim / 2 + kPrOwn + tid] = 0.f;
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // neither CTA leaves while the other may still reach into it
  tc_fence_after();
  if (warp == 9)
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512u));
}

}  // namespace

int launch_latent_pair(const LaunchCtx& ctx, const LatentAttendArgs& a, const LatentParams& lp) {
  static std::mutex mu;
  static bool ready[64] = {};
  {
    std::lock_guard<std::mutex> lk(mu);
    if (!ready[ctx.dev->device]) {
      if (cudaFuncSetAttribute(pkv_latent_pair_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                               int(PrSmem::bytes)) != cudaSuccess) {
        cudaGetLastError();
        return PKV_ERR_LAUNCH;
      }
      ready[ctx.dev->device] = true;
    }
  }
  const pkv_desc& d = a.desc;
  CUtensorMap tq, tk, tv;
  {
    const cuuint64_t dims[3] = {64, cuuint64_t(a.num_tokens) * d.num_q_heads, kLtChunks};
    const cuuint64_t strides[2] = {kLatentRow * 2, 128};
    const cuuint32_t box[3] = {64, kPrOwn, kLtChunks};
    if (!encode_tensor_map(&tq, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, a.q, 3, dims, strides, box)) return PKV_ERR_LAUNCH;
  }
  {
    const cuuint64_t dims[4] = {64, 8, kLtChunks, cuuint64_t(d.num_blocks) * 2};
    const cuuint64_t strides[3] = {kLatentRow * 2, 128, kLatentRow * 16};
    const cuuint32_t box_k[4] = {64, 8, 3, 2}, box_v[4] = {64, 8, 4, 2};
    if (!encode_tensor_map(&tk, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, a.cache, 4, dims, strides, box_k) ||
        !encode_tensor_map(&tv, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, a.cache, 4, dims, strides, box_v))
      return PKV_ERR_LAUNCH;
  }
  const unsigned pairs = unsigned(ctx.dev->sm_count / 2);
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = 2;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2 * pairs);
  cfg.blockDim = dim3(kPrThreads);
  cfg.dynamicSmemBytes = PrSmem::bytes;
  cfg.stream = ctx.stream;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  {
    TraceScope ts(ctx.stream, PKV_K_LATENT);
    cudaLaunchKernelEx(&cfg, pkv_latent_pair_kernel, tq, tk, tv, lp);
    if (int e = ts.done()) return e;
  }
  cfg.gridDim = dim3(pairs, lt_merge_blocks(kPrRows));
  cfg.blockDim = dim3(kLtMergeThreads);
  cfg.dynamicSmemBytes = 0;
  cfg.numAttrs = 1;
  TraceScope ts(ctx.stream, PKV_K_MERGE);
  cudaLaunchKernelEx(&cfg, pkv_latent_merge_kernel<kPrRows, true>, lp);
  return ts.done();
}

}  // namespace pkv
