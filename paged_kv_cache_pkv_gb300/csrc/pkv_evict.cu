// pkv_evict.cu -- eviction by accumulated attention weight: of every sequence
// above its budget each kv head keeps its first tokens, its most recent ones
// and those of the largest scores between, and moves them together in place.
//
// An item is one kv head of one sequence.  Many short items get a CTA of 256
// threads each that does everything; otherwise an item has a cluster of up to
// sixteen CTAs of 1024 threads for the selection (steps 1 to 3) and, in a second
// kernel, one for its K rows and one for its V rows (step 4).  The CTAs of a
// cluster split the candidates, the tokens between the first and the recent
// ones, into slices:
//  1. Scores become 32-bit keys of the same order (sign and magnitude turned
//     into an unsigned number), kept in shared memory (kKeys a CTA, the rest
//     of a very long slice is read again).
//  2. The key of the c-th largest by radix selection, 11 + 11 + 10 bits from
//     the top: a histogram of the keys that agree so far in every CTA, its
//     counts added up through distributed shared memory (only those that are
//     not 0 travel; all CTAs reading all histograms took half of the selection).
//     Attention weights spread over a few dozen powers of two, so the first
//     digit, exponent and two bits of the mantissa, already parts them; where
//     all of a bin stay, the digits behind it are not looked at.
//  3. Keys above it stay; of those equal to it the lowest tokens, as many as
//     are missing, counted over the slices in order.  The tokens that stay are
//     listed in the workspace (4 bytes each beside 512 or 258 bytes that move).
//  4. Rows move in rounds of kRows a CTA, row q of the list to the q-th row
//     behind the first tokens.  A kept token never moves up (src >= dst, as
//     the list is in order), so what a round writes can only be what the same
//     or an earlier round reads: a round's rows are all in registers, cluster
//     wide, before any of them is written, and nothing else has to wait.  Once
//     a round's first row comes from behind all that it writes, only earlier
//     rounds read there, and the barrier of the round before is enough.
//
// What bounds it: bytes, a row read and written once (2 x 512 bytes a token
// and head on bf16 pages); on few tokens the chain of steps 1 to 3.  From cold
// caches: one sequence of 131072 tokens cut to 32768, eight heads, bf16 pages, 73
// us (selection 23, moves 50 at 5.3 TB/s); 64 sequences of 512 to 4096 tokens cut
// to 1023, E4M3 pages, 55 us (moves at 5.8 TB/s).  With one kernel and a barrier
// a round the first took 213 us.
#include <cooperative_groups.h>

#include <atomic>
#include <mutex>

#include "pkv_common.cuh"
#include "pkv_internal.h"

namespace pkv {
namespace {

namespace cg = cooperative_groups;

constexpr int kSmallThreads = 256, kBigThreads = 1024;
constexpr int kBins = 2048;
constexpr int kMaxCluster = 16;

template <int kThreads>
struct EvictShared {
  // Keys of a slice that are held here: all that the kernel of 256 threads is
  // launched for, four CTAs of it an SM (6144, which halve what they leave L1 for
  // rows on their way: the E4M3 case above 66 us; two or three CTAs an SM of
  // more registers: 60 sequences of 4000 tokens 74 us, 64 as it is).
  static constexpr int kKeys = kThreads == kBigThreads ? 24576 : 4096;
  uint32_t hist[3][kBins];  // of each pass
  // A cluster's counts, of each pass: every CTA has those of the pairs of bins
  // that are its own, pair i the CTA i % cluster's.
  uint32_t total[kThreads == kBigThreads ? 3 : 1][kThreads == kBigThreads ? kBins : 2];
  uint32_t keys[kKeys];
  uint32_t warp_sum[kThreads / 32], warp_eq[kThreads / 32];
  uint32_t digit, rest, whole;  // of the last selection pass
  uint32_t count_gt, count_eq;  // of this CTA's slice
};

// A key that orders like the score: NaN as -infinity, -0 as 0.
__device__ __forceinline__ uint32_t order_key(float x) {
  if (x != x) x = -INFINITY;
  const uint32_t u = __float_as_uint(x + 0.0f);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// What one kv head of one sequence keeps: its first f tokens, c of the N between,
// the last r.
struct Cut {
  int b, g, L, f, r, c, N;
  const int32_t* table;
  int32_t* list;  // the c tokens
};

// False where nothing is cut: a short sequence, or (flagged by one thread, as new
// lengths are written by one) numbers that do not fit.  The same in all CTAs.
__device__ __forceinline__ bool cut_of(const EvictArgs& p, int item, int list_stride, bool speaks, Cut& x) {
  const int Hkv = p.desc.num_kv_heads;
  x.b = item / Hkv;
  x.g = item - x.b * Hkv;
  const int L = __ldg(p.seq_lens + x.b), m = __ldg(p.keep + x.b);
  const int first = p.first ? __ldg(p.first + x.b) : 0;
  const bool bad = L < 0 || m < 0 || first < 0 || (L > 0 && (L - 1) / kPage >= p.desc.max_blocks_per_seq);
  if (speaks && x.g == 0 && threadIdx.x == 0) {
    p.new_lens[x.b] = bad ? L : min(L, m);
    if (bad) flag_status(p.status, PKV_STATUS_BAD_QUERY);
  }
  x.L = L;
  x.f = min(first, m);
  x.r = min(p.recent, m - x.f);
  x.c = m - x.f - x.r;
  x.N = L - x.r - x.f;  // more than c
  x.table = p.block_tables + int64_t(x.b) * p.desc.max_blocks_per_seq;
  x.list = reinterpret_cast<int32_t*>(p.workspace) + int64_t(item) * list_stride;
  return !bad && L > m;
}

// A page's row of the head in the pools: [num_blocks][Hkv][16].
__device__ __forceinline__ int64_t pool_row(const EvictArgs& p, int g, int page, int token) {
  return (int64_t(page) * p.desc.num_kv_heads + g) * kPage + token % kPage;
}

// Steps 1 to 3 (see above): the list of c > 0 tokens.  When it returns, a single
// CTA has its list whole; of a cluster each CTA has written its own part, and
// the others' parts are there only for the kernel behind (the last cluster
// barrier is arrived at before the list is written: it lets the CTAs' shared
// memory go).
template <int kThreads>
__device__ __forceinline__ void select_tokens(const EvictArgs& p, const Cut& x, int cluster, int rank,
                                              EvictShared<kThreads>& sh) {
  constexpr int kWarps = kThreads / 32, kKeys = EvictShared<kThreads>::kKeys;
  const cg::cluster_group cl = cg::this_cluster();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

  // ---- this CTA's slice of the candidates, and their keys ----
  const int per = ((x.N + cluster - 1) / cluster + 31) / 32 * 32;
  const int s0 = min(x.N, rank * per), n = min(x.N, s0 + per) - s0;
  const int token0 = x.f + s0;
  // (eight table reads, then eight score reads of a thread on their way at once)
  constexpr int kBatch = 8;
  auto read_pages = [&](int i0, int (&page)[kBatch]) {
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const int i = i0 + k * kThreads;
      page[k] = i < n ? __ldg(x.table + (token0 + i) / kPage) : 0;
    }
  };
  auto read_scores = [&](int i0, const int (&page)[kBatch], float (&score)[kBatch]) {
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const int i = i0 + k * kThreads;
      score[k] = -INFINITY;
      if (page[k] < 0 || page[k] >= p.desc.num_blocks) flag_status(p.status, PKV_STATUS_BAD_BLOCK);
      else if (i < n) score[k] = __ldcg(p.scores + pool_row(p, x.g, page[k], token0 + i));
    }
  };
  // a key beyond those that shared memory holds
  auto read_key = [&](int i) {
    const int page = __ldg(x.table + (token0 + i) / kPage);
    if (page < 0 || page >= p.desc.num_blocks) return order_key(-INFINITY);
    return order_key(__ldcg(p.scores + pool_row(p, x.g, page, token0 + i)));
  };
  auto key_at = [&](int i) { return i < kKeys ? sh.keys[i] : read_key(i); };

  int page[kBatch];
  read_pages(tid, page);

  // ---- the c-th largest key, digit by digit ----
  // The first digit is counted while the keys come in.
  for (int i = tid; i < 3 * kBins; i += kThreads) (&sh.hist[0][0])[i] = 0;
  if constexpr (kThreads == kBigThreads) {
    if (cluster > 1) {
      for (int i = tid; i < 3 * kBins; i += kThreads) (&sh.total[0][0])[i] = 0;
      cluster_arrive();
    }
  }
  __syncthreads();
  for (int i0 = tid; i0 < n; i0 += kBatch * kThreads) {
    float score[kBatch];
    read_scores(i0, page, score);
    read_pages(i0 + kBatch * kThreads, page);
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const int i = i0 + k * kThreads;
      if (i < n) {
        const uint32_t key = order_key(score[k]);
        if (i < kKeys) sh.keys[i] = key;
        atomicAdd(&sh.hist[0][key >> 21], 1u);
      }
    }
  }
  // threshold, rest: keys above it stay, and so many of those equal to it.
  uint32_t threshold = 0, rest = uint32_t(x.c);
#pragma unroll 1
  for (int pass = 0; pass < 3; ++pass) {
    const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
    uint32_t* hist = sh.hist[pass];
    if (pass > 0) {
      const int above = pass == 1 ? 21 : 10;  // bits from here on are known
      const uint32_t mask = pass == 2 ? 1023u : 2047u;
#pragma unroll 4
      for (int i = tid; i < n; i += kThreads) {
        const uint32_t key = key_at(i);
        if (key >> above == threshold >> above) atomicAdd(&hist[(key >> shift) & mask], 1u);
      }
    }
    __syncthreads();
    // Bins from the top, kPer a thread, summed over the cluster.
    constexpr int kPer = kBins / kThreads;
    const int low = kBins - kPer * (tid + 1);
    const uint32_t* counts = hist;
    if constexpr (kThreads == kBigThreads) {
      if (cluster > 1) {
        if (pass == 0) cluster_wait();  // all counts are 0
        for (int i = tid; i < kBins; i += kThreads)
          if (const uint32_t v = hist[i]) atomicAdd(cl.map_shared_rank(&sh.total[pass][i], (i >> 1) % cluster), v);
        cl.sync();
        static_assert(kBins / kBigThreads == 2, "a thread reads one pair");
        counts = cl.map_shared_rank(sh.total[pass], (low >> 1) % cluster);
      }
    }
    uint32_t bin[kPer];  // of bins low + kPer - 1 down to low
#pragma unroll
    for (int i = 0; i < kPer; i += 2) {
      const uint2 v = *reinterpret_cast<const uint2*>(counts + low + i);
      bin[kPer - 1 - i] = v.x;
      bin[kPer - 2 - i] = v.y;
    }
    uint32_t mine = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) mine += bin[i];
    uint32_t incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    if (lane == 31) sh.warp_sum[warp] = incl;
    __syncthreads();
    const uint32_t others = __reduce_add_sync(0xffffffffu, lane < warp ? sh.warp_sum[lane % kWarps] : 0u);
    uint32_t before = others + incl - mine;
    if (before < rest && rest <= before + mine) {  // one thread: the digit is in its bins
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        if (before < rest && rest <= before + bin[i]) {
          sh.digit = uint32_t(low + kPer - 1 - i);
          sh.rest = rest - before;
          sh.whole = rest - before == bin[i];
        }
        before += bin[i];
      }
    }
    __syncthreads();
    threshold |= sh.digit << shift;
    rest = sh.rest;
    // All keys of the bin stay: no more digits.  (Of a few thousand scores 22 bits
    // part the last that stays from the next.  No key is 0.)
    if (sh.whole) {
      --threshold;
      rest = 0;
      break;
    }
  }

  // ---- how many stay of the slices before ----
  // Warps take whole words of 32 candidates in order, a contiguous run each.
  const int words = (n + 31) / 32;
  const int w_per = (words + kWarps - 1) / kWarps;
  const int w0 = min(words, warp * w_per), w1 = min(words, w0 + w_per);
  uint32_t gt = 0, eq = 0;
#pragma unroll 4
  for (int w = w0; w < w1; ++w) {
    const int i = 32 * w + lane;
    if (i < n) {
      const uint32_t key = key_at(i);
      gt += key > threshold;
      eq += key == threshold;
    }
  }
  gt = __reduce_add_sync(0xffffffffu, gt);
  eq = __reduce_add_sync(0xffffffffu, eq);
  if (lane == 0) {
    sh.warp_sum[warp] = gt;
    sh.warp_eq[warp] = eq;
  }
  __syncthreads();
  const uint32_t gt_mine = lane < kWarps ? sh.warp_sum[lane] : 0u, eq_mine = lane < kWarps ? sh.warp_eq[lane] : 0u;
  uint32_t gt_before = __reduce_add_sync(0xffffffffu, lane < warp ? gt_mine : 0u);
  uint32_t eq_before = __reduce_add_sync(0xffffffffu, lane < warp ? eq_mine : 0u);
  if (cluster > 1) {
    const uint32_t a = __reduce_add_sync(0xffffffffu, gt_mine), e = __reduce_add_sync(0xffffffffu, eq_mine);
    if (tid == 0) {
      sh.count_gt = a;
      sh.count_eq = e;
    }
    cl.sync();
    uint32_t g_other = 0, e_other = 0;
    if (lane < rank) {
      g_other = *cl.map_shared_rank(&sh.count_gt, lane);
      e_other = *cl.map_shared_rank(&sh.count_eq, lane);
    }
    gt_before += __reduce_add_sync(0xffffffffu, g_other);
    eq_before += __reduce_add_sync(0xffffffffu, e_other);
    cluster_arrive();  // nothing of the other CTAs is read any more
  }
  // ---- the list, in order ----
#pragma unroll 4
  for (int w = w0; w < w1; ++w) {
    const int i = 32 * w + lane;
    const uint32_t key = i < n ? key_at(i) : 0u;
    const bool above = i < n && key > threshold, same = i < n && key == threshold;
    const uint32_t gts = __ballot_sync(0xffffffffu, above), eqs = __ballot_sync(0xffffffffu, same);
    const uint32_t below = (1u << lane) - 1u;
    const uint32_t eq_rank = eq_before + __popc(eqs & below);
    if (above || (same && eq_rank < rest))
      x.list[gt_before + __popc(gts & below) + min(eq_rank, rest)] = token0 + i;
    gt_before += __popc(gts);
    eq_before += __popc(eqs);
  }
  if (cluster > 1) cluster_wait();
  else __syncthreads();
}

// Step 4.  kBoth: K and V rows of the item together, the lanes of a row's first
// half K's.  Otherwise those of `part`: 0 K's, 1 V's.  16 bytes a lane.
template <bool F8, int kThreads, bool kBoth>
__device__ __forceinline__ void move_rows(const EvictArgs& p, const Cut& x, int cluster, int rank, int part) {
  constexpr int kVecs = F8 ? 8 : 16;                  // 16-byte vectors of a row of K or of V
  constexpr int kLanes = kBoth ? 2 * kVecs : kVecs;
  constexpr int kSub = 32 / kLanes;                   // rows that a warp moves at a time
  constexpr int kDeep = 8;                            // times, all in flight
  constexpr int kWarpRows = kSub * kDeep;             // 8 to 32
  constexpr int kRows = kWarpRows * (kThreads / 32);  // rows of a CTA's round
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int f = x.f, c = x.c, L = x.L, r = x.r, total = c + r;
  const int sub = lane / kLanes, in_row = lane % kLanes;
  const bool is_v = kBoth ? in_row >= kVecs : part == 1;
  uint4* const pool = reinterpret_cast<uint4*>(is_v ? p.v_cache : p.k_cache);
  const int vec = in_row % kVecs;
  const bool moves_k = kBoth || part == 0, moves_v = kBoth || part == 1;  // their scales, K's the scores
  // Lane l < kWarpRows sees to row l of the warp's in a round: the token that it
  // comes from is read two rounds ahead, the pages one, so that neither the row
  // copies nor the barrier wait for a table.
  const int64_t round_rows = int64_t(cluster) * kRows;
  const int64_t mine = int64_t(rank) * kRows + warp * kWarpRows + lane;
  auto token_of = [&](int64_t q) {  // -1: no row
    return lane >= kWarpRows || q >= total ? -1 : q < c ? __ldcg(x.list + q) : L - r + int(q - c);
  };
  auto lowest_of = [&](int64_t base) {  // of a round's sources
    return base >= total ? 0 : base < c ? __ldcg(x.list + base) : L - r + int(base - c);
  };
  struct Pages {
    int src, dst;
  };
  auto pages_of = [&](int64_t q, int from) {
    if (from < 0) return Pages{0, 0};
    return Pages{__ldg(x.table + from / kPage), __ldg(x.table + (f + int(q)) / kPage)};
  };
  // Rows of the pools, -1 where nothing moves: it is in its place, or a page is
  // not one of the pool's.
  auto rows_of = [&](int64_t q, int from, Pages pg, int64_t& src, int64_t& dst) {
    const int to = f + int(q);
    src = dst = -1;
    if (from < 0 || from == to) return;
    if (pg.src < 0 || pg.src >= p.desc.num_blocks || pg.dst < 0 || pg.dst >= p.desc.num_blocks) {
      flag_status(p.status, PKV_STATUS_BAD_BLOCK);
      return;
    }
    src = pool_row(p, x.g, pg.src, from);
    dst = pool_row(p, x.g, pg.dst, to);
  };
  int from = token_of(mine);
  Pages pages = pages_of(mine, from);
  int lowest = cluster > 1 ? lowest_of(0) : 0;
  int next = token_of(mine + round_rows);
  for (int64_t base = 0; base < total; base += round_rows) {
    int64_t src, dst;
    rows_of(base + mine, from, pages, src, dst);
    from = next;
    pages = pages_of(base + round_rows + mine, from);
    next = token_of(base + 2 * round_rows + mine);
    const bool ahead = lowest >= f + base + round_rows;
    if (cluster > 1) lowest = lowest_of(base + round_rows);
    // 0 and not undefined, so that the loads are predicated and not branched
    // around, and in one kernel with the selection past L1: 240 sequences of 500
    // tokens 144 -> 130 -> 124 us.  (Loads that stream, in kernels of their own:
    // 30 sequences of 4000 tokens 64 us, 66 past L1.)
    uint4 v[kDeep] = {};
#pragma unroll
    for (int i = 0; i < kDeep; ++i) {
      const int64_t s = __shfl_sync(0xffffffffu, src, i * kSub + sub);
      if (s >= 0) v[i] = kBoth ? __ldcg(pool + s * kVecs + vec) : __ldcs(pool + s * kVecs + vec);
    }
    float score = 0.f;
    uint8_t ks = 0, vs = 0;
    if (src >= 0) {
      if (moves_k) score = __ldcg(p.scores + src);
      if constexpr (F8) {
        if (moves_k) ks = __ldcg(p.k_scale + src);
        if (moves_v) vs = __ldcg(p.v_scale + src);
      }
    }
    // Every row that these writes may hit has been read (release and acquire
    // order reads too).
    if (cluster == 1) {
      __syncthreads();
    } else {
      if (base > 0) cluster_wait();  // rounds before
      cluster_arrive();
      if (!ahead) {
        cluster_wait();
        cluster_arrive();  // (so that one is always under way)
      }
    }
#pragma unroll
    for (int i = 0; i < kDeep; ++i) {
      const int64_t d = __shfl_sync(0xffffffffu, dst, i * kSub + sub);
      if (d >= 0) pool[d * kVecs + vec] = v[i];
    }
    if (dst >= 0) {
      if (moves_k) p.scores[dst] = score;
      if constexpr (F8) {
        if (moves_k) p.k_scale[dst] = ks;
        if (moves_v) p.v_scale[dst] = vs;
      }
    }
  }
  if (cluster > 1 && total > 0) cluster_wait();
}

// Everything read here may be the work of the kernel before.  No early start for
// the one behind a kernel that writes new lengths: pkv_attend reads lengths before
// it waits.

// A CTA an item, selection and move.
template <bool F8>
__global__ void __launch_bounds__(kSmallThreads, 4) pkv_evict_kernel(const EvictArgs p, int list_stride) {
  extern __shared__ __align__(16) uint8_t smem_raw[];
  griddep_wait();
  Cut x;
  if (!cut_of(p, blockIdx.x, list_stride, true, x)) return;
  if (x.c > 0) select_tokens<kSmallThreads>(p, x, 1, 0, *reinterpret_cast<EvictShared<kSmallThreads>*>(smem_raw));
  move_rows<F8, kSmallThreads, true>(p, x, 1, 0, 0);
}

// A cluster an item: the selection.
__global__ void __launch_bounds__(kBigThreads, 1) pkv_evict_select_kernel(const EvictArgs p, int cluster,
                                                                          int list_stride) {
  extern __shared__ __align__(16) uint8_t smem_raw[];
  griddep_launch_dependents();  // pkv_evict_move_kernel, which waits first and itself starts nothing early
  griddep_wait();
  const int rank = blockIdx.x % cluster;
  Cut x;
  if (!cut_of(p, blockIdx.x / cluster, list_stride, false, x) || x.c == 0) return;  // the whole cluster
  select_tokens<kBigThreads>(p, x, cluster, rank, *reinterpret_cast<EvictShared<kBigThreads>*>(smem_raw));
}

// A cluster for the K rows of an item, one for its V rows: they have nothing to do
// with each other once the list is there, and with few items twice the SMs take
// part.  (Clusters for halves of rows took as long or longer.)
template <bool F8>
__global__ void __launch_bounds__(kBigThreads, 1) pkv_evict_move_kernel(const EvictArgs p, int cluster,
                                                                        int list_stride) {
  griddep_wait();
  const int rank = blockIdx.x % cluster, part = blockIdx.x / cluster;
  Cut x;
  if (!cut_of(p, part / 2, list_stride, rank == 0 && part % 2 == 0, x)) return;
  move_rows<F8, kBigThreads, false>(p, x, cluster, rank, part % 2);
}

int list_stride(const pkv_desc& d) { return d.max_blocks_per_seq * kPage; }

cudaLaunchConfig_t config(cudaLaunchAttribute (&attr)[2], cudaStream_t stream, int64_t ctas, int cluster, int threads,
                          size_t smem) {
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = unsigned(cluster);
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(ctas));
  cfg.blockDim = dim3(unsigned(threads));
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cfg;
}

// Cluster sizes in use, and how many clusters of each a device runs at once with
// a CTA of 1024 threads an SM (a cluster stays within a GPC), asked once.
constexpr int kSizes[] = {1, 2, 3, 4, 6, 8, 12, 16};
struct Resident {
  int most[sizeof(kSizes) / sizeof(kSizes[0])];
};

template <bool F8>
const Resident* resident(int device) {
  static Resident facts[64];
  static std::atomic<bool> done[64] = {};
  static std::mutex asking;
  if (device < 0 || device >= 64) return nullptr;
  if (done[device].load(std::memory_order_acquire)) return &facts[device];
  std::lock_guard<std::mutex> lock(asking);
  // (another thread may have been through meanwhile: what others read is written once)
  if (done[device].load(std::memory_order_relaxed)) return &facts[device];
  auto set = [](auto kernel, size_t smem) {
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem)) == cudaSuccess &&
           cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) == cudaSuccess;
  };
  constexpr size_t smem = sizeof(EvictShared<kBigThreads>);
  if (!set(pkv_evict_kernel<F8>, sizeof(EvictShared<kSmallThreads>)) || !set(pkv_evict_select_kernel, smem) ||
      !set(pkv_evict_move_kernel<F8>, 0)) {
    cudaGetLastError();
    return nullptr;
  }
  int i = 0;
  for (int size : kSizes) {
    cudaLaunchAttribute attr[2];
    const cudaLaunchConfig_t cfg = config(attr, nullptr, size, size, kBigThreads, smem);
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, pkv_evict_select_kernel, &cfg) != cudaSuccess) {
      cudaGetLastError();  // a size that this device cannot run
      n = 0;
    }
    facts[device].most[i++] = n;
  }
  done[device].store(true, std::memory_order_release);
  return &facts[device];
}

// CTAs a cluster: as many as let all clusters run at once, none for less than
// 512 tokens of the widest sequence.
int cluster_size(const Resident& r, int64_t clusters, int64_t tokens) {
  int n = 1, i = 0;
  for (int size : kSizes)
    if (clusters <= r.most[i++] && tokens >= int64_t(512) * size) n = size;
  return n;
}

}  // namespace

size_t evict_workspace_bytes(const pkv_desc& d, int32_t num_seqs) {
  return align_up(sizeof(int32_t) * size_t(num_seqs) * size_t(d.num_kv_heads) * size_t(list_stride(d)), 256);
}

int launch_evict(const LaunchCtx& ctx, const EvictArgs& a, bool fp8) {
  if (a.workspace_bytes < evict_workspace_bytes(a.desc, a.num_seqs)) return PKV_ERR_WORKSPACE;
  const Resident* facts = fp8 ? resident<true>(ctx.dev->device) : resident<false>(ctx.dev->device);
  if (!facts) return PKV_ERR_LAUNCH;
  const int64_t items = int64_t(a.num_seqs) * a.desc.num_kv_heads;
  const int64_t tokens = int64_t(a.desc.max_blocks_per_seq) * kPage;
  if (items * 2 * kMaxCluster > INT32_MAX) return PKV_ERR_RANGE;
  const int stride = list_stride(a.desc);
  cudaLaunchAttribute attr[2];
  // Items of few tokens are better off with a CTA each of one kernel where they
  // fill the GPU (us, one kernel against two, 8 heads, bf16: 240 sequences of 500
  // tokens 105 against 187, 64 of 2000 100 against 116, 60 of 4000 102 against 113,
  // on E4M3 pages 63 against 82, 20 of 4000 48 against 50; but 16 of 4000 44
  // against 38, 8 of 4000 38 against 29, 60 of 8000 210 against 197).  So are two
  // tokens a thread (16 sequences of 500 13 against 18, 1 of 500 15 against 14).
  if (tokens <= EvictShared<kSmallThreads>::kKeys && (items > ctx.dev->sm_count || tokens <= 2 * kSmallThreads)) {
    const cudaLaunchConfig_t cfg =
        config(attr, ctx.stream, items, 1, kSmallThreads, sizeof(EvictShared<kSmallThreads>));
    TraceScope ts(ctx.stream, PKV_K_EVICT);
    cudaLaunchKernelEx(&cfg, fp8 ? pkv_evict_kernel<true> : pkv_evict_kernel<false>, a, stride);
    return ts.done();
  }
  {
    const int cluster = cluster_size(*facts, items, tokens);
    const cudaLaunchConfig_t cfg =
        config(attr, ctx.stream, items * cluster, cluster, kBigThreads, sizeof(EvictShared<kBigThreads>));
    TraceScope ts(ctx.stream, PKV_K_EVICT);
    cudaLaunchKernelEx(&cfg, pkv_evict_select_kernel, a, cluster, stride);
    if (int e = ts.done()) return e;
  }
  const int cluster = cluster_size(*facts, items * 2, tokens);
  const cudaLaunchConfig_t cfg = config(attr, ctx.stream, items * 2 * cluster, cluster, kBigThreads, 0);
  TraceScope ts(ctx.stream, PKV_K_EVICT);
  cudaLaunchKernelEx(&cfg, fp8 ? pkv_evict_move_kernel<true> : pkv_evict_move_kernel<false>, a, cluster, stride);
  return ts.done();
}

}  // namespace pkv
