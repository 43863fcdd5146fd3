// pkv_evict.cu -- eviction by accumulated attention weight: of every sequence
// above its budget each kv head keeps its first tokens, its most recent ones
// and those of the largest scores between, and moves them together in place.
//
// One cluster of CTAs (one to sixteen) an item, an item being one kv head of
// one sequence.  Its CTAs split the candidates, the tokens between the first
// and the recent ones, into slices:
//  1. Scores become 32-bit keys of the same order (sign and magnitude turned
//     into an unsigned number), kept in shared memory (kKeys a CTA, the rest
//     of a very long slice is read again).
//  2. The key of the c-th largest by radix selection, 11 + 11 + 10 bits from
//     the top: a histogram of the keys that agree so far in every CTA, read by
//     all through distributed shared memory.  Attention weights spread over a
//     few dozen powers of two, so the first digit, exponent and two bits of
//     the mantissa, already parts them.
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
// Items that fill the GPU get 256 threads each, four CTAs an SM; fewer items a
// cluster of CTAs of 1024 threads, one an SM (one sequence of 131072 tokens,
// eight heads: 16 CTAs of 256 threads and a barrier a round took 258 us).
//
// What bounds it: bytes, a row read and written once (2 x 512 bytes a token
// and head on bf16 pages); on few tokens the chain of steps 1 to 3.
#include <cooperative_groups.h>

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
  static constexpr int kKeys = kThreads == kBigThreads ? 24576 : 8192;  // of a slice, held here
  uint32_t hist[2][kBins];
  uint32_t keys[kKeys];
  uint32_t warp_sum[kThreads / 32], warp_eq[kThreads / 32];
  uint32_t digit, rest;         // of the last selection pass
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

template <bool F8, int kThreads>
__global__ void __launch_bounds__(kThreads, kThreads == kBigThreads ? 1 : 4)
    pkv_evict_kernel(const EvictArgs p, int cluster, int list_stride) {
  extern __shared__ __align__(16) uint8_t smem_raw[];
  using Shared = EvictShared<kThreads>;
  Shared& sh = *reinterpret_cast<Shared*>(smem_raw);
  constexpr int kWarps = kThreads / 32, kKeys = Shared::kKeys;
  const cg::cluster_group cl = cg::this_cluster();
  auto sync_all = [&] {
    if (cluster > 1) cl.sync();
    else __syncthreads();
  };
  // Everything read here may be the work of the kernel before.  No early start
  // for the one behind: pkv_attend reads lengths before it waits, and these
  // are new ones.
  griddep_wait();
  const int rank = blockIdx.x % cluster;
  const int item = blockIdx.x / cluster;
  const int Hkv = p.desc.num_kv_heads;
  const int b = item / Hkv, g = item - b * Hkv;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

  const int L = __ldg(p.seq_lens + b), m = __ldg(p.keep + b);
  const int first = p.first ? __ldg(p.first + b) : 0;
  const bool bad = L < 0 || m < 0 || first < 0 || (L > 0 && (L - 1) / kPage >= p.desc.max_blocks_per_seq);
  if (g == 0 && rank == 0 && tid == 0) {
    p.new_lens[b] = bad ? L : min(L, m);
    if (bad) flag_status(p.status, PKV_STATUS_BAD_QUERY);
  }
  if (bad || L <= m) return;  // the whole cluster
  const int f = min(first, m);
  const int r = min(p.recent, m - f);
  const int c = m - f - r;   // candidates that stay
  const int N = L - r - f;   // candidates, more than c
  const int32_t* table = p.block_tables + int64_t(b) * p.desc.max_blocks_per_seq;
  // The page of a token, or -1.
  auto page_of = [&](int token) {
    const int id = __ldg(table + token / kPage);
    return id >= 0 && id < p.desc.num_blocks ? id : -1;
  };
  // A page's row of this head in the pools: [num_blocks][Hkv][16].
  auto row_of = [&](int page, int token) { return (int64_t(page) * Hkv + g) * kPage + token % kPage; };
  int32_t* list = reinterpret_cast<int32_t*>(p.workspace) + int64_t(item) * list_stride;

  if (c > 0) {
    // ---- this CTA's slice of the candidates, and their keys ----
    const int per = ((N + cluster - 1) / cluster + 31) / 32 * 32;
    const int s0 = min(N, rank * per), s1 = min(N, s0 + per);
    const int n = s1 - s0;
    auto read_key = [&](int i) {
      const int token = f + s0 + i;
      const int page = page_of(token);
      if (page < 0) {
        flag_status(p.status, PKV_STATUS_BAD_BLOCK);
        return order_key(-INFINITY);
      }
      return order_key(__ldcg(p.scores + row_of(page, token)));
    };
    auto key_at = [&](int i) { return i < kKeys ? sh.keys[i] : read_key(i); };
    // (eight table reads, then eight score reads of a thread on their way at once)
    constexpr int kBatch = 8;
    for (int i0 = tid; i0 < min(n, kKeys); i0 += kBatch * kThreads) {
      int page[kBatch];
      float score[kBatch];
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        const int i = i0 + k * kThreads;
        page[k] = i < min(n, kKeys) ? __ldg(table + (f + s0 + i) / kPage) : 0;
      }
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        const int i = i0 + k * kThreads;
        score[k] = -INFINITY;
        if (page[k] < 0 || page[k] >= p.desc.num_blocks) flag_status(p.status, PKV_STATUS_BAD_BLOCK);
        else if (i < min(n, kKeys)) score[k] = __ldcg(p.scores + row_of(page[k], f + s0 + i));
      }
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        const int i = i0 + k * kThreads;
        if (i < min(n, kKeys)) sh.keys[i] = order_key(score[k]);
      }
    }

    // ---- the c-th largest key, digit by digit ----
    uint32_t prefix = 0, rest = uint32_t(c);
#pragma unroll 1
    for (int pass = 0; pass < 3; ++pass) {
      const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
      const int above = pass == 0 ? 32 : pass == 1 ? 21 : 10;  // bits from here on are known
      const uint32_t mask = pass == 2 ? 1023u : 2047u;
      uint32_t* hist = sh.hist[pass & 1];
      // (its readers of two passes ago have been through the barrier of the last)
      for (int i = tid; i < kBins; i += kThreads) hist[i] = 0;
      __syncthreads();
      for (int i = tid; i < n; i += kThreads) {
        const uint32_t key = key_at(i);
        if (above == 32 || key >> above == prefix >> above) atomicAdd(&hist[(key >> shift) & mask], 1u);
      }
      sync_all();
      // Bins from the top, kPer a thread, summed over the cluster.
      constexpr int kPer = kBins / kThreads;
      const int low = kBins - kPer * (tid + 1);
      uint32_t bin[kPer] = {};  // of bins low + kPer - 1 down to low
#pragma unroll 8
      for (int k = 0; k < cluster; ++k) {
        const uint32_t* h = (cluster > 1 ? cl.map_shared_rank(hist, k) : hist) + low;
#pragma unroll
        for (int i = 0; i < kPer; i += 2) {
          const uint2 v = *reinterpret_cast<const uint2*>(h + i);
          bin[kPer - 1 - i] += v.x;
          bin[kPer - 2 - i] += v.y;
        }
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
      uint32_t before = incl - mine;
      for (int w = 0; w < warp; ++w) before += sh.warp_sum[w];
      if (before < rest && rest <= before + mine) {  // one thread: the digit is in its bins
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
          if (before < rest && rest <= before + bin[i]) {
            sh.digit = uint32_t(low + kPer - 1 - i);
            sh.rest = rest - before;
          }
          before += bin[i];
        }
      }
      __syncthreads();
      prefix |= sh.digit << shift;
      rest = sh.rest;
    }
    const uint32_t threshold = prefix;  // rest: so many of the keys equal to it stay

    // ---- how many stay of the slices before ----
    // Warps take whole words of 32 candidates in order, a contiguous run each.
    const int words = (n + 31) / 32;
    const int w_per = (words + kWarps - 1) / kWarps;
    const int w0 = min(words, warp * w_per), w1 = min(words, w0 + w_per);
    uint32_t gt = 0, eq = 0;
    for (int w = w0; w < w1; ++w) {
      const int i = 32 * w + lane;
      const uint32_t key = i < n ? key_at(i) : 0u;
      gt += __popc(__ballot_sync(0xffffffffu, i < n && key > threshold));
      eq += __popc(__ballot_sync(0xffffffffu, i < n && key == threshold));
    }
    if (lane == 0) {
      sh.warp_sum[warp] = gt;
      sh.warp_eq[warp] = eq;
    }
    __syncthreads();
    if (tid == 0) {
      uint32_t a = 0, e = 0;
      for (int w = 0; w < kWarps; ++w) {
        a += sh.warp_sum[w];
        e += sh.warp_eq[w];
      }
      sh.count_gt = a;
      sh.count_eq = e;
    }
    sync_all();
    uint32_t gt_before = 0, eq_before = 0;
    for (int k = 0; k < rank; ++k) {
      gt_before += *cl.map_shared_rank(&sh.count_gt, k);
      eq_before += *cl.map_shared_rank(&sh.count_eq, k);
    }
    for (int w = 0; w < warp; ++w) {
      gt_before += sh.warp_sum[w];
      eq_before += sh.warp_eq[w];
    }
    // ---- the list, in order ----
    for (int w = w0; w < w1; ++w) {
      const int i = 32 * w + lane;
      const uint32_t key = i < n ? key_at(i) : 0u;
      const bool above = i < n && key > threshold, same = i < n && key == threshold;
      const uint32_t gts = __ballot_sync(0xffffffffu, above), eqs = __ballot_sync(0xffffffffu, same);
      const uint32_t below = (1u << lane) - 1u;
      const uint32_t eq_rank = eq_before + __popc(eqs & below);
      if (above || (same && eq_rank < rest))
        list[gt_before + __popc(gts & below) + min(eq_rank, rest)] = f + s0 + i;
      gt_before += __popc(gts);
      eq_before += __popc(eqs);
    }
    sync_all();
  }

  // ---- move ----
  // Rows q = 0 .. c + r - 1 go to token f + q: the listed ones, then the recent.
  // bf16: a warp moves a row at a time, K in its first half and V in its
  // second, 16 bytes a lane; E4M3 rows are half as long and a warp moves two.
  constexpr int kVecs = F8 ? 8 : 16;            // 16-byte vectors of a row of K or of V
  constexpr int kLanes = 2 * kVecs;             // lanes a row
  constexpr int kSub = 32 / kLanes;             // rows that a warp moves at a time
  constexpr int kDeep = 8;                      // times, all in flight
  constexpr int kWarpRows = kSub * kDeep;       // 8 or 16
  constexpr int kRows = kWarpRows * kWarps;   // rows of a CTA's round
  const int total = c + r;
  const int sub = lane / kLanes, in_row = lane % kLanes;
  uint4* const pool = reinterpret_cast<uint4*>(in_row < kVecs ? p.k_cache : p.v_cache);
  const int vec = in_row % kVecs;
  // Lane l < kWarpRows sees to row l of the warp's in a round: the token that it
  // comes from is read two rounds ahead, the pages one, so that neither the row
  // copies nor the barrier wait for a table.
  const int64_t round_rows = int64_t(cluster) * kRows;
  const int64_t mine = int64_t(rank) * kRows + warp * kWarpRows + lane;
  auto token_of = [&](int64_t q) {  // -1: no row
    return lane >= kWarpRows || q >= total ? -1 : q < c ? __ldcg(list + q) : L - r + int(q - c);
  };
  auto lowest_of = [&](int64_t base) {  // of a round's sources
    return base >= total ? 0 : base < c ? __ldcg(list + base) : L - r + int(base - c);
  };
  struct Pages {
    int src, dst;
  };
  auto pages_of = [&](int64_t q, int from) {
    if (from < 0) return Pages{0, 0};
    return Pages{__ldg(table + from / kPage), __ldg(table + (f + int(q)) / kPage)};
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
    src = row_of(pg.src, from);
    dst = row_of(pg.dst, to);
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
    uint4 v[kDeep];
#pragma unroll
    for (int i = 0; i < kDeep; ++i) {
      const int64_t s = __shfl_sync(0xffffffffu, src, i * kSub + sub);
      if (s >= 0) v[i] = __ldcs(pool + s * kVecs + vec);
    }
    float score = 0.f;
    uint8_t ks = 0, vs = 0;
    if (src >= 0) {
      score = __ldcg(p.scores + src);
      if constexpr (F8) {
        ks = __ldcg(p.k_scale + src);
        vs = __ldcg(p.v_scale + src);
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
      p.scores[dst] = score;
      if constexpr (F8) {
        p.k_scale[dst] = ks;
        p.v_scale[dst] = vs;
      }
    }
  }
  if (cluster > 1 && total > 0) cluster_wait();
}

int list_stride(const pkv_desc& d) { return d.max_blocks_per_seq * kPage; }

using Kernel = void (*)(EvictArgs, int, int);

cudaLaunchConfig_t config(cudaLaunchAttribute (&attr)[2], cudaStream_t stream, int64_t items, int cluster, bool big) {
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = unsigned(cluster);
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(items * cluster));
  cfg.blockDim = dim3(unsigned(big ? kBigThreads : kSmallThreads));
  cfg.dynamicSmemBytes = big ? sizeof(EvictShared<kBigThreads>) : sizeof(EvictShared<kSmallThreads>);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cfg;
}

// How many clusters of 1, 2, 4, 8 and 16 CTAs of 1024 threads run at once on a
// device, asked once (a cluster stays within a GPC).
template <bool F8>
const int* resident_clusters(int device) {
  static int most[64][5];
  static bool done[64] = {};
  if (device < 0 || device >= 64) return nullptr;
  if (!done[device]) {
    const Kernel big = pkv_evict_kernel<F8, kBigThreads>, small = pkv_evict_kernel<F8, kSmallThreads>;
    if (cudaFuncSetAttribute(big, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             int(sizeof(EvictShared<kBigThreads>))) != cudaSuccess ||
        cudaFuncSetAttribute(small, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             int(sizeof(EvictShared<kSmallThreads>))) != cudaSuccess ||
        cudaFuncSetAttribute(big, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess) {
      cudaGetLastError();
      return nullptr;
    }
    for (int i = 0; i < 5; ++i) {
      cudaLaunchAttribute attr[2];
      cudaLaunchConfig_t cfg = config(attr, nullptr, 1, 1 << i, true);
      cfg.numAttrs = 1;
      int n = 0;
      if (cudaOccupancyMaxActiveClusters(&n, big, &cfg) != cudaSuccess) {
        cudaGetLastError();
        n = 0;  // a size that this device cannot run
      }
      most[device][i] = n;
    }
    done[device] = true;
  }
  return most[device];
}

// CTAs of 1024 threads an item: as many as let all items run at once, none for
// less than 512 tokens of the widest sequence.  0: items or tables too small for
// them, a CTA of 256 threads each.
int cluster_size(const int* most, const pkv_desc& d, int64_t items) {
  const int64_t tokens = int64_t(d.max_blocks_per_seq) * kPage;
  if (items > most[0] || tokens < 4 * 512) return 0;
  int n = 1;
  for (int i = 1; i < 5; ++i)
    if (items <= most[i] && tokens >= int64_t(512) << i) n = 1 << i;
  return n;
}

}  // namespace

size_t evict_workspace_bytes(const pkv_desc& d, int32_t num_seqs) {
  return align_up(sizeof(int32_t) * size_t(num_seqs) * size_t(d.num_kv_heads) * size_t(list_stride(d)), 256);
}

int launch_evict(const LaunchCtx& ctx, const EvictArgs& a, bool fp8) {
  if (a.workspace_bytes < evict_workspace_bytes(a.desc, a.num_seqs)) return PKV_ERR_WORKSPACE;
  const int* most = fp8 ? resident_clusters<true>(ctx.dev->device) : resident_clusters<false>(ctx.dev->device);
  if (!most) return PKV_ERR_LAUNCH;
  const int64_t items = int64_t(a.num_seqs) * a.desc.num_kv_heads;
  if (items * kMaxCluster > INT32_MAX) return PKV_ERR_RANGE;
  const int n = cluster_size(most, a.desc, items), cluster = n ? n : 1;
  const Kernel kernel = n ? (fp8 ? pkv_evict_kernel<true, kBigThreads> : pkv_evict_kernel<false, kBigThreads>)
                          : (fp8 ? pkv_evict_kernel<true, kSmallThreads> : pkv_evict_kernel<false, kSmallThreads>);
  cudaLaunchAttribute attr[2];
  const cudaLaunchConfig_t cfg = config(attr, ctx.stream, items, cluster, n != 0);
  TraceScope ts(ctx.stream, PKV_K_EVICT);
  cudaLaunchKernelEx(&cfg, kernel, a, cluster, list_stride(a.desc));
  return ts.done();
}

}  // namespace pkv
