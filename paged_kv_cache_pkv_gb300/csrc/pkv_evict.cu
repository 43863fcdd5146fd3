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
//     wide, before any of them is written, and nothing else has to wait.
//
// What bounds it: bytes, a row read and written once (2 x 512 bytes a token
// and head on bf16 pages); on few tokens the chain of steps 1 to 3.
#include <cooperative_groups.h>

#include "pkv_common.cuh"
#include "pkv_internal.h"

namespace pkv {
namespace {

namespace cg = cooperative_groups;

constexpr int kEvThreads = 256;
constexpr int kEvWarps = kEvThreads / 32;
constexpr int kKeys = 8192;   // keys of a slice held in shared memory
constexpr int kBins = 2048;
constexpr int kMaxCluster = 16;

struct EvictShared {
  uint32_t hist[2][kBins];
  uint32_t keys[kKeys];
  uint32_t warp_sum[kEvWarps], warp_eq[kEvWarps];
  uint32_t digit, rest;         // of the last selection pass
  uint32_t count_gt, count_eq;  // of this CTA's slice
};

// A key that orders like the score: NaN as -infinity, -0 as 0.
__device__ __forceinline__ uint32_t order_key(float x) {
  if (x != x) x = -INFINITY;
  const uint32_t u = __float_as_uint(x + 0.0f);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

template <bool F8>
__global__ void __launch_bounds__(kEvThreads, 4) pkv_evict_kernel(const EvictArgs p, int cluster, int list_stride) {
  extern __shared__ __align__(16) uint8_t smem_raw[];
  EvictShared& sh = *reinterpret_cast<EvictShared*>(smem_raw);
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
    for (int i = tid; i < min(n, kKeys); i += kEvThreads) sh.keys[i] = read_key(i);

    // ---- the c-th largest key, digit by digit ----
    uint32_t prefix = 0, rest = uint32_t(c);
#pragma unroll 1
    for (int pass = 0; pass < 3; ++pass) {
      const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
      const int above = pass == 0 ? 32 : pass == 1 ? 21 : 10;  // bits from here on are known
      const uint32_t mask = pass == 2 ? 1023u : 2047u;
      uint32_t* hist = sh.hist[pass & 1];
      // (its readers of two passes ago have been through the barrier of the last)
      for (int i = tid; i < kBins; i += kEvThreads) hist[i] = 0;
      __syncthreads();
      for (int i = tid; i < n; i += kEvThreads) {
        const uint32_t key = key_at(i);
        if (above == 32 || key >> above == prefix >> above) atomicAdd(&hist[(key >> shift) & mask], 1u);
      }
      sync_all();
      // Bins from the top: thread t has bins 2047 - 8t .. 2040 - 8t, summed over the cluster.
      uint32_t bin[8] = {};
      for (int k = 0; k < cluster; ++k) {
        const uint32_t* h = cluster > 1 ? cl.map_shared_rank(hist, k) : hist;
        const uint4 hi = *reinterpret_cast<const uint4*>(h + kBins - 8 - 8 * tid + 4);
        const uint4 lo = *reinterpret_cast<const uint4*>(h + kBins - 8 - 8 * tid);
        bin[0] += hi.w, bin[1] += hi.z, bin[2] += hi.y, bin[3] += hi.x;
        bin[4] += lo.w, bin[5] += lo.z, bin[6] += lo.y, bin[7] += lo.x;
      }
      uint32_t mine = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) mine += bin[i];
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
        for (int i = 0; i < 8; ++i) {
          if (before < rest && rest <= before + bin[i]) {
            sh.digit = uint32_t(kBins - 1 - 8 * tid - i);
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
    const int w_per = (words + kEvWarps - 1) / kEvWarps;
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
      for (int w = 0; w < kEvWarps; ++w) {
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
  constexpr int kRows = kWarpRows * kEvWarps;   // rows of a CTA's round
  const int total = c + r;
  const int sub = lane / kLanes, in_row = lane % kLanes;
  uint4* const pool = reinterpret_cast<uint4*>(in_row < kVecs ? p.k_cache : p.v_cache);
  const int vec = in_row % kVecs;
  // lane l < kWarpRows: source and destination of the warp's row l of a round
  auto places = [&](int64_t q, int64_t& src, int64_t& dst) {
    src = dst = -1;
    if (lane >= kWarpRows || q >= total) return;
    const int to = f + int(q);
    const int from = q < c ? __ldcg(list + q) : L - r + int(q - c);
    if (from == to) return;  // in its place
    const int ps = page_of(from), pd = page_of(to);
    if (ps < 0 || pd < 0) {
      flag_status(p.status, PKV_STATUS_BAD_BLOCK);
      return;
    }
    src = row_of(ps, from);
    dst = row_of(pd, to);
  };
  const int64_t round_rows = int64_t(cluster) * kRows;
  int64_t src, dst;
  const int64_t mine = int64_t(rank) * kRows + warp * kWarpRows + lane;
  places(mine, src, dst);
  for (int64_t base = 0; base < total; base += round_rows) {
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
    int64_t next_src, next_dst;
    places(base + round_rows + mine, next_src, next_dst);
    sync_all();  // every row of the round is in registers
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
    src = next_src;
    dst = next_dst;
  }
}

// CTAs an item: as many as fill the GPU twice, none with less than 256 tokens
// of the widest sequence.
int cluster_size(const DeviceInfo& dev, const pkv_desc& d, int64_t items) {
  int n = 1;
  while (n < kMaxCluster && items * n * 2 <= 2 * dev.sm_count &&
         int64_t(d.max_blocks_per_seq) * kPage >= int64_t(n) * 2 * 256)
    n *= 2;
  return n;
}

int list_stride(const pkv_desc& d) { return d.max_blocks_per_seq * kPage; }

template <bool F8>
int ensure_attr(int device) {
  static bool done[64] = {};
  if (device < 0 || device >= 64) return PKV_ERR_DEVICE;
  if (!done[device]) {
    if (cudaFuncSetAttribute(pkv_evict_kernel<F8>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             int(sizeof(EvictShared))) != cudaSuccess ||
        cudaFuncSetAttribute(pkv_evict_kernel<F8>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) !=
            cudaSuccess) {
      cudaGetLastError();
      return PKV_ERR_LAUNCH;
    }
    done[device] = true;
  }
  return PKV_OK;
}

}  // namespace

size_t evict_workspace_bytes(const pkv_desc& d, int32_t num_seqs) {
  return align_up(sizeof(int32_t) * size_t(num_seqs) * size_t(d.num_kv_heads) * size_t(list_stride(d)), 256);
}

int launch_evict(const LaunchCtx& ctx, const EvictArgs& a, bool fp8) {
  if (a.workspace_bytes < evict_workspace_bytes(a.desc, a.num_seqs)) return PKV_ERR_WORKSPACE;
  if (int e = fp8 ? ensure_attr<true>(ctx.dev->device) : ensure_attr<false>(ctx.dev->device)) return e;
  const int64_t items = int64_t(a.num_seqs) * a.desc.num_kv_heads;
  const int cluster = cluster_size(*ctx.dev, a.desc, items);
  if (items * cluster > INT32_MAX) return PKV_ERR_RANGE;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(items * cluster));
  cfg.blockDim = dim3(kEvThreads);
  cfg.dynamicSmemBytes = sizeof(EvictShared);
  cfg.stream = ctx.stream;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  TraceScope ts(ctx.stream, PKV_K_EVICT);
  cudaLaunchKernelEx(&cfg, fp8 ? pkv_evict_kernel<true> : pkv_evict_kernel<false>, a, cluster, list_stride(a.desc));
  return ts.done();
}

}  // namespace pkv
