// pkv_latent_merge.cuh -- the partials that latent attention leaves for a tile
// cut between CTAs, and the kernel that joins them.
#pragma once

#include "pkv_latent.cuh"

namespace pkv {
namespace {

// A partial: O in the order in which the softmax warps hold it, [4 blocks of
// 128 dims][4 warps][N/4 groups of rows][32 dims][4 rows], then m [N], l [N].
constexpr int kLtPartialFloats = 64 * kLatentDim + 2 * 64;

// Joins the pieces of the cut tiles.  With weights w_i = 2^(m_i - M), M the
// largest reference of a piece that saw a key:
//   out = sum w_i O_i / sum w_i l_i.
// CTA c's share ends inside at most one tile, whose pieces are c's second
// partial and the first partials of c + 1 .. last.  A warp joins four rows
// (a float4 a lane of the partials' layout).  Most tiles have two or three
// pieces: there the warps of blocks (c, *) take four rows and four or eight
// times 32 dims each.  A long sequence alone is one tile with a piece a CTA:
// there the blocks of all its CTAs take units of four rows and 32 dims, and a
// block's warps share the pieces.  What bounds it: reads that wait for one
// another (the join record, then O; O does not wait for the weights), at 2000
// cycles each while all SMs read at once, and fetching its own instructions, so
// its loops are rolled and it divides once.  Registers hold what is under way:
// 80 of them and three blocks an SM (64 decode rows of 128 heads 61.9 us for the
// call; with 64 and four blocks 63.4, with 128 and two 64.6).  Asynchronous
// copies into shared memory in their place took 3 us longer, and bulk copies into
// a ring that eight warps add up 10: fewer warps that add, and blocks that find
// no room beside the main kernel's CTAs before these end.
constexpr int kLtMergeThreads = 256;
constexpr int kLtMergeWarps = kLtMergeThreads / 32;
constexpr int kLtFewPieces = 6;
constexpr int kLtBatch = 8;  // pieces that a warp has under way

// Batches of four times 32 dims that a warp goes through for its rows, and the
// blocks a CTA of the main kernel that makes.
constexpr int lt_merge_batches(int N) { return N >= 64 ? 2 : 1; }
constexpr int lt_merge_blocks(int N) { return N / kLtMergeWarps / lt_merge_batches(N); }

__device__ __forceinline__ float4 f4(float v) { return make_float4(v, v, v, v); }
// a * x + y where a is not 0, else y: an O that saw no key was not written
__device__ __forceinline__ float fma_seen(float a, float x, float y) { return a != 0.f ? fmaf(a, x, y) : y; }
__device__ __forceinline__ float4 fma_seen(const float4& a, const float4& x, const float4& y) {
  return make_float4(fma_seen(a.x, x.x, y.x), fma_seen(a.y, x.y, y.y), fma_seen(a.z, x.z, y.z),
                     fma_seen(a.w, x.w, y.w));
}
__device__ __forceinline__ float4 f4_max(const float4& a, const float4& b) {
  return make_float4(fmaxf(a.x, b.x), fmaxf(a.y, b.y), fmaxf(a.z, b.z), fmaxf(a.w, b.w));
}
// references, those of pieces that saw no key put below all others
__device__ __forceinline__ float4 f4_seen(const float4& m, const float4& l) {
  constexpr float none = -INFINITY;
  return make_float4(l.x != 0.f ? m.x : none, l.y != 0.f ? m.y : none, l.z != 0.f ? m.z : none,
                     l.w != 0.f ? m.w : none);
}
__device__ __forceinline__ float weight(float m, float M) { return m == -INFINITY ? 0.f : ex2(m - M); }
__device__ __forceinline__ float4 f4_weight(const float4& m, const float4& M) {
  return make_float4(weight(m.x, M.x), weight(m.y, M.y), weight(m.z, M.z), weight(m.w, M.w));
}
__device__ __forceinline__ float4 f4_shfl_xor(const float4& v, int o) {
  return make_float4(__shfl_xor_sync(0xffffffffu, v.x, o), __shfl_xor_sync(0xffffffffu, v.y, o),
                     __shfl_xor_sync(0xffffffffu, v.z, o), __shfl_xor_sync(0xffffffffu, v.w, o));
}

// PAIR: the parts are pairs of CTAs with tiles of N = 128 rows.  CTA i of a pair
// holds dims 256 i .. of all rows, and the references and sums of rows 64 i ..
template <int N, bool PAIR>
__global__ void __launch_bounds__(kLtMergeThreads, 3) pkv_latent_merge_kernel(const LatentParams p) {
  constexpr int kParts = PAIR ? 2 : 1;    // partials of a piece
  constexpr int kRows = N / kParts;       // rows whose m and l are in one
  constexpr int kDq = 16 / kParts;        // groups of 32 dims in one
  constexpr int kO = N * kLatentDim / kParts;
  __shared__ float4 s_max[kLtMergeWarps], s_sum[kLtMergeWarps];
  __shared__ float4 s_w[kLtMergeThreads];  // of a piece; the grid has fewer CTAs
  __shared__ float4 s_acc[kLtMergeWarps][32];
  griddep_wait();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  // piece i of the tile that c's share ends inside, its partial of CTA `of`
  auto part = [&](int c, int i, int of) {
    const size_t cta = size_t(c + i) * kParts + of;
    return p.partials + (cta * 2 + (i == 0 ? 1 : 0)) * kLtPartialFloats;
  };
  auto m_of = [&](int c, int i, int rq) {
    return __ldcg(reinterpret_cast<const float4*>(part(c, i, rq * 4 / kRows) + kO) + rq % (kRows / 4));
  };
  auto l_of = [&](int c, int i, int rq) {
    return __ldcg(reinterpret_cast<const float4*>(part(c, i, rq * 4 / kRows) + kO + kRows) + rq % (kRows / 4));
  };
  auto o_of = [&](int c, int i, int rq, int dq) {  // 32 dims dq, rows 4 rq .. + 3
    return __ldcg(reinterpret_cast<const float4*>(part(c, i, dq / kDq)) + (dq % kDq * (N / 4) + rq) * 32 + lane);
  };
  // rows 4 rq .. + 3 of a tile, dim 32 dq + lane of each; even lanes store a
  // pair of dims of the first of two rows, odd lanes of the second
  auto put = [&](const int4& join, int rq, int dq, const float4& a) {
    const float v[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int e = 0; e < 4; e += 2) {
      const float other = __shfl_xor_sync(0xffffffffu, (lane & 1) ? v[e] : v[e + 1], 1);
      const int r = rq * 4 + e + (lane & 1);
      if (r < join.y)
        *(reinterpret_cast<uint32_t*>(p.out + size_t(join.x + r) * kLatentDim + dq * 32) + (lane >> 1)) =
            (lane & 1) ? pack_bf16x2(other, v[e + 1]) : pack_bf16x2(v[e], other);
    }
  };
  const int4 own = __ldcg(p.joins + blockIdx.x);
  const bool own_many = own.y > 0 && own.z - int(blockIdx.x) + 1 > kLtFewPieces;
  if (own.y > 0 && !own_many) {
    constexpr int kWarps = 4 / lt_merge_batches(N);  // that share four rows
    constexpr int kGroups = kLtMergeWarps / kWarps;  // of four rows, a block
    const int c = blockIdx.x, group = warp / kWarps, first = int(blockIdx.y) * kGroups;
    const int rq = first + group, pieces = own.z - c + 1;
    const bool work = rq * 4 < own.y;
    float4 acc[4], o[4];
    auto read = [&](int b) {  // (a cut tile has two pieces at least)
      const int d0 = (warp % kWarps * lt_merge_batches(N) + b) * 4;
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[e] = o_of(c, 0, rq, d0 + e);
#pragma unroll
      for (int e = 0; e < 4; ++e) o[e] = o_of(c, 1, rq, d0 + e);
    };
    if (work) read(0);
    if (warp == 0) {
      // lane (g, k): piece k's weight for the block's rows 4 g .. + 3, divided
      // by the rows' sums; a warp for all, since every warp for its own rows
      // takes as long as the reads
      const int g = lane >> 3, k = lane & 7;
      float4 l = f4(0.f), m = f4(-INFINITY);
      if (g < kGroups && k < pieces) {
        l = l_of(c, k, first + g);
        m = m_of(c, k, first + g);
      }
      m = f4_seen(m, l);
      float4 M = m;
#pragma unroll
      for (int d = 4; d >= 1; d >>= 1) M = f4_max(M, f4_shfl_xor(M, d));
      const float4 w = f4_weight(m, M);
      float4 sum = make_float4(w.x * l.x, w.y * l.y, w.z * l.z, w.w * l.w);
#pragma unroll
      for (int d = 4; d >= 1; d >>= 1) {
        const float4 x = f4_shfl_xor(sum, d);
        sum = make_float4(sum.x + x.x, sum.y + x.y, sum.z + x.z, sum.w + x.w);
      }
      s_w[lane] = make_float4(w.x / sum.x, w.y / sum.y, w.z / sum.z, w.w / sum.w);
    }
    __syncthreads();
    if (work) {
#pragma unroll 1
      for (int b = 0; b < lt_merge_batches(N); ++b) {
        if (b > 0) read(b);
        float4 wk = s_w[group * 8];
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[e] = fma_seen(wk, acc[e], f4(0.f));
#pragma unroll 1
        for (int q = 1;;) {
          wk = s_w[group * 8 + q];
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[e] = fma_seen(wk, o[e], acc[e]);
          if (++q >= pieces) break;
          const int d0 = (warp % kWarps * lt_merge_batches(N) + b) * 4;
#pragma unroll
          for (int e = 0; e < 4; ++e) o[e] = o_of(c, q, rq, d0 + e);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) put(own, rq, (warp % kWarps * lt_merge_batches(N) + b) * 4 + e, acc[e]);
      }
    }
  }
  for (int which = 0; which < 2; ++which) {
    const int c = which == 0 ? own.w : own_many ? int(blockIdx.x) : -1;
    if (c < 0) continue;
    const int4 join = __ldcg(p.joins + c);
    const int pieces = join.z - c + 1;
    if (pieces <= kLtFewPieces) continue;
    const int team = pieces * gridDim.y;
    for (int u = (blockIdx.x - c) * gridDim.y + blockIdx.y; u < (join.y + 3) / 4 * 16; u += team) {
      const int rq = u >> 4, dq = u & 15;
      float4 o[kLtBatch];
      auto read = [&](int first) {
#pragma unroll
        for (int i = 0; i < kLtBatch; ++i) {
          const int k = first + i * kLtMergeWarps;
          if (k < pieces) o[i] = o_of(c, k, rq, dq);
        }
      };
      read(warp);
      float4 l = f4(0.f), m = f4(-INFINITY);
      if (tid < pieces) {
        l = l_of(c, tid, rq);
        m = f4_seen(m_of(c, tid, rq), l);
      }
      float4 M = m;
#pragma unroll
      for (int d = 16; d >= 1; d >>= 1) M = f4_max(M, f4_shfl_xor(M, d));
      if (lane == 0) s_max[warp] = M;
      __syncthreads();
      for (int w = 0; w < kLtMergeWarps; ++w) M = f4_max(M, s_max[w]);
      const float4 w = f4_weight(m, M);
      s_w[tid] = w;
      float4 sum = make_float4(w.x * l.x, w.y * l.y, w.z * l.z, w.w * l.w);
#pragma unroll
      for (int d = 16; d >= 1; d >>= 1) sum = fma_seen(f4(1.f), f4_shfl_xor(sum, d), sum);
      if (lane == 0) s_sum[warp] = sum;
      __syncthreads();
      float4 acc = f4(0.f);
      for (int first = warp; first < pieces; first += kLtBatch * kLtMergeWarps) {
        if (first > warp) read(first);
#pragma unroll
        for (int i = 0; i < kLtBatch; ++i) {
          const int k = first + i * kLtMergeWarps;
          if (k < pieces) acc = fma_seen(s_w[k], o[i], acc);
        }
      }
      s_acc[warp][lane] = acc;
      __syncthreads();
      if (warp == 0) {
        sum = s_sum[0];
        for (int i = 1; i < kLtMergeWarps; ++i) {
          acc = fma_seen(f4(1.f), s_acc[i][lane], acc);
          sum = fma_seen(f4(1.f), s_sum[i], sum);
        }
        put(join, rq, dq, make_float4(acc.x / sum.x, acc.y / sum.y, acc.z / sum.z, acc.w / sum.w));
      }
      __syncthreads();
    }
  }
  // Not before the partials are read: the workspace is the caller's again
  // behind this call on the stream, and a kernel let in, if it is not one of
  // this library's, may write to it before it waits (earlier, a call of this
  // kind behind this one gains 2-4 us).  A block's first thread to say so
  // speaks for all of them, hence the barrier.
  __syncthreads();
  griddep_launch_dependents();
}

}  // namespace
}  // namespace pkv
