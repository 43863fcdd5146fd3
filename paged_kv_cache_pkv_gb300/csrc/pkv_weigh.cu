// pkv_weigh.cu -- accumulated attention weights: for every cached token and kv
// head the sum of the softmax weights that this step's query rows give it,
// added to paged scores.
//
//   lse[j, h] = log sum_{k <= pos j} exp(scale q[j, h] . K[k])
//   w[k]      = sum_{j, h: k <= pos j} exp(scale q[j, h] . K[k] - lse[j, h])
//
// A weight needs its row's sum over all keys first, so there are two passes:
// one over the keys of each row, one over the rows of each key.  Both work in
// the log2 domain (exp2), sums in fp32.
#include <cmath>

#include <cuda_fp8.h>

#include "pkv_common.cuh"
#include "pkv_internal.h"

namespace pkv {
namespace {

constexpr int kWeighThreads = 128;

struct Sequence {
  int q0, n, L;
};

// Sequence b's rows and length; false (and flagged) where they do not fit.
__device__ __forceinline__ bool sequence_of(const WeighArgs& p, int b, Sequence& s) {
  const int q0 = __ldg(p.query_start_loc + b), q1 = __ldg(p.query_start_loc + b + 1), L = __ldg(p.seq_lens + b);
  s = {q0, 0, 0};
  if (q0 < 0 || q1 < q0 || q1 > p.num_tokens || L < 0 || q1 - q0 > L ||
      (L > 0 && (L - 1) / kPage >= p.desc.max_blocks_per_seq) || (b == 0 && q0 != 0) || q1 - q0 > p.max_rows) {
    flag_status(p.status, PKV_STATUS_BAD_QUERY);
    return false;
  }
  s.n = q1 - q0;
  s.L = L;
  return true;
}

template <bool F8>
__device__ __forceinline__ float dot(const WeighArgs& p, const float* q, int64_t row) {
  float acc = 0.f;
  if constexpr (F8) {
    const uint8_t* k = static_cast<const uint8_t*>(p.k_cache) + row * kHeadDim;
    for (int d = 0; d < kHeadDim; ++d) {
      __nv_fp8_e4m3 c;
      c.__x = k[d];
      acc = fmaf(q[d], float(c), acc);
    }
    return acc * __uint_as_float(uint32_t(p.k_scale[row]) << 23);
  } else {
    const uint32_t* k = static_cast<const uint32_t*>(p.k_cache) + row * (kHeadDim / 2);
    for (int d = 0; d < kHeadDim / 2; ++d) {
      acc = fmaf(q[2 * d], bf_lo(k[d]), acc);
      acc = fmaf(q[2 * d + 1], bf_hi(k[d]), acc);
    }
    return acc;
  }
}

__device__ __forceinline__ int64_t key_row(const WeighArgs& p, int b, int g, int k) {
  int id = __ldg(p.block_tables + int64_t(b) * p.desc.max_blocks_per_seq + k / kPage);
  if (id < 0 || id >= p.desc.num_blocks) {
    flag_status(p.status, PKV_STATUS_BAD_BLOCK);
    return -1;
  }
  return (int64_t(id) * p.desc.num_kv_heads + g) * kPage + k % kPage;
}

// One warp a (query row, head): lanes take keys in turn.
template <bool F8>
__global__ void __launch_bounds__(kWeighThreads) pkv_weigh_sums_kernel(const WeighArgs p) {
  griddep_wait();
  __shared__ float sq[kWeighThreads / 32][kHeadDim];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int Hq = p.desc.num_q_heads, G = Hq / p.desc.num_kv_heads;
  const int64_t item = int64_t(blockIdx.x) * (kWeighThreads / 32) + warp;
  if (item >= int64_t(p.num_tokens) * Hq) return;
  const int t = int(item / Hq), h = int(item % Hq);
  int lo = 0, hi = p.num_seqs;  // last b with query_start_loc[b] <= t
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (__ldg(p.query_start_loc + mid) <= t) lo = mid;
    else hi = mid;
  }
  Sequence s;
  if (!sequence_of(p, lo, s) || t >= s.q0 + s.n) return;
  for (int d = lane; d < kHeadDim; d += 32) {
    const uint16_t x = p.q[item * kHeadDim + d];
    sq[warp][d] = __uint_as_float(uint32_t(x) << 16);
  }
  __syncwarp();
  const int last = s.L - s.n + (t - s.q0);
  float m = -INFINITY, l = 0.f;
  for (int k = lane; k <= last; k += 32) {
    const int64_t row = key_row(p, lo, h / G, k);
    const float x = row < 0 ? 0.f : dot<F8>(p, sq[warp], row) * p.qscale;
    const float mn = fmaxf(m, x);
    l = l * ex2(m - mn) + ex2(x - mn);
    m = mn;
  }
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) {
    const float mo = __shfl_xor_sync(0xffffffffu, m, o), lo_ = __shfl_xor_sync(0xffffffffu, l, o);
    const float mn = fmaxf(m, mo);
    l = (m == -INFINITY ? 0.f : l * ex2(m - mn)) + (mo == -INFINITY ? 0.f : lo_ * ex2(mo - mn));
    m = mn;
  }
  if (lane == 0) static_cast<float*>(p.workspace)[item] = m + __log2f(l);
}

// One warp a (sequence, kv head, key): lanes take rows in turn.
template <bool F8>
__global__ void __launch_bounds__(kWeighThreads) pkv_weigh_add_kernel(const WeighArgs p) {
  griddep_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int Hq = p.desc.num_q_heads, Hkv = p.desc.num_kv_heads, G = Hq / Hkv;
  const int b = blockIdx.y / Hkv, g = blockIdx.y % Hkv;
  Sequence s;
  if (!sequence_of(p, b, s) || s.n == 0) return;
  const float* lse = static_cast<const float*>(p.workspace);
  const int first = p.first ? max(0, __ldg(p.first + b)) : 0;
  const int scored = p.scored ? __ldg(p.scored + b) : s.L - s.n;
  for (int k = first + blockIdx.x * (kWeighThreads / 32) + warp; k < s.L; k += gridDim.x * (kWeighThreads / 32)) {
    const int64_t row = key_row(p, b, g, k);
    if (row < 0) continue;
    const int j0 = max(0, k - (s.L - s.n));
    float w = 0.f;
    for (int i = j0 * G + lane; i < s.n * G; i += 32) {
      const int64_t item = int64_t(s.q0 + i / G) * Hq + g * G + i % G;
      float q[kHeadDim];
      for (int d = 0; d < kHeadDim; ++d) q[d] = __uint_as_float(uint32_t(p.q[item * kHeadDim + d]) << 16);
      w += ex2(dot<F8>(p, q, row) * p.qscale - lse[item]);
    }
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) w += __shfl_xor_sync(0xffffffffu, w, o);
    if (lane == 0) p.scores[row] = (k < scored && p.decay != 0.f ? p.decay * p.scores[row] : 0.f) + w;
  }
}

template <class Kernel>
int launch(const LaunchCtx& ctx, Kernel kernel, dim3 grid, const WeighArgs& a) {
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(kWeighThreads);
  cfg.stream = ctx.stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  TraceScope ts(ctx.stream, PKV_K_WEIGH);
  cudaLaunchKernelEx(&cfg, kernel, a);
  return ts.done();
}

}  // namespace

size_t weigh_workspace_bytes(const DeviceInfo&, const pkv_desc& d, int32_t, int32_t num_tokens, int32_t, int64_t) {
  return align_up(sizeof(float) * size_t(num_tokens) * size_t(d.num_q_heads), 256);
}

int launch_weigh(const LaunchCtx& ctx, const WeighArgs& a, bool fp8) {
  if (a.workspace_bytes < weigh_workspace_bytes(*ctx.dev, a.desc, a.num_seqs, a.num_tokens, a.max_rows, a.num_keys))
    return PKV_ERR_WORKSPACE;
  const int64_t warps = int64_t(a.num_tokens) * a.desc.num_q_heads;
  const int64_t pairs = int64_t(a.num_seqs) * a.desc.num_kv_heads;
  if (pairs > 65535) return PKV_ERR_RANGE;
  constexpr int per = kWeighThreads / 32;
  if (int e = launch(ctx, fp8 ? pkv_weigh_sums_kernel<true> : pkv_weigh_sums_kernel<false>,
                     dim3(unsigned((warps + per - 1) / per)), a))
    return e;
  return launch(ctx, fp8 ? pkv_weigh_add_kernel<true> : pkv_weigh_add_kernel<false>, dim3(64, unsigned(pairs)), a);
}

}  // namespace pkv
