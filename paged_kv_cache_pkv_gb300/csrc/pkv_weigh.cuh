// pkv_weigh.cuh -- what the kernels of accumulated attention weights share: a
// sequence's place in the batch and the way its units of work are counted.
#pragma once

#include "pkv_common.cuh"
#include "pkv_internal.h"

namespace pkv {

// Running maxima start here, below any score, instead of at -infinity, whose
// difference with itself is not a number; a masked score, -infinity, adds
// exp2(-inf) = 0.
constexpr float kWeighNoScore = -3.402823466e38f;

struct WeighSequence {
  int q0, n, L;
};

// Sequence b's first row, rows and length; false where they do not fit.  Any
// int32 may stand there.
__device__ __forceinline__ bool weigh_sequence(const WeighArgs& p, int b, WeighSequence& s) {
  const int q0 = __ldg(p.query_start_loc + b), q1 = __ldg(p.query_start_loc + b + 1), L = __ldg(p.seq_lens + b);
  if (q0 < 0 || q1 < q0 || q1 > p.num_tokens || L < 0 || q1 - q0 > L ||
      (L > 0 && (L - 1) / kPage >= p.desc.max_blocks_per_seq) || (b == 0 && q0 != 0) || q1 - q0 > p.max_rows) {
    s = {0, 0, 0};
    return false;
  }
  s = {q0, q1 - q0, L};
  return true;
}

// Exclusive prefix sums of N counts over the block's threads, in thread order;
// the totals come back in `total`.
template <int kThreads, int N>
__device__ __forceinline__ void block_scan(int64_t (&x)[N], int64_t (&total)[N], int64_t (*warp_sums)[N]) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int64_t incl[N];
#pragma unroll
  for (int i = 0; i < N; ++i) incl[i] = x[i];
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int64_t v = __shfl_up_sync(0xffffffffu, incl[i], o);
      if (lane >= o) incl[i] += v;
    }
  }
  if (lane == 31) {
#pragma unroll
    for (int i = 0; i < N; ++i) warp_sums[warp][i] = incl[i];
  }
  __syncthreads();
  static_assert(kThreads <= 1024, "a lane a warp");
#pragma unroll
  for (int i = 0; i < N; ++i) {
    int64_t sums = lane < kThreads / 32 ? warp_sums[lane][i] : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t v = __shfl_up_sync(0xffffffffu, sums, o);
      if (lane >= o) sums += v;
    }
    total[i] = __shfl_sync(0xffffffffu, sums, 31);
    const int64_t before = __shfl_sync(0xffffffffu, sums, (warp + 31) & 31);  // of the warps before
    x[i] = (warp ? before : 0) + incl[i] - x[i];
  }
}

// Quotient and remainder of counts, which hardly ever need 64 bits.
__device__ __forceinline__ int64_t divide(int64_t a, int64_t b, int64_t& rest) {
  int64_t q;
  if (((a | b) >> 31) == 0) q = uint32_t(a) / uint32_t(b);
  else q = a / b;
  rest = a - q * b;
  return q;
}

}  // namespace pkv
