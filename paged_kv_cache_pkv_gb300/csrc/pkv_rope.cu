// pkv_rope.cu -- appends that rotate by position on the way: the K/V append of
// pkv_write and pkv_write_fp8 with the rotation of K and of the queries in the
// same pass, and the append to latent pages.
//
// Rotation of a pair (a, b) at position p with the table's c = cos, s = sin of
// its angle:  (a, b) -> (a c - b s, b c + a s).  The arithmetic is fp32 with
// every product and every sum rounded (no fused multiply-add), so that the
// result does not depend on how a compiler contracts it: on 8-bit pages one
// bit of it can move a code by a whole step.  The result is rounded once, to
// bf16 or (under the row's power of two) to E4M3; it is not rounded to bf16
// before E4M3, which would round twice.
//
// What bounds it: bytes.  Every row is read once and written once; the table
// adds rotary_dim * 4 bytes a token.  A unit of work is 16 elements of one
// row, two 16-byte vectors whose elements pair up: vectors j and
// j + rotary_dim/16 of the row in the half-split pairing, vectors 2j and
// 2j + 1 in the interleaved one; both use entries 8j..8j+7 of the table's
// cosines and sines, which the thread keeps in registers over all the heads
// that it handles of its token.
#include <cuda_fp8.h>

#include "pkv_common.cuh"
#include "pkv_internal.h"

namespace pkv {
namespace {

constexpr int kRopeThreads = 128;

struct Pair16 {
  uint4 a, b;
};

// The rotated fp32 values of one unit: out[0..7] for vector a's elements,
// out[8..15] for vector b's.
__device__ __forceinline__ void turn(const Pair16& x, const float (&c)[8], const float (&s)[8],
                                     bool interleaved, float (&out)[16]) {
  const uint32_t w[8] = {x.a.x, x.a.y, x.a.z, x.a.w, x.b.x, x.b.y, x.b.z, x.b.w};
  float v[16];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    v[2 * i] = bf_lo(w[i]);
    v[2 * i + 1] = bf_hi(w[i]);
  }
  if (interleaved) {  // pair i = elements 2i, 2i + 1 of the unit
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      out[2 * i] = __fsub_rn(__fmul_rn(v[2 * i], c[i]), __fmul_rn(v[2 * i + 1], s[i]));
      out[2 * i + 1] = __fadd_rn(__fmul_rn(v[2 * i + 1], c[i]), __fmul_rn(v[2 * i], s[i]));
    }
  } else {  // pair i = element i of a, element i of b
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      out[i] = __fsub_rn(__fmul_rn(v[i], c[i]), __fmul_rn(v[8 + i], s[i]));
      out[8 + i] = __fadd_rn(__fmul_rn(v[8 + i], c[i]), __fmul_rn(v[i], s[i]));
    }
  }
}

__device__ __forceinline__ Pair16 to_bf16(const float (&o)[16]) {
  Pair16 r;
  r.a = make_uint4(pack_bf16x2(o[0], o[1]), pack_bf16x2(o[2], o[3]), pack_bf16x2(o[4], o[5]),
                   pack_bf16x2(o[6], o[7]));
  r.b = make_uint4(pack_bf16x2(o[8], o[9]), pack_bf16x2(o[10], o[11]), pack_bf16x2(o[12], o[13]),
                   pack_bf16x2(o[14], o[15]));
  return r;
}

__device__ __forceinline__ void spread(const float4& x, const float4& y, float (&v)[8]) {
  v[0] = x.x, v[1] = x.y, v[2] = x.z, v[3] = x.w;
  v[4] = y.x, v[5] = y.y, v[6] = y.z, v[7] = y.w;
}

__device__ __forceinline__ void load8(const float* p, float (&v)[8]) {
  spread(__ldg(reinterpret_cast<const float4*>(p)), __ldg(reinterpret_cast<const float4*>(p) + 1), v);
}

// Vectors of unit j of a row: the first `units` units are rotated, the rest
// are the row's remaining vectors, two by two.
__device__ __forceinline__ void unit_vectors(int j, int units, bool interleaved, int& va, int& vb) {
  const bool split = j < units && !interleaved;
  va = split ? j : 2 * j;
  vb = split ? j + units : 2 * j + 1;
}

// Scale exponent of a row from its largest magnitude (finite): the smallest e
// in [-126, 127] with amax <= 448 * 2^e; amax = (1 + f) * 2^E needs E - 8, one
// more where 1 + f exceeds 448 / 2^8 = 1.75.
__device__ __forceinline__ int row_exponent_f32(float amax) {
  const uint32_t u = __float_as_uint(amax);
  const int e = int(u >> 23) - 127 - 8 + ((u & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return e < -126 ? -126 : (e > 127 ? 127 : e);
}

__device__ __forceinline__ uint2 to_e4m3(const float* o, float inv) {
  uint32_t h[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    h[i] = __nv_cvt_float2_to_fp8x2(make_float2(o[2 * i] * inv, o[2 * i + 1] * inv), __NV_SATFINITE,
                                    __NV_E4M3);
  return make_uint2(h[0] | (h[1] << 16), h[2] | (h[3] << 16));
}

// One block handles one token at a time (blockIdx.x) and the share
// blockIdx.y of its rows: query heads (if any), K heads, V heads.  Eight
// threads a row, one unit each.
// AXES, several positions a token: a thread a pair reads the entries of its
// pair's axis, and the block's rows have them from shared memory; the next
// token's are on their way while this one's rows are turned.  (Read by every
// thread for itself, axes in turn took three rows' vectors a unit: 4099 tokens of
// 32 + 8 heads 21.5 us between others in a graph, 14.3 as it is.)  Its blocks are
// bound to the registers of as many as the grid has an SM: 21.5 -> 16.8 us from
// cold caches.
template <bool F8, bool AXES>
__global__ void __launch_bounds__(kRopeThreads, AXES ? (F8 ? 8 : 9) : 1) pkv_write_rope_kernel(const RopeWriteArgs p) {
  // What the stream did before: the projections, and calls that read the pools.
  griddep_wait();
  constexpr int kUnits = kHeadDim / 16;  // 8
  constexpr int kRows = kRopeThreads / kUnits;
  const int j = threadIdx.x % kUnits;
  const int units = p.rotary_dim / 16;
  const bool rotated = j < units;
  const int rows = p.num_q_heads + 2 * p.num_kv_heads;
  const int first = (p.q ? 0 : p.num_q_heads) + blockIdx.y * kRows + threadIdx.x / kUnits;
  const int step = gridDim.y * kRows;
  int va, vb;
  unit_vectors(j, units, p.interleaved != 0, va, vb);
  // AXES: thread i reads positions, cosine and sine for pair i, threads behind the
  // pairs the positions of the axes once more (one may have no pair).
  __shared__ float4 table[AXES ? 2 : 1][AXES ? 2 : 1][AXES ? kHeadDim / 8 : 1];  // [by turns][cosines, sines]
  const int half = p.rotary_dim / 2;
  const int64_t* axis_pos = nullptr;
  int64_t pos_ahead = 0, slot_ahead = AXES ? __ldg(p.slots + blockIdx.x) : 0;
  float cos_ahead = 0.f, sin_ahead = 0.f;
  bool bad_ahead = false;
  auto look_up = [&] {  // the table's entries at pos_ahead
    bad_ahead = axis_pos && (pos_ahead < 0 || pos_ahead >= p.max_position);
    if (int(threadIdx.x) < half && !bad_ahead) {
      const float* row = p.cos_sin + pos_ahead * p.rotary_dim + threadIdx.x;
      cos_ahead = __ldg(row);
      sin_ahead = __ldg(row + half);
    }
  };
  if constexpr (AXES) {
    int axis = int(threadIdx.x) - half;
    if (axis < 0)
      for (axis = 0; !(p.axis_pairs[axis] >> threadIdx.x & 1); ++axis) {}
    if (axis < p.num_axes) axis_pos = p.positions + axis * p.position_stride;
    if (axis_pos) pos_ahead = __ldg(axis_pos + blockIdx.x);
    look_up();
    const int64_t next = blockIdx.x + int64_t(gridDim.x);
    if (axis_pos && next < p.num_tokens) pos_ahead = __ldg(axis_pos + next);
  }
  int turn_of = 0;
  for (int64_t t = blockIdx.x; t < p.num_tokens; t += gridDim.x, turn_of ^= 1) {
    int64_t pos = 0, slot;
    bool bad_pos;
    if constexpr (AXES) {
      slot = slot_ahead;
      if (int(threadIdx.x) < half) {
        reinterpret_cast<float*>(table[turn_of][0])[threadIdx.x] = cos_ahead;
        reinterpret_cast<float*>(table[turn_of][1])[threadIdx.x] = sin_ahead;
      }
      // (one barrier a token: the buffer is written again two tokens on)
      bad_pos = __syncthreads_or(bad_ahead);
      const int64_t next = t + int64_t(gridDim.x);
      if (next < p.num_tokens) {
        slot_ahead = __ldg(p.slots + next);
        look_up();
        if (axis_pos && next + gridDim.x < p.num_tokens) pos_ahead = __ldg(axis_pos + next + gridDim.x);
      }
    } else {
      pos = __ldg(p.positions + t);
      bad_pos = pos < 0 || pos >= p.max_position;
      slot = __ldg(p.slots + t);
    }
    const int64_t page = slot / kPage;
    const int r = int(slot % kPage);
    const bool store = slot >= 0 && page < p.num_blocks && !bad_pos;
    if (threadIdx.x == 0 && blockIdx.y == 0) {
      const unsigned bits = (slot >= 0 && page >= p.num_blocks ? PKV_STATUS_BAD_SLOT : 0u) |
                            (bad_pos ? PKV_STATUS_BAD_POSITION : 0u);
      if (bits) flag_status(p.status, bits);
    }
    if (bad_pos) continue;  // no angle: nothing of this token is written
    float c[8], s[8];
    if (rotated) {
      if constexpr (AXES) {
        spread(table[turn_of][0][2 * j], table[turn_of][0][2 * j + 1], c);
        spread(table[turn_of][1][2 * j], table[turn_of][1][2 * j + 1], s);
      } else {
        const float* row = p.cos_sin + pos * p.rotary_dim;
        load8(row + 8 * j, c);
        load8(row + p.rotary_dim / 2 + 8 * j, s);
      }
    }
    for (int h = first; h < rows; h += step) {
      const bool is_q = h < p.num_q_heads;
      if (!is_q && !store) break;  // K and V rows come last
      const int hk = h - p.num_q_heads;
      const bool is_v = hk >= p.num_kv_heads;
      const uint16_t* src = is_q   ? p.q + t * p.q_stride + h * kHeadDim
                            : is_v ? p.v + t * p.v_stride + (hk - p.num_kv_heads) * kHeadDim
                                   : p.k + t * p.k_stride + hk * kHeadDim;
      Pair16 x;
      x.a = *(reinterpret_cast<const uint4*>(src) + va);
      x.b = *(reinterpret_cast<const uint4*>(src) + vb);
      const bool turned = rotated && !is_v;
      float o[16];
      if (turned) {
        turn(x, c, s, p.interleaved != 0, o);
        if (is_q || !F8) x = to_bf16(o);
      }
      if (is_q) {
        uint4* dst = reinterpret_cast<uint4*>(p.q_out + (t * p.num_q_heads + h) * kHeadDim);
        dst[va] = x.a;
        dst[vb] = x.b;
        continue;
      }
      const int64_t ph = page * p.num_kv_heads + (is_v ? hk - p.num_kv_heads : hk);
      if constexpr (!F8) {
        uint4* dst = reinterpret_cast<uint4*>(is_v ? p.v_cache : p.k_cache) +
                     (ph * kPage + r) * (kHeadDim / 8);
        dst[va] = x.a;
        dst[vb] = x.b;
      } else {
        if (!turned) {
          const uint32_t w[8] = {x.a.x, x.a.y, x.a.z, x.a.w, x.b.x, x.b.y, x.b.z, x.b.w};
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            o[2 * i] = bf_lo(w[i]);
            o[2 * i + 1] = bf_hi(w[i]);
          }
        }
        float amax = 0.f;
#pragma unroll
        for (int i = 0; i < 16; ++i) amax = fmaxf(amax, fabsf(o[i]));
        const unsigned group = 0xFFu << (threadIdx.x & 24);  // the row's eight lanes
#pragma unroll
        for (int d = 4; d >= 1; d >>= 1) amax = fmaxf(amax, __shfl_xor_sync(group, amax, d));
        const int e = row_exponent_f32(amax);
        const float inv = __uint_as_float(uint32_t(127 - e) << 23);  // 2^-e, a normal float
        uint2* dst = reinterpret_cast<uint2*>(is_v ? p.v_cache : p.k_cache) +
                     (ph * kPage + r) * (kHeadDim / 8);
        dst[va] = to_e4m3(o, inv);
        dst[vb] = to_e4m3(o + 8, inv);
        if (j == 0) (is_v ? p.v_scale : p.k_scale)[ph * kPage + r] = uint8_t(e + 127);
      }
    }
  }
  // Let a dependent attention kernel start its set-up; it reads the pools and
  // the queries after this grid has finished.  (Not at the start: a kernel that
  // is not one of this library's may write before it waits, to memory that the
  // caller has back from this call's inputs.  And behind a barrier: a block's
  // first thread to say so speaks for all of them, also for those still
  // reading.)
  __syncthreads();
  griddep_launch_dependents();
}

// Latent pages: row = [512 latent values | 64 rotated key values].  One block
// handles one token at a time: rows of four units (the shared key part and
// each query head's rotated part) and the latent's 64 vectors.
__global__ void __launch_bounds__(kRopeThreads) pkv_write_latent_kernel(const LatentWriteArgs p) {
  griddep_wait();
  constexpr int kUnits = kLatentRope / 16;  // 4
  constexpr int kRows = kRopeThreads / kUnits;
  constexpr int kVecs = kLatentDim / 8;     // 64
  const int j = threadIdx.x % kUnits;
  int va, vb;
  unit_vectors(j, kUnits, p.interleaved != 0, va, vb);
  // row 0 is the shared key part, row h + 1 query head h
  const int rows = p.q_pe ? p.num_heads + 1 : 1;
  for (int64_t t = blockIdx.x; t < p.num_tokens; t += gridDim.x) {
    const int64_t pos = __ldg(p.positions + t);
    const int64_t slot = __ldg(p.slots + t);
    const bool bad_pos = pos < 0 || pos >= p.max_position;
    const bool store = slot >= 0 && slot / kPage < p.num_blocks && !bad_pos;
    if (threadIdx.x == 0 && blockIdx.y == 0) {
      const unsigned bits = (slot >= 0 && slot / kPage >= p.num_blocks ? PKV_STATUS_BAD_SLOT : 0u) |
                            (bad_pos ? PKV_STATUS_BAD_POSITION : 0u);
      if (bits) flag_status(p.status, bits);
    }
    if (bad_pos) continue;
    uint4* dst = reinterpret_cast<uint4*>(p.cache + slot * kLatentRow);  // page rows are contiguous
    if (store && blockIdx.y == 0 && threadIdx.x < kVecs)
      dst[threadIdx.x] = *(reinterpret_cast<const uint4*>(p.c_new + t * p.c_stride) + threadIdx.x);
    float c[8], s[8];
    const float* row = p.cos_sin + pos * kLatentRope;
    load8(row + 8 * j, c);
    load8(row + kLatentRope / 2 + 8 * j, s);
    for (int h = blockIdx.y * kRows + threadIdx.x / kUnits; h < rows; h += gridDim.y * kRows) {
      if (h == 0 && !store) continue;
      const uint4* src = reinterpret_cast<const uint4*>(
          h == 0 ? p.k_pe + t * p.k_stride : p.q_pe + t * p.q_stride + (h - 1) * p.q_head_stride);
      Pair16 x;
      x.a = src[va];
      x.b = src[vb];
      float o[16];
      turn(x, c, s, p.interleaved != 0, o);
      x = to_bf16(o);
      uint4* to = h == 0 ? dst + kVecs
                         : reinterpret_cast<uint4*>(p.q_out + (t * p.num_heads + h - 1) * kLatentRow + kLatentDim);
      to[va] = x.a;
      to[vb] = x.b;
    }
  }
  __syncthreads();  // as above
  griddep_launch_dependents();
}

// Blocks over tokens, and over the rows of a token while there are few
// tokens: as many as are resident at once (nine of 128 threads an SM; 16 a SM
// took 34.2 us for 8191 tokens of 32 + 8 heads, 9 take 33.1).
dim3 token_grid(const DeviceInfo& dev, int64_t tokens, int rows, int rows_per_block, int blocks_per_sm = 9) {
  const int64_t want = int64_t(dev.sm_count) * blocks_per_sm;
  const int64_t gx = tokens < want ? tokens : want;
  const int most = (rows + rows_per_block - 1) / rows_per_block;
  int64_t gy = want / gx;
  gy = gy < 1 ? 1 : gy > most ? most : gy;
  return dim3(unsigned(gx), unsigned(gy));
}

// Launched while the stream's last kernel may still run, if that is one of this
// library's (64 tokens 2.4 -> 2.0 us on FP8 pages and 2.6 -> 2.2 on latent ones,
// between others in a graph).
template <class Args>
int launch(const LaunchCtx& ctx, void (*kernel)(Args), dim3 grid, const Args& args) {
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(kRopeThreads);
  cfg.stream = ctx.stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  TraceScope ts(ctx.stream, PKV_K_WRITE);
  cudaLaunchKernelEx(&cfg, kernel, args);
  return ts.done();
}

}  // namespace

int launch_write_rope(const LaunchCtx& ctx, const RopeWriteArgs& a, bool fp8) {
  const int rows = (a.q ? a.num_q_heads : 0) + 2 * a.num_kv_heads;
  // (with several axes on E4M3 pages eight are)
  const dim3 grid = token_grid(*ctx.dev, a.num_tokens, rows, kRopeThreads / (kHeadDim / 16), fp8 && a.num_axes ? 8 : 9);
  if (a.num_axes)
    return launch(ctx, fp8 ? pkv_write_rope_kernel<true, true> : pkv_write_rope_kernel<false, true>, grid, a);
  return launch(ctx, fp8 ? pkv_write_rope_kernel<true, false> : pkv_write_rope_kernel<false, false>, grid, a);
}

int launch_write_latent(const LaunchCtx& ctx, const LatentWriteArgs& a) {
  const dim3 grid = token_grid(*ctx.dev, a.num_tokens, a.q_pe ? a.num_heads + 1 : 1,
                               kRopeThreads / (kLatentRope / 16));
  return launch(ctx, pkv_write_latent_kernel, grid, a);
}

}  // namespace pkv
