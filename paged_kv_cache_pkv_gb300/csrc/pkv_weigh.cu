// pkv_weigh.cu -- accumulated attention weights: for every cached token and kv
// head the sum of the softmax weights that this step's query rows give it,
// added to paged scores.
//
//   lse[j, h] = log sum_{k <= pos j} exp(scale q[j, h] . K[k])
//   w[k]      = sum_{j, h: k <= pos j} exp(scale q[j, h] . K[k] - lse[j, h])
//
// A weight needs its row's sum over all keys first, so there are two passes.
// Both work in the log2 domain (exp2), sums in fp32.
//
// Few rows (up to kSmallRows query rows x heads of a kv head a sequence):
// bound by the bytes of K, which are read once.  Between others in a graph: 64
// sequences of 512 to 4096 tokens, 32 + 8 heads, 58.5 us (K alone 47 at the copy
// rate; 6.0 TB/s while K streams); a long-tailed batch of 256 sequences on E4M3
// pages 240 us (K 1.10 GB, 200 us of them at 5.5 TB/s).
//  * pkv_weigh_scores_kernel: K pages against the rows on warp-level MMAs, the
//    page's 16 keys as M, the rows as N (8, 16, 24 or 32).  A product of two
//    vectors does not go by the order of their elements, so a lane takes 16
//    contiguous bytes of a key's row as its elements of two k-steps, and the
//    queries' fragments are permuted alike: pages go from HBM to registers in
//    16-byte loads, without shared memory or barriers, as many pages of a warp
//    in flight as registers allow.  Each lane keeps running maxima and sums of its
//    own keys, reduced over lanes once a piece.  Scores go to the workspace, 4
//    bytes a (row, key), a key's rounded up to 16: at one row of four heads a
//    sixteenth of K's bytes, and mostly read back from L2.  Four rows' scores of
//    a page's 16 keys lie together, so that both kernels touch whole sectors (a
//    key's scores together: 8 rows of 4 heads 134 us, now 117; 2 to 5 rows 87,
//    now 84, and 81 since the second kernel has a form for 24 rows).
//  * pkv_weigh_add_kernel: joins the pieces' sums and turns scores into
//    weights, one key a lane, with the update of the paged score.  Its work is
//    little and its reads depend on one another, so all that do not are on
//    their way before the first is used.
//  * Units of work are pages of a kv head in the order (sequence, head, page);
//    a warp takes an equal share of them, so that lengths of any mixture load
//    all warps alike.  In a batch of many pages a head's first page counts as
//    kHeadUnits more: what begins a piece, queries, tables and the first pages'
//    way, takes as long as that (a long-tailed batch of 256 sequences on 8-bit
//    pages: 344 us without, 275, 246 and 242 with 4, 8 and 16).  A piece has the
//    record (items before it + warps before it), unique as one of them grows
//    from piece to piece.
//  * E4M3 pages: codes become f16 exactly; the bf16 queries become f16 under a
//    power of two a row that takes its largest element to [2^14, 2^15).  What
//    that loses of an element is below 2^-24 in f16's units, 2^-38 of the
//    largest: less than fp32 sums of 128 terms lose.  The key's scale is
//    applied to the finished score.
//
// Sequences of more rows go to the tensor cores (pkv_weigh_tc.cu).
#include <cuda_fp16.h>

#include <atomic>

#include "pkv_weigh.cuh"

namespace pkv {
namespace {

constexpr int kSmallRows = 32;
constexpr int kHeadUnits = 16;
constexpr int kWsThreads = 256;
constexpr int kWsWarps = kWsThreads / 32;

// The workspace of a call.
struct WeighLayout {
  size_t records, scores, many, total;
};

// What the kernels of few rows need beside the call's arguments.
struct SmallParams {
  WeighArgs a;
  float2* records;  // [items + warps][columns]: (maximum, sum) of a piece
  float4* scores;   // of each sequence [pages of its kv heads][quads][16 keys]
  int64_t max_quads;
  int32_t small_rows;   // rows x heads of a sequence that they take
  int32_t head_units;   // kHeadUnits or 0
  int32_t share_warps;  // warps of pkv_weigh_scores_kernel
};

// Score quads of a key.
__device__ __forceinline__ int quads_of(int rows) { return (rows + 3) >> 2; }

__device__ __forceinline__ int64_t share_of(const SmallParams& p, int64_t units) {
  int64_t rest;
  return max(int64_t(1), divide(units + p.share_warps - 1, p.share_warps, rest));
}

// Units and score quads before each sequence, in shared memory: [num_seqs + 1].
// Sequences of other sizes, without rows or beyond the workspace have none.
__device__ __forceinline__ void plan_units(const SmallParams& p, int64_t* before, int64_t* quads,
                                           int64_t (*warp_sums)[2]) {
  const int B = p.a.num_seqs, Hkv = p.a.desc.num_kv_heads, G = p.a.desc.num_q_heads / Hkv;
  const int per = (B + kWsThreads - 1) / kWsThreads;
  const int b0 = min(B, int(threadIdx.x) * per), b1 = min(B, b0 + per);
  int64_t sum[2] = {0, 0}, total[2];
  bool bad = false;
  for (int b = b0; b < b1; ++b) {
    WeighSequence s;
    bad = !weigh_sequence(p.a, b, s) || bad;
    const bool mine = s.n > 0 && int64_t(s.n) * G <= p.small_rows;
    const int pages = (s.L + kPage - 1) / kPage;
    before[b] = mine ? int64_t(Hkv) * (pages + p.head_units) : 0;
    quads[b] = mine ? int64_t(Hkv) * pages * kPage * quads_of(s.n * G) : 0;
    sum[0] += before[b];
    sum[1] += quads[b];
  }
  // The first sequence that does not fit the workspace whole ends the list.
  __shared__ unsigned long long limit;
  if (threadIdx.x == 0) limit = ~0ull;
  block_scan<kWsThreads, 2>(sum, total, warp_sums);
  for (int b = b0; b < b1; ++b) {
    const int64_t units = before[b], q = quads[b];
    if (units > 0 && sum[1] + q > p.max_quads) {
      atomicMin(&limit, static_cast<unsigned long long>(sum[0]));
      bad = true;
    }
    before[b] = sum[0];
    quads[b] = sum[1];
    sum[0] += units;
    sum[1] += q;
  }
  __syncthreads();
  const int64_t top = int64_t(min(limit, 0x7FFFFFFFFFFFFFFFull));
  for (int b = b0; b < b1; ++b) before[b] = min(before[b], top);
  if (threadIdx.x == 0) {
    before[B] = min(total[0], top);
    quads[B] = total[1];
  }
  if (bad && blockIdx.x == 0) flag_status(p.a.status, PKV_STATUS_BAD_QUERY);
  __syncthreads();
}

// Last sequence with before[b] <= unit (one that has units).
__device__ __forceinline__ int sequence_at(const int64_t* before, int B, int64_t unit) {
  int lo = 0, hi = B;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (before[mid] <= unit) lo = mid;
    else hi = mid;
  }
  return lo;
}

// 16 bytes that are read once: past L1.
__device__ __forceinline__ uint4 load_once(const void* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

template <bool F16>
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  if constexpr (F16)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, "
        "%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, "
        "%2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t word(const uint4& v, int i) {
  return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w;
}

// Four E4M3 codes (lowest byte first) -> two f16x2, exactly.
__device__ __forceinline__ void codes_f16(uint32_t w, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(w));
}

// One page of K as a lane holds it: rows lane / 4 and lane / 4 + 8, of each row
// the 16-byte pieces lane % 4, lane % 4 + 4, ...
template <bool F8>
struct KeyPage {
  static constexpr int kPieces = F8 ? 2 : 4;
  uint4 lo[kPieces], hi[kPieces];
  uint32_t sc_lo, sc_hi;  // E4M3: the rows' scale bytes
};

// Width of the records of a call with NT MMA tiles of columns.
__host__ __device__ constexpr int record_columns(int NT) { return NT == 3 ? 32 : 8 * NT; }

// E4M3 pages against two or three tiles of rows: the rows' fragments wait in
// shared memory, 2 KB a tile and warp, so that 16 warps an SM widen codes instead
// of eight (32 sequences of 256 to 8192 tokens, 12 rows a kv head 57 -> 53 us, 8
// to 20 rows 73 -> 63).  Four tiles (104 -> 103 us) and bf16 pages (three tiles,
// 82 -> 80), bound by their bytes, would gain too little for another path.
__host__ __device__ constexpr bool fragments_shared(int NT, bool F8) { return F8 && (NT == 2 || NT == 3); }
__host__ __device__ constexpr size_t fragment_bytes(int NT, bool F8) {
  return fragments_shared(NT, F8) ? size_t(NT) * kWsWarps * 2048 : 0;
}
// Blocks of the scores kernel on an SM; kScoresCtas at most.
constexpr int kScoresCtas = 2;
__host__ __device__ constexpr int scores_ctas(int NT, bool F8) { return NT == 1 || fragments_shared(NT, F8) ? 2 : 1; }

template <int NT, bool F8>
__global__ void __launch_bounds__(kWsThreads, scores_ctas(NT, F8)) pkv_weigh_scores_kernel(const SmallParams p) {
  constexpr bool kShared = fragments_shared(NT, F8);
  extern __shared__ uint4 fragments[];  // [warp][tile][4][lane]: of two k-steps
  uint4* const frag = fragments + (threadIdx.x >> 5) * NT * 128 + (threadIdx.x & 31);
  __shared__ int64_t before[kMaxSeqs + 1], quads_before[kMaxSeqs + 1];
  __shared__ int64_t warp_sums[kWsWarps][2];
  griddep_wait();
  griddep_launch_dependents();  // only pkv_weigh_add_kernel follows; it waits
  plan_units(p, before, quads_before, warp_sums);
  const WeighArgs& a = p.a;
  const int B = a.num_seqs, Hkv = a.desc.num_kv_heads, Hq = a.desc.num_q_heads, G = Hq / Hkv;
  const int lane = threadIdx.x & 31;
  const int row = lane >> 2, t = lane & 3;
  const int64_t units = before[B], share = share_of(p, units);
  const int64_t warp = int64_t(blockIdx.x) * kWsWarps + (threadIdx.x >> 5);
  int64_t u = min(units, warp * share);
  const int64_t end = min(units, u + share);
  if (u >= end) return;
  constexpr int kPieces = KeyPage<F8>::kPieces;
  // Pages of a warp in flight: 64 to 128 KB an SM.
  constexpr int kDeep = F8 ? (kShared ? 2 : 4) : NT == 2 ? 4 : NT == 3 ? 3 : 2;
  constexpr int kPieceBytes = 64;        // of a row, between a lane's pieces
  constexpr int kRowBytes = F8 ? kHeadDim : 2 * kHeadDim;
  int b = sequence_at(before, B, u);
  while (u < end) {
    WeighSequence s;
    weigh_sequence(a, b, s);
    const int pages = (s.L + kPage - 1) / kPage;
    int64_t rest;
    const int g = int(divide(u - before[b], pages + p.head_units, rest));
    const int taken = int(min(end - u, pages + p.head_units - rest));
    const int first = max(0, int(rest) - p.head_units), count = max(0, int(rest) + taken - p.head_units) - first;
    const int rows = s.n * G;  // the group's rows, j * G + h
    const int quads = quads_of(rows);
    // the lane's two columns of its first key: half of quad t / 2
    float* const scores = reinterpret_cast<float*>(p.scores + quads_before[b] +
                                                   ((int64_t(g) * pages + first) * quads + (t >> 1)) * kPage + row) +
                          2 * (t & 1);
    float2* const rec = p.records + (int64_t(b) * Hkv + g + warp) * record_columns(NT) + 2 * t;
    if (count == 0) {  // the head's first units alone
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
        if (row == 0)
          *reinterpret_cast<float4*>(rec + nt * 8) = make_float4(kWeighNoScore, 0.f, kWeighNoScore, 0.f);
      u += taken;
      continue;
    }

    // ---- the rows, as B fragments: lane's column row, its elements as in a key ----
    uint32_t qf[kShared ? 1 : NT][8][2];
    float unscale[NT][2];  // E4M3: of the lane's two score columns
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int col = nt * 8 + row;
      const bool live = col < rows;
      const uint16_t* qr = a.q + (int64_t(s.q0 + (live ? col / G : 0)) * Hq + g * G + (live ? col % G : 0)) * kHeadDim;
      if constexpr (!F8) {
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          uint4 v = make_uint4(0, 0, 0, 0);
          if (live) v = __ldg(reinterpret_cast<const uint4*>(qr + c * 32 + t * 8));
          qf[nt][2 * c][0] = v.x, qf[nt][2 * c][1] = v.y;
          qf[nt][2 * c + 1][0] = v.z, qf[nt][2 * c + 1][1] = v.w;
        }
      } else {
        uint4 v[2][2];
        float top = 0.f;
#pragma unroll
        for (int c = 0; c < 2; ++c) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            v[c][h] = make_uint4(0, 0, 0, 0);
            if (live) v[c][h] = __ldg(reinterpret_cast<const uint4*>(qr + c * 64 + t * 16 + h * 8));
#pragma unroll
            for (int i = 0; i < 4; ++i)
              top = fmaxf(top, fmaxf(fabsf(bf_lo(word(v[c][h], i))), fabsf(bf_hi(word(v[c][h], i)))));
          }
        }
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
        // 2^x takes top to [2^14, 2^15); x is bounded so that 2^x and 2^-x are
        // normal floats (a row below 2^-100 then has elements below 1)
        const int x = top == 0.f ? 0 : max(-113, min(114, 14 + 127 - int(__float_as_uint(top) >> 23)));
        const float up = __uint_as_float(uint32_t(127 + x) << 23), down = __uint_as_float(uint32_t(127 - x) << 23);
#pragma unroll
        for (int c = 0; c < 2; ++c) {
#pragma unroll
          for (int i = 0; i < 8; ++i) {  // words of two elements
            const uint32_t w = word(v[c][i >> 2], i & 3);
            const __half2 h = __floats2half2_rn(bf_lo(w) * up, bf_hi(w) * up);
            qf[kShared ? 0 : nt][c * 4 + (i >> 1)][i & 1] = *reinterpret_cast<const uint32_t*>(&h);
          }
        }
        unscale[nt][0] = __shfl_sync(0xffffffffu, down, 8 * t);
        unscale[nt][1] = __shfl_sync(0xffffffffu, down, 8 * t + 4);
      }
      if constexpr (kShared) {  // each lane reads what it wrote
#pragma unroll
        for (int c = 0; c < 4; ++c)
          frag[(nt * 4 + c) * 32] =
              make_uint4(qf[0][2 * c][0], qf[0][2 * c][1], qf[0][2 * c + 1][0], qf[0][2 * c + 1][1]);
      }
    }
    float m[NT][2], l[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      m[nt][0] = m[nt][1] = kWeighNoScore;
      l[nt][0] = l[nt][1] = 0.f;
    }

    // ---- pages ----
    // Page ids 32 at a time, one a lane; an id outside the pool is flagged and
    // page 0 read in its place, and the piece's maxima say so: the sequence's scores
    // are left alone.
    const int32_t* table = a.block_tables + int64_t(b) * a.desc.max_blocks_per_seq + first;
    int ids = 0;
    auto page_id = [&](int i) {
      if ((i & 31) == 0) {
        ids = i + lane < count ? __ldg(table + i + lane) : 0;
        const bool bad = ids < 0 || ids >= a.desc.num_blocks;
        if (bad) {
          flag_status(a.status, PKV_STATUS_BAD_BLOCK);
          ids = 0;
        }
        if (__any_sync(0xffffffffu, bad)) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) m[nt][0] = m[nt][1] = INFINITY;
        }
      }
      return __shfl_sync(0xffffffffu, ids, i & 31);
    };
    auto fetch = [&](KeyPage<F8>& k, int i) {
      const int64_t r = (int64_t(page_id(i)) * Hkv + g) * kPage + row;
      const char* at = static_cast<const char*>(a.k_cache) + r * kRowBytes + t * 16;
#pragma unroll
      for (int c = 0; c < kPieces; ++c) {
        k.lo[c] = load_once(at + c * kPieceBytes);
        k.hi[c] = load_once(at + 8 * kRowBytes + c * kPieceBytes);
      }
      if constexpr (F8) {
        k.sc_lo = __ldg(a.k_scale + r);
        k.sc_hi = __ldg(a.k_scale + r + 8);
      }
    };
    auto weigh_page = [&](const KeyPage<F8>& k, int i) {
      float d[NT][4];
      uint4 pair[NT];  // fragments of two k-steps
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) d[nt][0] = d[nt][1] = d[nt][2] = d[nt][3] = 0.f;
#pragma unroll
      for (int ks = 0; ks < 8; ++ks) {
        uint32_t a0, a1, a2, a3;
        if constexpr (F8) {
          codes_f16(word(k.lo[ks >> 2], ks & 3), a0, a2);
          codes_f16(word(k.hi[ks >> 2], ks & 3), a1, a3);
        } else {
          const int w = (ks & 1) * 2;
          a0 = word(k.lo[ks >> 1], w), a2 = word(k.lo[ks >> 1], w + 1);
          a1 = word(k.hi[ks >> 1], w), a3 = word(k.hi[ks >> 1], w + 1);
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          if (NT > 1 && nt * 8 >= rows) continue;
          if constexpr (kShared) {
            if ((ks & 1) == 0) pair[nt] = frag[(nt * 4 + (ks >> 1)) * 32];
            mma16816<F8>(d[nt], a0, a1, a2, a3, word(pair[nt], 2 * (ks & 1)), word(pair[nt], 2 * (ks & 1) + 1));
          } else {
            mma16816<F8>(d[nt], a0, a1, a2, a3, qf[nt][ks][0], qf[nt][ks][1]);
          }
        }
      }
      const int key = (first + i) * kPage + row;
      const bool edge = (first + i) * kPage + kPage - 1 > s.L - s.n;  // some row does not see all of the page
      float* out = scores + int64_t(i) * quads * (4 * kPage);
      float klo = 1.f, khi = 1.f;
      if constexpr (F8) {
        klo = __uint_as_float(k.sc_lo << 23);
        khi = __uint_as_float(k.sc_hi << 23);
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        if (NT > 1 && nt * 8 >= rows) break;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          float x = d[nt][j], y = d[nt][2 + j];
          if constexpr (F8) {
            x *= klo * unscale[nt][j];
            y *= khi * unscale[nt][j];
          }
          if (edge) {
            const int last = s.L - s.n + (nt * 8 + 2 * t + j) / G;
            if (key > last) x = -INFINITY;
            if (key + 8 > last) y = -INFINITY;
          }
          const float mn = fmaxf(m[nt][j], fmaxf(x, y));
          l[nt][j] = l[nt][j] * ex2((m[nt][j] - mn) * a.qscale) + ex2((x - mn) * a.qscale) + ex2((y - mn) * a.qscale);
          m[nt][j] = mn;
          d[nt][j] = x;
          d[nt][2 + j] = y;
        }
        if (nt * 2 + (t >> 1) < quads) {
          *reinterpret_cast<float2*>(out + nt * (8 * kPage)) = make_float2(d[nt][0], d[nt][1]);
          *reinterpret_cast<float2*>(out + nt * (8 * kPage) + 8 * 4) = make_float2(d[nt][2], d[nt][3]);
        }
      }
    };
    KeyPage<F8> k[kDeep];
#pragma unroll
    for (int i = 0; i < kDeep; ++i)
      if (i < count) fetch(k[i], i);
    for (int i = 0; i < count; i += kDeep) {
#pragma unroll
      for (int j = 0; j < kDeep; ++j) {
        if (i + j >= count) break;
        weigh_page(k[j], i + j);
        if (i + j + kDeep < count) fetch(k[j], i + j + kDeep);
      }
    }

    // ---- the piece's maxima and sums, over the lanes of a column ----
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) {
          const float mo = __shfl_xor_sync(0xffffffffu, m[nt][j], o), lo = __shfl_xor_sync(0xffffffffu, l[nt][j], o);
          const float mn = fmaxf(m[nt][j], mo);
          l[nt][j] = l[nt][j] * ex2((m[nt][j] - mn) * a.qscale) + lo * ex2((mo - mn) * a.qscale);
          m[nt][j] = mn;
        }
      }
      if (row == 0)
        *reinterpret_cast<float4*>(rec + nt * 8) = make_float4(m[nt][0], l[nt][0], m[nt][1], l[nt][1]);
    }
    u += taken;
    while (b + 1 < B && before[b + 1] <= u) ++b;  // u < end: some later sequence has it
  }
}

// Blocks of the kernel below on an SM.  One or two quads a key: three, whose
// registers let a lane have six or three keys on their way (decode 60.7 -> 59.3 us
// against four blocks and four keys, drafts of two rows 63.7 -> 61.9; five or six
// blocks spill: 63 and 72).
__host__ __device__ constexpr int add_ctas(int quads) { return quads == 8 ? 2 : quads == 4 ? 4 : 3; }

// Scores -> weights -> paged scores.  QUADS: most score quads of a key; COLUMNS:
// the records' width.
template <int QUADS, int COLUMNS>
__global__ void __launch_bounds__(kWsThreads, add_ctas(QUADS)) pkv_weigh_add_kernel(const SmallParams p) {
  __shared__ int64_t before[kMaxSeqs + 1], quads_before[kMaxSeqs + 1];
  __shared__ int64_t warp_sums[kWsWarps][2];
  const WeighArgs& a = p.a;
  const int B = a.num_seqs, Hkv = a.desc.num_kv_heads, G = a.desc.num_q_heads / Hkv;
  const int lane = threadIdx.x & 31;
  plan_units(p, before, quads_before, warp_sums);  // of arrays that the kernel before only reads
  griddep_wait();
  const int64_t units = before[B], share = share_of(p, units);
  const int64_t warps = int64_t(gridDim.x) * kWsWarps;
  int64_t spare;
  const int64_t mine = divide(units + warps - 1, warps, spare);
  int64_t u = min(units, (int64_t(blockIdx.x) * kWsWarps + (threadIdx.x >> 5)) * mine);
  const int64_t end = min(units, u + mine);
  int b = u < end ? sequence_at(before, B, u) : 0;
  while (u < end) {
    int64_t rest;
    const int units_a_head = int(divide(before[b + 1] - before[b], Hkv, rest)), pages = units_a_head - p.head_units;
    const int g = int(divide(u - before[b], units_a_head, rest));
    const int taken = int(min(end - u, units_a_head - rest));
    const int first = max(0, int(rest) - p.head_units), count = max(0, int(rest) + taken - p.head_units) - first;
    u += taken;
    if (count == 0) continue;  // the head's first units alone
    const int32_t* table = a.block_tables + int64_t(b) * a.desc.max_blocks_per_seq;
    // a lane's page of 32 keys from the piece's page i on, its entry or -1
    auto entry_of = [&](int i) {
      return i + (lane >> 4) < count ? __ldg(table + first + i + (lane >> 4)) : -1;
    };
    constexpr int kDeep = QUADS == 1 ? 6 : QUADS == 2 ? 3 : 1;  // 32 keys each, at a time
    int ids[kDeep];
#pragma unroll
    for (int d = 0; d < kDeep; ++d) ids[d] = entry_of(2 * d);
    WeighSequence s;
    weigh_sequence(a, b, s);
    const int from = a.first ? __ldg(a.first + b) : 0;
    const int given = a.scored ? __ldg(a.scored + b) : 0;

    // ---- log-sums of the rows: a column a lane, pieces in turn ----
    constexpr int kCols = COLUMNS < 32 ? COLUMNS : 32;
    const int64_t u0 = before[b] + int64_t(g) * units_a_head;
    const int64_t w0 = divide(u0, share, rest), w1 = divide(u0 + units_a_head - 1, share, rest);
    const float2* rec = p.records + (int64_t(b) * Hkv + g) * COLUMNS + lane % kCols;
    float m = kWeighNoScore, l = 0.f;
#pragma unroll 4
    for (int64_t w = w0 + lane / kCols; w <= w1; w += 32 / kCols) {
      const float2 x = __ldcg(rec + w * COLUMNS);
      const float mn = fmaxf(m, x.x);
      l = l * ex2((m - mn) * a.qscale) + x.y * ex2((x.x - mn) * a.qscale);
      m = mn;
    }
#pragma unroll
    for (int o = kCols; o < 32; o <<= 1) {
      const float mo = __shfl_xor_sync(0xffffffffu, m, o), lo = __shfl_xor_sync(0xffffffffu, l, o);
      const float mn = fmaxf(m, mo);
      l = l * ex2((m - mn) * a.qscale) + lo * ex2((mo - mn) * a.qscale);
      m = mn;
    }
    const float mine_lse = m * a.qscale + __log2f(l);
    const int rows = s.n * G, quads = quads_of(rows);
    // A page of the sequence is not the pool's.  (Columns behind the rows' may never
    // have been written.)
    const bool damaged = __any_sync(0xffffffffu, lane % kCols < rows && m == INFINITY);
    const int scored = a.decay == 0.f ? 0 : a.scored ? given : s.L - s.n;
    float lse[4 * QUADS];  // a column without a row: weight 0
#pragma unroll
    for (int c = 0; c < 4 * QUADS; ++c) {
      lse[c] = __shfl_sync(0xffffffffu, mine_lse, c % kCols);
      if (c >= rows) lse[c] = INFINITY;
    }

    // ---- a key a lane ----
    const float4* src = p.scores + quads_before[b] +
                        (int64_t(g) * pages + first + (lane >> 4)) * quads * kPage + (lane & 15);
    for (int i = damaged ? count : 0; i < count; i += 2 * kDeep) {
      int64_t at[kDeep];
      float old[kDeep];
      float4 x[kDeep][QUADS];
#pragma unroll
      for (int d = 0; d < kDeep; ++d) {
        const int key = (first + i + 2 * d) * kPage + lane;
        const bool live = i + 2 * d + (lane >> 4) < count && key >= from && key < s.L && ids[d] >= 0 &&
                          ids[d] < a.desc.num_blocks;  // flagged where its keys were read
        at[d] = live ? (int64_t(ids[d]) * Hkv + g) * kPage + (lane & 15) : -1;
        old[d] = 0.f;
        if (live && key < scored) old[d] = __ldcg(a.scores + at[d]);
#pragma unroll
        for (int c = 0; c < QUADS; ++c) {
          x[d][c] = make_float4(0.f, 0.f, 0.f, 0.f);
          if (live && c < quads) x[d][c] = __ldcg(src + (int64_t(i + 2 * d) * quads + c) * kPage);
        }
        ids[d] = entry_of(i + 2 * (kDeep + d));
      }
#pragma unroll
      for (int d = 0; d < kDeep; ++d) {
        if (at[d] < 0) continue;
        float w = 0.f;
#pragma unroll
        for (int c = 0; c < QUADS; ++c) {
          if (c >= quads) break;
          w += (ex2(fmaf(x[d][c].x, a.qscale, -lse[4 * c])) + ex2(fmaf(x[d][c].y, a.qscale, -lse[4 * c + 1]))) +
               (ex2(fmaf(x[d][c].z, a.qscale, -lse[4 * c + 2])) + ex2(fmaf(x[d][c].w, a.qscale, -lse[4 * c + 3])));
        }
        a.scores[at[d]] = fmaf(a.decay, old[d], w);
      }
    }
    while (b + 1 < B && before[b + 1] <= u) ++b;
  }
  // (behind a barrier: a block's first thread to say so speaks for all of them)
  __syncthreads();
  griddep_launch_dependents();
}

// Launched while the kernel before may still run, if that lets it.
template <class... Params, class... Args>
int launch(const LaunchCtx& ctx, void (*kernel)(Params...), int grid, size_t smem, const Args&... args) {
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(grid));
  cfg.blockDim = dim3(kWsThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = ctx.stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  TraceScope ts(ctx.stream, PKV_K_WEIGH);
  cudaLaunchKernelEx(&cfg, kernel, args...);
  return ts.done();
}

// MMA columns of the few-rows kernels: rows x heads, rounded up.
int column_tiles(int64_t rows) { return rows <= 8 ? 1 : rows <= 16 ? 2 : rows <= 24 ? 3 : 4; }

// Score quads of a key at most.
int most_quads(int64_t rows) { return int((rows + 3) / 4); }

// Rows x heads of a kv head that the few-rows kernels are launched for.
int64_t small_rows(const pkv_desc& d, int32_t max_rows) {
  const int64_t rows = int64_t(max_rows) * (d.num_q_heads / d.num_kv_heads);
  return rows < kSmallRows ? rows : kSmallRows;
}

// Whether a sequence may have more.
bool has_many(const pkv_desc& d, int32_t max_rows) {
  return int64_t(max_rows) * (d.num_q_heads / d.num_kv_heads) > kSmallRows;
}

// Whether a sequence may have no more.  Where the tokens are as many as the
// sequences at the most rows each, all have that many; should the bound not hold
// (a replay with fewer rows), the tensor cores take any number.
bool has_small(const pkv_desc& d, int32_t num_seqs, int32_t num_tokens, int32_t max_rows) {
  return !has_many(d, max_rows) || int64_t(num_seqs) * max_rows != num_tokens;
}

using AddKernel = void (*)(SmallParams);

// QUADS of pkv_weigh_add_kernel for so many at most.
int add_quads(int quads) { return quads <= 2 ? quads : quads <= 4 ? 4 : quads <= 6 ? 6 : 8; }

AddKernel add_kernel(int quads) {
  return quads <= 1   ? pkv_weigh_add_kernel<1, 8>
         : quads == 2 ? pkv_weigh_add_kernel<2, 8>
         : quads == 4 ? pkv_weigh_add_kernel<4, 16>
         : quads == 6 ? pkv_weigh_add_kernel<6, 32>
                      : pkv_weigh_add_kernel<8, 32>;
}

// A batch of few pages is spread over all warps page by page.
int head_units(const DeviceInfo& dev, const pkv_desc& d, int64_t num_keys) {
  return num_keys / kPage * d.num_kv_heads > int64_t(dev.sm_count) * 64 ? kHeadUnits : 0;
}

int scores_grid(const DeviceInfo& dev, const pkv_desc& d, int ctas, int64_t num_keys) {
  const int64_t units = num_keys / kPage * d.num_kv_heads;
  const int64_t most = int64_t(dev.sm_count) * ctas;
  const int64_t want = (units + kWsWarps - 1) / kWsWarps;
  return int(want < 1 ? 1 : want < most ? want : most);
}

int add_grid(const DeviceInfo& dev, const pkv_desc& d, int quads, int64_t num_keys) {
  const int64_t units = num_keys / kPage * d.num_kv_heads;
  const int64_t most = int64_t(dev.sm_count) * add_ctas(quads);
  const int64_t want = (units + 2 * kWsWarps - 1) / (2 * kWsWarps);
  return int(want < 1 ? 1 : want < most ? want : most);
}

template <int NT, bool F8>
int launch_scores(const LaunchCtx& ctx, int grid, const SmallParams& p) {
  constexpr size_t smem = fragment_bytes(NT, F8);
  if constexpr (smem > 0) {  // beside the static arrays more than a kernel has unasked
    static std::atomic<bool> done[64] = {};
    const int device = ctx.dev->device;
    if (device < 0 || device >= 64) return PKV_ERR_DEVICE;
    if (!done[device].load(std::memory_order_acquire)) {
      if (cudaFuncSetAttribute(pkv_weigh_scores_kernel<NT, F8>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                               int(smem)) != cudaSuccess) {
        cudaGetLastError();
        return PKV_ERR_LAUNCH;
      }
      done[device].store(true, std::memory_order_release);
    }
  }
  return launch(ctx, pkv_weigh_scores_kernel<NT, F8>, grid, smem, p);
}

template <bool F8>
int launch_scores(const LaunchCtx& ctx, int tiles, int grid, const SmallParams& p) {
  return tiles == 1   ? launch_scores<1, F8>(ctx, grid, p)
         : tiles == 2 ? launch_scores<2, F8>(ctx, grid, p)
         : tiles == 3 ? launch_scores<3, F8>(ctx, grid, p)
                      : launch_scores<4, F8>(ctx, grid, p);
}

WeighLayout layout(const DeviceInfo& dev, const pkv_desc& d, int32_t num_seqs, int32_t num_tokens, int32_t max_rows,
                   int64_t num_keys) {
  WeighLayout w{};
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t at = off;
    off = align_up(off + bytes, 256);
    return at;
  };
  if (!has_small(d, num_seqs, num_tokens, max_rows)) {
    w.total = weigh_tc_workspace_bytes(dev, d, num_seqs, num_tokens, num_keys);
    return w;
  }
  const int64_t rows = small_rows(d, max_rows);
  const size_t slots = size_t(num_seqs) * d.num_kv_heads +
                       size_t(scores_grid(dev, d, kScoresCtas, num_keys)) * kWsWarps;
  w.records = take(slots * record_columns(column_tiles(rows)) * sizeof(float2));
  w.scores = take(size_t(num_keys / kPage) * d.num_kv_heads * kPage * size_t(most_quads(rows)) * sizeof(float4));
  w.many = off;
  if (has_many(d, max_rows)) take(weigh_tc_workspace_bytes(dev, d, num_seqs, num_tokens, num_keys));
  w.total = off;
  return w;
}

}  // namespace

size_t weigh_workspace_bytes(const DeviceInfo& dev, const pkv_desc& d, int32_t num_seqs, int32_t num_tokens,
                             int32_t max_rows, int64_t num_keys) {
  return layout(dev, d, num_seqs, num_tokens, max_rows, num_keys).total;
}

int launch_weigh(const LaunchCtx& ctx, const WeighArgs& a, bool fp8) {
  const pkv_desc& d = a.desc;
  const WeighLayout w = layout(*ctx.dev, d, a.num_seqs, a.num_tokens, a.max_rows, a.num_keys);
  if (a.workspace_bytes < w.total) return PKV_ERR_WORKSPACE;
  uint8_t* ws = static_cast<uint8_t*>(a.workspace);
  const int64_t rows = small_rows(d, a.max_rows);
  const int tiles = column_tiles(rows);
  const int grid = scores_grid(*ctx.dev, d, scores_ctas(tiles, fp8), a.num_keys);
  const bool small = has_small(d, a.num_seqs, a.num_tokens, a.max_rows);
  if (small) {
    const SmallParams p{a,
                        reinterpret_cast<float2*>(ws + w.records),
                        reinterpret_cast<float4*>(ws + w.scores),
                        a.num_keys / kPage * d.num_kv_heads * kPage * most_quads(rows),
                        int32_t(rows),
                        head_units(*ctx.dev, d, a.num_keys),
                        grid * kWsWarps};
    if (int e = fp8 ? launch_scores<true>(ctx, tiles, grid, p) : launch_scores<false>(ctx, tiles, grid, p)) return e;
    const int quads = add_quads(most_quads(rows));
    if (int e = launch(ctx, add_kernel(quads), add_grid(*ctx.dev, d, quads, a.num_keys), 0, p))
      return e;
  }
  if (!has_many(d, a.max_rows)) return PKV_OK;
  return launch_weigh_tc(ctx, a, fp8, small ? int32_t(rows) : 0, ws + w.many);
}

}  // namespace pkv
