// pkv_latent.cuh -- what the kernels of latent attention share: the batch's
// parameters and the work split over CTAs (or pairs of them).
#pragma once

#include "pkv_internal.h"
#include "pkv_tcgen05.cuh"

namespace pkv {

constexpr int kLtChunks = kLatentRow / 64;  // 9 chunks of 64 dims (the last is rotated, keys only)

struct LatentParams {
  const int32_t *block_tables, *seq_lens, *qsl;
  uint16_t* out;
  const uint16_t* cache;
  float* partials;     // [CTAs][2][partial_stride]
  // [CTAs] the tile that the CTA's share ends inside (first row, rows, last
  // CTA with a piece of it; 0 rows: none), and the first CTA of the tile that
  // its share begins inside (-1: none)
  int4* joins;
  unsigned* status;
  int32_t B, T, H, max_blocks, num_blocks;
  uint32_t inv_heads;  // floor(2^32 / H), at most 2^32 - 1
  float qscale;        // scale * log2(e)
};

// Weights of the work split, in units of (keys x heads): tile j of a sequence
// of n query tokens and ctx = L - n earlier ones weighs H * (ctx + kLtTileCost)
// + (j + 1) * N, which is H times its last row's keys plus a constant for
// loading its queries and writing its result; the sum over tiles is closed.
constexpr int kLtTileCost = 128;
// A share is at least this many keys: below it a second CTA's start and the
// merge cost more than the keys.
constexpr int kLtMinShare = 256 + kLtTileCost;
// Keys a piece where tiles have CTAs of their own: fewer than the least cost
// more to join than they save; above the most, equal shares of the weight are
// the better balance.
constexpr int kLtLeastOwn = 256, kLtMostOwn = 1024;

// row / H (row >= 0): the product is one short of it at most.
__device__ __forceinline__ int lt_token(const LatentParams& p, int row) {
  const int t = int(__umulhi(uint32_t(row), p.inv_heads));
  return row - t * p.H >= p.H ? t + 1 : t;
}

struct LtSeq {
  int q0, n, L, rows, tiles;  // tiles == 0: no rows, or inconsistent
  bool bad;
};

template <int N>
__device__ __forceinline__ LtSeq lt_seq(const LatentParams& p, int b, int q0, int q1, int L) {
  LtSeq s;
  s.q0 = q0;
  s.L = L;
  s.n = q1 - q0;
  s.bad = q0 < 0 || s.n < 0 || q1 > p.T || s.n > L || L < 0 || (L + kPage - 1) / kPage > p.max_blocks ||
          (b == 0 && q0 != 0);
  if (s.bad) s.n = 0;
  s.rows = s.n * p.H;
  s.tiles = (s.rows + N - 1) / N;
  return s;
}
template <int N>
__device__ __forceinline__ LtSeq lt_seq(const LatentParams& p, int b) {
  return lt_seq<N>(p, b, __ldg(p.qsl + b), __ldg(p.qsl + b + 1), __ldg(p.seq_lens + b));
}

// Weight of the first j tiles of a sequence.
template <int N>
__device__ __forceinline__ int64_t lt_weight(const LatentParams& p, const LtSeq& s, int64_t j) {
  return j * (int64_t(p.H) * (s.L - s.n + kLtTileCost)) + N * (j * (j + 1) / 2);
}

// Key blocks that tile j of a sequence sees.
template <int N, int KEYS>
__device__ __forceinline__ int lt_blocks(const LatentParams& p, const LtSeq& s, int j) {
  const int last_row = min(s.rows, (j + 1) * N) - 1;
  const int keys = s.L - s.n + lt_token(p, last_row) + 1;
  return (keys + KEYS - 1) / KEYS;
}

// A place in the work: key block k of tile j of sequence b (b == B: the end).
struct LtPos {
  int b, j, k;
};

// A piece of one tile: key blocks [k0, k1) of its `blocks`.
struct LtPiece {
  int b, j, k0, k1, blocks;
  int row0, rows;   // of the tile: first row in q and out, rows
  int local_row;    // the first row's index within the sequence's rows
  int n, L;
};

// A walk over a share's pieces.  The sequence it is in is kept: its numbers
// are read once.
struct LtWalk {
  LtPos at, end;
  LtSeq s;  // of sequence at.b
};

// The next piece (never empty); false at the share's end.
template <int N, int KEYS>
__device__ __forceinline__ bool lt_next(const LatentParams& p, LtWalk& w, LtPiece& x) {
  for (;;) {
    const LtPos& e = w.end;
    if (w.at.b >= p.B || w.at.b > e.b || (w.at.b == e.b && (w.at.j > e.j || (w.at.j == e.j && w.at.k >= e.k))))
      return false;
    if (w.at.j >= w.s.tiles) {
      w.at.b += 1;
      w.at.j = w.at.k = 0;
      if (w.at.b < p.B) w.s = lt_seq<N>(p, w.at.b);
      continue;
    }
    x.b = w.at.b;
    x.j = w.at.j;
    x.k0 = w.at.k;
    x.blocks = lt_blocks<N, KEYS>(p, w.s, w.at.j);
    x.k1 = (w.at.b == e.b && w.at.j == e.j) ? e.k : x.blocks;
    x.local_row = w.at.j * N;
    x.rows = min(N, w.s.rows - w.at.j * N);
    x.row0 = w.s.q0 * p.H + w.at.j * N;
    x.n = w.s.n;
    x.L = w.s.L;
    w.at.j += 1;
    w.at.k = 0;
    return true;
  }
}

// Shared memory that the plan borrows: weight before each sequence, and its
// query_start_loc[b], [b + 1] and seq_lens[b].
constexpr int kLtPlanBytes = (PKV_MAX_SEQS + 2) * 8 + PKV_MAX_SEQS * 16;

// Sum over the threads before this one of their `v`, and over all of `v` and
// of `u`.
template <int THREADS>
__device__ __forceinline__ int64_t block_scan(int64_t v, int64_t u, longlong2* s_wsum, longlong2& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int64_t incl = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t x = __shfl_up_sync(0xffffffffu, incl, o);
    u += __shfl_xor_sync(0xffffffffu, u, o);
    if (lane >= o) incl += x;
  }
  if (lane == 31) s_wsum[warp] = make_longlong2(incl, u);
  __syncthreads();
  int64_t run = incl - v;
  total = make_longlong2(0, 0);
#pragma unroll
  for (int x = 0; x < THREADS / 32; ++x) {
    const longlong2 s = s_wsum[x];
    if (x < warp) run += s.x;
    total.x += s.x;
    total.y += s.y;
  }
  return run;
}

// The share of part `part` of `parts` (a CTA, or a pair of them): begin in
// share[0..2], end in [4..6], in [7] the last part with a piece of the tile that
// the share ends inside, in [8..10] the numbers of the first sequence, in [11]
// the first part of the tile that the share begins inside (-1: none).  All
// threads of the block take part; the caller synchronises behind it.
template <int N, int KEYS, int THREADS>
__device__ __forceinline__ void lt_plan(const LatentParams& p, int part, int parts, uint8_t* scratch,
                                        longlong2* s_wsum, int* s_share) {
  const int tid = threadIdx.x;
  int64_t* s_scan = reinterpret_cast<int64_t*>(scratch);      // weight before sequence b
  int4* s_seq = reinterpret_cast<int4*>(s_scan + PKV_MAX_SEQS + 2);  // its q0, q1, L
  const int per = (p.B + THREADS - 1) / THREADS;
  const int b0 = min(p.B, tid * per), b1 = min(p.B, b0 + per);
  // Tiles and key blocks of the batch ride along in one word, each capped
  // far above what the choice below looks at.
  int64_t local = 0, tiles_of = 0, blocks_of = 0;
  for (int b = b0; b < b1; ++b) {
    const int4 raw = make_int4(__ldg(p.qsl + b), __ldg(p.qsl + b + 1), __ldg(p.seq_lens + b), 0);
    s_seq[b] = raw;
    const LtSeq s = lt_seq<N>(p, b, raw.x, raw.y, raw.z);
    if (s.bad && part == 0) flag_status(p.status, PKV_STATUS_BAD_QUERY);
    const int64_t w = lt_weight<N>(p, s, s.tiles);
    s_scan[b] = w;
    local += w;
    tiles_of += s.tiles;
    blocks_of += int64_t(s.tiles) * ((s.L + KEYS - 1) / KEYS);
  }
  longlong2 sums;
  int64_t run = block_scan<THREADS>(local, (min(tiles_of, int64_t(1) << 20) << 32) | min(blocks_of, int64_t(1) << 20), s_wsum, sums);
  const int64_t total = sums.x;
  const int tiles = int(sums.y >> 32), blocks_all = int(sums.y & 0xFFFFFFFF);
  for (int b = b0; b < b1; ++b) {
    const int64_t w = s_scan[b];
    s_scan[b] = run;
    run += w;
  }
  if (tid == 0) s_scan[p.B] = total;
  __syncthreads();
  // Few tiles: each has parts of its own, pieces of `own` key blocks, so that
  // a part has one piece and no tile is cut that need not be (four sequences
  // of up to 255 tokens: 16.3 -> 13.4 us).  The pieces fit the grid because
  // ceil(n / own) sums to no more than tiles + blocks / own.
  int own = 0;
  if (tiles > 0 && tiles < parts) {
    const float t = float(blocks_all) / float(parts - tiles);
    if (t <= float(kLtMostOwn / KEYS)) own = max(kLtLeastOwn / KEYS, int(ceilf(t)));
  }
  if (own > 0) {
    auto cuts = [&](const LtSeq& s) {  // pieces of a tile
      const int n = (s.L + KEYS - 1) / KEYS;
      return n <= 2 * own ? 1 : (n + own - 1) / own;
    };
    int64_t count = 0;
    for (int b = b0; b < b1; ++b) {
      const int4 raw = s_seq[b];
      const LtSeq s = lt_seq<N>(p, b, raw.x, raw.y, raw.z);
      count += int64_t(s.tiles) * cuts(s);
    }
    int first_cta = int(block_scan<THREADS>(count, 0, s_wsum + THREADS / 32, sums));
    if (tid == 0) {
      *reinterpret_cast<int4*>(s_share) = make_int4(p.B, 0, 0, -1);
      *reinterpret_cast<int4*>(s_share + 4) = make_int4(p.B, 0, 0, -1);
      *reinterpret_cast<int4*>(s_share + 8) = make_int4(0, 0, 0, -1);
    }
    __syncthreads();
    for (int b = b0; b < b1; ++b) {
      const int4 raw = s_seq[b];
      const LtSeq s = lt_seq<N>(p, b, raw.x, raw.y, raw.z);
      const int n = cuts(s), r = part - first_cta;
      first_cta += s.tiles * n;
      if (r < 0 || r >= s.tiles * n) continue;
      const int j = r / n, i = r - j * n, blocks = lt_blocks<N, KEYS>(p, s, j);
      const int k0 = i * blocks / n, k1 = (i + 1) * blocks / n;  // blocks <= the cap's few thousand
      // a tile of fewer blocks than pieces begins at the first piece that has one
      const int head = k0 > 0 ? part - i + (n + blocks - 1) / blocks - 1 : -1;
      *reinterpret_cast<int4*>(s_share) = make_int4(b, j, k0, 0);
      *reinterpret_cast<int4*>(s_share + 4) =
          k1 == blocks ? make_int4(b, j + 1, 0, 0) : make_int4(b, j, k1, part - i + n - 1);
      *reinterpret_cast<int4*>(s_share + 8) = make_int4(raw.x, raw.y, raw.z, head);
    }
  } else if (tid < 2) {  // thread 0: the share's start, thread 1: its end
    // Where a share begins is a product of floats: it only has to be the
    // same for the CTAs on both sides and to rise with c, and exact
    // divisions, of 64-bit integers above all, cost as much as a key block.
    const int g = max(1, min(parts, int(__fdividef(float(total), float(p.H) * kLtMinShare))));
    const float each = __fdividef(float(total), float(g));  // a share's weight
    auto start = [&](int c) { return min(total - 1, int64_t(float(c) * each)); };
    const int c = part + tid;
    LtPos at{p.B, 0, 0};
    int last = -1;
    if (total > 0 && c < g) {
      const int64_t x = start(c);
      int lo = 0, hi = p.B;  // last b with s_scan[b] <= x
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (s_scan[mid] <= x) lo = mid; else hi = mid;
      }
      const int4 raw = s_seq[lo];
      const LtSeq s = lt_seq<N>(p, lo, raw.x, raw.y, raw.z);
      const int64_t y = x - s_scan[lo];
      int jl = 0, jh = s.tiles;  // last j with weight(j) <= y
      while (jh - jl > 1) {
        const int mid = (jl + jh) >> 1;
        if (lt_weight<N>(p, s, mid) <= y) jl = mid; else jh = mid;
      }
      const int64_t w0 = lt_weight<N>(p, s, jl), w1 = lt_weight<N>(p, s, jl + 1);
      const int blocks = lt_blocks<N, KEYS>(p, s, jl);
      at.b = lo;
      at.j = jl;
      at.k = min(blocks - 1, int(__fdividef(float(y - w0), float(w1 - w0)) * float(blocks)));
      // the last CTA whose share starts before this tile's end
      const int64_t e = s_scan[lo] + w1;
      last = max(c, min(g - 1, int(__fdividef(float(e), each))));
      while (last + 1 < g && start(last + 1) < e) ++last;
      while (last > c && start(last) >= e) --last;
      if (tid == 0) {
        *reinterpret_cast<int4*>(s_share + 8) = raw;
        // the CTA that has this tile's first block: the last one whose
        // share does not begin behind it
        int head = -1;
        if (at.k > 0) {
          const int64_t t0 = s_scan[lo] + w0;
          auto behind = [&](int h) {
            const int64_t v = start(h) - t0;
            return v > 0 && min(blocks - 1, int(__fdividef(float(v), float(w1 - w0)) * float(blocks))) > 0;
          };
          head = max(0, min(c - 1, int(__fdividef(float(t0), each))));
          while (head + 1 < c && !behind(head + 1)) ++head;
          while (head > 0 && behind(head)) --head;
        }
        s_share[11] = head;
      }
    } else if (tid == 0) {
      s_share[11] = -1;
    }
    s_share[tid * 4] = at.b;
    s_share[tid * 4 + 1] = at.j;
    s_share[tid * 4 + 2] = at.k;
    s_share[tid * 4 + 3] = last;
  }
  // the scan's words are rewritten by the copy engine
  fence_proxy_async_smem();
}

// Sequences of more than 64 rows, on pairs of CTAs (pkv_latent_pair.cu).
int launch_latent_pair(const LaunchCtx& ctx, const LatentAttendArgs& a, const LatentParams& lp);

}  // namespace pkv
