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
  int4* joins;         // nullptr: nothing is cut, and the workspace is not touched
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
// On pairs of CTAs (N = 128) the first tile of a sequence weighs this much more:
// its pages come from HBM (8 % more a key over long sequences; later tiles find
// them in L2), and decode rows' tiles are cut almost always, which costs a pair
// four cache tiles' time.  64 decode rows of 128 heads 67.3 -> 64.7 us, 32
// drafts 54.5 -> 50.2, chunks beside decode rows 574 -> 565; 512 on every tile
// gives 64.8, 50.1 and 590, and on one CTA 128 and no more is best.
template <int N>
constexpr int kLtFirstCost = N == 128 ? 384 : 0;
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
  // (any int32 may stand there: no sum or difference of them before its bounds
  // are known; the host has checked that max_blocks * kPage is an int32)
  s.bad = q0 < 0 || q1 < q0 || q1 > p.T || L < 0 || q1 - q0 > L || L > p.max_blocks * kPage || (b == 0 && q0 != 0);
  s.q0 = q0;
  s.L = s.bad ? 0 : L;
  s.n = s.bad ? 0 : q1 - q0;
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
  return j * (int64_t(p.H) * (s.L - s.n + kLtTileCost)) + N * (j * (j + 1) / 2) +
         (j > 0 ? p.H * kLtFirstCost<N> : 0);
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

// A tile among the batch's weights: where it starts, its weight, its blocks.
struct LtTile {
  int64_t start, weight;
  int blocks;
  // the tile's key block at weight x
  __device__ __forceinline__ int block(int64_t x) const {
    return min(blocks - 1, int(__fdividef(float(x - start), float(weight)) * float(blocks)));
  }
};

// Equal shares of a batch's weight: `count` of them, share c starting at
// start(c).  Where that is, is a product of floats: it only has to be the same
// for the parts on both sides and to rise with c, and exact divisions, of
// 64-bit integers above all, cost as much as a key block.
struct LtShares {
  int64_t total;
  int count;
  float each;  // weight of a share
  __device__ __forceinline__ LtShares(int64_t total_, int H, int parts) {
    total = total_;
    count = max(1, min(parts, int(__fdividef(float(total_), float(H) * kLtMinShare))));
    each = __fdividef(float(total_), float(count));
  }
  __device__ __forceinline__ int64_t start(int c) const { return min(total - 1, int64_t(float(c) * each)); }
  // the last part, from c on, whose share starts before the tile's end
  __device__ __forceinline__ int last_before(int c, const LtTile& t) const {
    const int64_t e = t.start + t.weight;
    int last = max(c, min(count - 1, int(__fdividef(float(e), each))));
    while (last + 1 < count && start(last + 1) < e) ++last;
    while (last > c && start(last) >= e) --last;
    return last;
  }
  // the part that has the tile's first block, where c's share begins behind
  // it: the last one whose share does not
  __device__ __forceinline__ int head_of(int c, const LtTile& t) const {
    auto behind = [&](int h) { return start(h) > t.start && t.block(start(h)) > 0; };
    int head = max(0, min(c - 1, int(__fdividef(float(t.start), each))));
    while (head + 1 < c && !behind(head + 1)) ++head;
    while (head > 0 && behind(head)) --head;
    return head;
  }
};

// What the plan leaves in shared memory.
struct LtPlan {
  LtPos begin, end;     // of the share
  int own;              // key blocks a piece where tiles have parts of their own; 0: equal shares
  int last, head;       // of the tile that the share ends (begins) inside, the last (first) part with a piece
  int q0, q1, L;        // query_start_loc[b], [b + 1] and seq_lens[b] of sequence begin.b
  LtTile tile0, tile1;  // that begin and end are in (equal shares)
  int64_t total;
};
static_assert(sizeof(LtPlan) <= 128, "the plan's place in the kernels' shared memory");

// a / b, for a < 2^24 and b > 0: exact, and a quarter of an integer division.
__device__ __forceinline__ int lt_div(int a, int b) {
  const int q = int(__fdividef(float(a), float(b)));
  return q - (q * b > a) + ((q + 1) * b <= a);
}

// Sum over the threads before this one of their `v`, and over all of `v` and
// of `u`.  warp_only: over the first warp, which is alone here.
template <int THREADS>
__device__ __forceinline__ int64_t block_scan(int64_t v, int64_t u, bool warp_only, longlong2* s_wsum, longlong2& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int64_t incl = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t x = __shfl_up_sync(0xffffffffu, incl, o);
    u += __shfl_xor_sync(0xffffffffu, u, o);
    if (lane >= o) incl += x;
  }
  int64_t run = incl - v;
  if (warp_only) {
    total = make_longlong2(__shfl_sync(0xffffffffu, incl, 31), u);
    return run;
  }
  if (lane == 31) s_wsum[warp] = make_longlong2(incl, u);
  __syncthreads();
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

// The place at weight x, which is in sequence b, whose tiles start at `run`.
template <int N, int KEYS>
__device__ __forceinline__ LtPos lt_place(const LatentParams& p, int b, const LtSeq& s, int64_t run, int64_t x,
                                          LtTile& tile) {
  int lo = 0, hi = s.tiles;  // last tile that starts at or before x
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (run + lt_weight<N>(p, s, mid) <= x) lo = mid; else hi = mid;
  }
  LtTile t;
  t.start = run + lt_weight<N>(p, s, lo);
  t.weight = run + lt_weight<N>(p, s, lo + 1) - t.start;
  t.blocks = lt_blocks<N, KEYS>(p, s, lo);
  tile = t;
  return LtPos{b, lo, t.block(x)};
}

// The share of part `part` of `parts` (a CTA, or a pair of them).  Every one of
// the THREADS reads its sequences once and, after one scan, whichever thread
// owns the sequence that a bound falls into writes it down; the caller
// synchronises behind it.  s_wsum: 2 * THREADS / 32 words.
template <int N, int KEYS, int THREADS>
__device__ __forceinline__ void lt_plan(const LatentParams& p, int part, int parts, longlong2* s_wsum, LtPlan* plan) {
  const bool warp_only = p.B <= 32;  // a warp plans alone: no barrier
  if (warp_only && threadIdx.x >= 32) return;
  const int tid = threadIdx.x;
  const int per = (p.B + THREADS - 1) / THREADS;
  const int b0 = min(p.B, tid * per), b1 = min(p.B, b0 + per);
  // Tiles and key blocks of the batch ride along in one word, each capped far
  // above what the choice below looks at.
  int64_t weight = 0, tiles_of = 0, blocks_of = 0;
  for (int b = b0; b < b1; ++b) {
    const LtSeq s = lt_seq<N>(p, b);
    if (s.bad && part == 0) flag_status(p.status, PKV_STATUS_BAD_QUERY);
    weight += lt_weight<N>(p, s, s.tiles);
    tiles_of += s.tiles;
    blocks_of += int64_t(s.tiles) * ((s.L + KEYS - 1) / KEYS);
  }
  if (tid == 0) {
    plan->begin = plan->end = LtPos{p.B, 0, 0};
    plan->q0 = plan->q1 = plan->L = 0;
    plan->last = plan->head = -1;
  }
  constexpr int64_t cap = int64_t(1) << 20;
  longlong2 sums;
  int64_t run = block_scan<THREADS>(weight, (min(tiles_of, cap) << 32) | min(blocks_of, cap), warp_only, s_wsum,
                                    sums);
  const int64_t total = sums.x;
  const int tiles = int(sums.y >> 32), blocks_all = int(sums.y & 0xFFFFFFFF);
  // Few tiles: each has parts of its own, pieces of `own` key blocks, so that a
  // part has one piece and no tile is cut that need not be (four sequences of
  // up to 255 tokens: 16.3 -> 12.1 us).  The pieces fit the grid because
  // ceil(n / own) sums to no more than tiles + blocks / own.
  int own = 0;
  if (tiles > 0 && tiles < parts) {
    const float t = float(blocks_all) / float(parts - tiles);
    if (t <= float(kLtMostOwn / KEYS)) own = max(kLtLeastOwn / KEYS, int(ceilf(t)));
  }
  if (tid == 0) {
    plan->own = own;
    plan->total = total;
  }
  if (own > 0) {
    auto cuts = [&](const LtSeq& s) {  // pieces of a tile
      const int n = (s.L + KEYS - 1) / KEYS;
      return n <= 2 * own ? 1 : (n + own - 1) / own;
    };
    int64_t count = 0;
    for (int b = b0; b < b1; ++b) {
      const LtSeq s = lt_seq<N>(p, b);
      count += int64_t(s.tiles) * cuts(s);
    }
    int first = int(block_scan<THREADS>(count, 0, warp_only, s_wsum + THREADS / 32, sums));
    for (int b = b0; b < b1; ++b) {
      const LtSeq s = lt_seq<N>(p, b);
      const int n = cuts(s), r = part - first;
      first += s.tiles * n;
      if (r < 0 || r >= s.tiles * n) continue;
      // (r < parts, and blocks are at most kLtMostOwn / KEYS times the parts)
      const int j = lt_div(r, n), i = r - j * n, blocks = lt_blocks<N, KEYS>(p, s, j);
      const int k0 = lt_div(i * blocks, n), k1 = lt_div((i + 1) * blocks, n);
      plan->begin = LtPos{b, j, k0};
      plan->end = k1 == blocks ? LtPos{b, j + 1, 0} : LtPos{b, j, k1};
      plan->last = part - i + n - 1;
      // a tile of fewer blocks than pieces begins at the first piece that has one
      if (k0 > 0) plan->head = part - i + (n + blocks - 1) / blocks - 1;
      plan->q0 = s.q0;
      plan->q1 = s.q0 + s.n;
      plan->L = s.L;
    }
  } else if (total > 0) {
    const LtShares shares(total, p.H, parts);
    const int64_t x0 = shares.start(part), x1 = shares.start(part + 1);
    for (int b = b0; b < b1; ++b) {
      const LtSeq s = lt_seq<N>(p, b);
      const int64_t w = lt_weight<N>(p, s, s.tiles);
      if (part < shares.count && x0 >= run && x0 < run + w) {
        plan->begin = lt_place<N, KEYS>(p, b, s, run, x0, plan->tile0);
        plan->q0 = s.q0;
        plan->q1 = s.q0 + s.n;
        plan->L = s.L;
      }
      if (part + 1 < shares.count && x1 >= run && x1 < run + w)
        plan->end = lt_place<N, KEYS>(p, b, s, run, x1, plan->tile1);
      run += w;
    }
  }
}

// What the merge needs to know of a share (LatentParams::joins).  Not part of
// the plan: nothing waits for it.
template <int N>
__device__ __forceinline__ int4 lt_join(const LatentParams& p, const LtPlan& plan, int part, int parts) {
  const LtPos &begin = plan.begin, &end = plan.end;
  if (begin.b >= p.B) return make_int4(0, 0, 0, -1);
  int last = plan.last, head = plan.head;
  if (plan.own == 0) {
    const LtShares shares(plan.total, p.H, parts);
    if (end.b < p.B) last = shares.last_before(part, plan.tile1);
    if (begin.k > 0) head = shares.head_of(part, plan.tile0);
  }
  // its last tile is cut, and the tile's first block is in this share
  if (end.b < p.B && end.k > 0 &&
      (begin.b < end.b || (begin.b == end.b && (begin.j < end.j || (begin.j == end.j && begin.k == 0))))) {
    const LtSeq s = lt_seq<N>(p, end.b);
    return make_int4(s.q0 * p.H + end.j * N, min(N, s.rows - end.j * N), last, head);
  }
  return make_int4(0, 0, 0, head);
}

// Sequences of more than 64 rows, on pairs of CTAs (pkv_latent_pair.cu).
int launch_latent_pair(const LaunchCtx& ctx, const LatentAttendArgs& a, const LatentParams& lp);

}  // namespace pkv
