// page_walk.cuh -- how lbx_paged_attention shares out its work: tiles of a request's
// query rows, blocks of keys, one list of the blocks of all tiles cut into equal
// ranges, one per CTA (or pair).
//
// A tile is two or four subtiles of whole tokens, as many as fit 128 rows of G heads each.
// Its keys are the positions up to its last token's (all of a tree's), in blocks of
// 128; a chunk's tiles are as much longer as they stand later.  The list runs over
// (layer, KV head), request, tile, block; every tile begins with kLead blocks that
// stand for what beginning and ending it costs.  Range c starts at c * total / n: where
// that leaves a piece of fewer than kLeast blocks of a tile on either side, at the tile's
// edge.  All is derived from the requests' lengths by every CTA for itself; only
// the sums over the requests are shared.
#pragma once

#include "page_common.cuh"

namespace lbx {
namespace paged {

constexpr int kBlk = 128;   // keys per block (its logarithm, 7, stands in entries_upto)
constexpr int kRows = 128;  // rows per subtile
constexpr int kLead = 2, kLeast = 2;
constexpr int kMinRange = 3;  // entries of the list per CTA, at least

typedef long long i64;

// a / b of numbers that are not negative; in 32 bits where they fit (a 64-bit division
// takes hundreds of cycles).
__host__ __device__ inline i64 quot(i64 a, i64 b) {
  if (((a | b) >> 32) == 0) return (uint32_t)a / (uint32_t)b;
  return a / b;
}

struct Shape {
  int W;       // tokens per tile
  int period;  // tiles after which (position mod kBlk) repeats; a power of two
  int tree;
};

__host__ __device__ inline Shape shape_of(int G, int subtiles, bool tree) {
  Shape s;
  s.W = subtiles * (kRows / G);
  const int low = s.W & -s.W;  // gcd with kBlk, a power of two
  s.period = low >= kBlk ? 1 : kBlk / low;
  s.tree = tree;
  return s;
}

__host__ __device__ inline int tiles_of(const Shape &s, int n) { return (n + s.W - 1) / s.W; }

// Blocks of tile t of a request of ctx cached and n new tokens.
__host__ __device__ inline int blocks_of(const Shape &s, int ctx, int n, int t) {
  const i64 end = s.tree || (i64)(t + 1) * s.W >= n ? (i64)ctx + n : (i64)ctx + (i64)(t + 1) * s.W;
  return (int)((end + kBlk - 1) >> 7);
}

// Entries of the list of a request's first k tiles, none of them its last (unless k is
// all of them).  With x_i = c + i W the sum of floor(x_i / 128) over whole periods
// is (sum of x_i - sum of x_i mod 128) / 128, where the remainders of a period are
// c mod g, c mod g + g, .. (g = 128 / period); the rest is added one by one.
__host__ __device__ inline i64 entries_upto(const Shape &s, int ctx, int n, int k) {
  if (s.tree) return (i64)k * (kLead + blocks_of(s, ctx, n, 0));
  const int all = tiles_of(s, n), m = k < all ? k : all - 1;  // tiles that are not the last
  i64 sum = (i64)k * kLead;
  if (k >= all && all > 0) sum += blocks_of(s, ctx, n, all - 1);
  if (m <= 0) return sum;
  const uint32_t c = (uint32_t)ctx + s.W + kBlk - 1;  // (positions end at 2^30)
  const int whole = m & -s.period, g = kBlk / s.period;
  const i64 x = (i64)whole * c + (i64)whole * (whole - 1) / 2 * s.W;
  const i64 rest = (i64)whole * (c & (g - 1)) + (i64)whole * (g * (s.period - 1)) / 2;
  sum += (x - rest) >> 7;
#ifdef __CUDA_ARCH__
#pragma unroll 4
#endif
  for (int i = whole; i < m; ++i) sum += (c + (uint32_t)i * s.W) >> 7;
  return sum;
}

__host__ __device__ inline i64 entries_of(const Shape &s, int ctx, int n) {
  return n > 0 ? entries_upto(s, ctx, n, tiles_of(s, n)) : 0;
}

// How the list is cut: n ranges of `total` entries.
struct Cut {
  i64 total;
  int n;
  __host__ __device__ i64 at(int c) const { return quot((i64)c * total, n); }
  // the first boundary at or past x, and the last one at or before it
  __host__ __device__ int first(i64 x) const { return (int)quot(x * n + total - 1, total); }
  __host__ __device__ int last(i64 x) const { return (int)quot((x + 1) * n + total - 1, total) - 1; }
};

__host__ __device__ inline Cut cut_of(i64 total, int ctas) {
  const i64 n = quot(total, kMinRange);
  return {total, n < 1 ? 1 : n < ctas ? (int)n : ctas};
}

// A tile's share of range `me`, from `from` = cut.at(me) to `to` = cut.at(me + 1): its
// blocks, and the tile's pieces.  X: the tile's first entry, nb: its blocks.
struct Piece {
  int blk0, blk1;
  int pieces, mine, owner;  // owner: the range of the first piece
  bool last;                // the range ends in this tile
};
__host__ __device__ inline bool piece_of(const Cut &c, int me, i64 from, i64 to, i64 X, int nb,
                                         Piece &p) {
  const i64 lo = X + kLead + kLeast, hi = X + kLead + nb - kLeast;  // boundaries inside: lo..hi
  // the range ends before the tile, or goes to the tile's edge
  if (me + 1 < c.n && to < lo && to < X + kLead + nb) return false;
  const bool begins = me > 0 && from >= lo && from <= hi;
  p.last = me + 1 < c.n && to >= lo && to <= hi;
  p.blk0 = begins ? (int)(from - X - kLead) : 0;
  p.blk1 = p.last ? (int)(to - X - kLead) : nb;
  p.pieces = 1, p.mine = 0, p.owner = me;
  if (begins || p.last) {
    int a = c.first(lo), z = c.last(hi);
    if (a < 1) a = 1;
    if (z > c.n - 1) z = c.n - 1;
    p.pieces = z - a + 2, p.owner = a - 1, p.mine = me - p.owner;
  }
  return true;
}

}  // namespace paged
}  // namespace lbx
