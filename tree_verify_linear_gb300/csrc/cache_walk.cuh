// cache_walk.cuh -- how the tensor-core kernels of the cache operators share
// out the keys: units of 64 keys, blocks of units, one list of the blocks of
// all (request, layer, KV head) streams cut into one range per CTA.
#pragma once

#include <cuda.h>

#include "cache_common.cuh"

namespace lbx {
namespace cache {

constexpr int kUnit = 64;          // keys per unit
constexpr int kPiece = 16 * 1024;  // bytes per ring stage
constexpr int kMaxCtas = 160;      // largest grid
constexpr int kRows = 128;         // query rows per CTA
constexpr int kMaxGroup = 8;       // most row tiles that run side by side

// Row tiles of a stream: `sets` sets of up to `group` tiles each, a tile of one
// CTA's 128 rows, or of a pair's whole nodes (whose queries one tensor copy
// brings: G heads of 128 / G nodes per CTA).
struct Tiling {
  int rows, tiles, sets, group, ctas, per_cta;  // ctas: per tile; per_cta: rows
};
inline Tiling tiling(long long rows, int G, int dh) {
  Tiling t;
  t.rows = (int)rows;
  t.ctas = rows > kRows && dh >= 128 && G <= kRows ? 2 : 1;
  t.per_cta = t.ctas == 2 ? kRows / G * G : kRows;
  t.tiles = (int)((rows + t.ctas * t.per_cta - 1) / (t.ctas * t.per_cta));
  t.sets = (t.tiles + kMaxGroup - 1) / kMaxGroup;
  t.group = (t.tiles + t.sets - 1) / t.sets;
  return t;
}

struct AttnMaps {
  CUtensorMap k, v;    // (dh, Hkv, positions, layer x request), boxes of 64 columns
  CUtensorMap kt, vt;  // the tree's
  CUtensorMap q;       // (dh, Hq, nodes, lists), boxes of 64 columns of a pair's Q rows
};

// (dh, Hkv, len, lists) view of a [lists][len][Hkv][dh] array of 16-bit values;
// box: 64 columns of one head's `keys` consecutive positions.
bool encode_list(CUtensorMap *map, const void *base, const lbx_attn_cfg *c, int len, int lists,
                 int keys);
// SMs of the current device, at most kMaxCtas (0 if a CUDA call fails).
int grid_limit();

// A position in a ring of N stages and the parity of its round.
template <int N>
struct Ring {
  int st = 0;
  uint32_t ph = 0;
  __device__ __forceinline__ void step() {
    if (++st == N) st = 0, ph ^= 1u;
  }
};

// Division of a row number by the heads of a group: exact while row * G < 2^32.
struct PerGroup {
  uint64_t inv;  // 2^32 / G, rounded up
  __device__ __forceinline__ int node(int row) const {
    return (int)(((uint64_t)(uint32_t)row * inv) >> 32);
  }
};
inline PerGroup per_group(int G) { return {((1ull << 32) + (unsigned)G - 1) / (unsigned)G}; }

// The low k (0..64) bits.
__device__ __forceinline__ uint64_t low_bits(int k) {
  return k >= 64 ? ~0ull : k <= 0 ? 0ull : (1ull << k) - 1;
}

// Unit u of a key list (ctx, w0, s_eff, ns, nw of S): the position (or tree
// node) of its first key, whether it is the tree's, and how many of its keys any
// query sees.  A unit past the last is empty: a copy of it lies outside its
// array and fills in zeros.
template <class S>
__device__ __forceinline__ void unit_of(const S &s, bool prefix, int N, int u, int &start,
                                        bool &tree, int &cnt) {
  const int ns = s.ns, first_tree = ns + s.nw;
  tree = u >= first_tree && !prefix;
  if (u >= first_tree + (prefix ? 0 : 1)) {
    start = tree ? N : s.ctx, cnt = 0;
    return;
  }
  start = u < ns ? u * kUnit : tree ? 0 : s.w0 + (u - ns) * kUnit;
  const int end = u < ns ? s.s_eff : tree ? N : s.ctx;
  cnt = end - start < kUnit ? end - start : kUnit;
}

// Walks a CTA's range of the block list (blocks of BU units).  Used by whole
// warps, each lane alike; the CTAs of a pair walk alike.
// A stream also costs what it takes to begin and end it, LEAD blocks that come
// before its own in the list.  Where whole streams per group come out within
// Args::join blocks (the price of joining the pieces of a cut stream) of equal
// ranges, a stream counts as one entry of the list and is not cut.  Args also has
// the shapes: L, Hkv, N, n_req, fixed, window, n_sink, ctx_len and til.
template <int BU, int LEAD, class Args>
struct Walk {
  const Args &A;
  // the list's entries and how they are cut: `more` ranges of each + 1 entries,
  // then ranges of `each`; per_b_base: first entry of request b
  int total, groups, each, more, cg, x, x_end, per_b_base;
  int slot_in_group, b, nblk, ctx;
  bool uncut;
  // the current segment
  int l, h, set, tile, blk0, blk1;
  int first, last;  // its entries: of the stream's first and last block
  bool live;  // this CTA has a tile of the stream

  // units of a request's key list
  int w0, s_eff, ns, nw, units;

  __device__ __forceinline__ void plan(int len) {  // of length `len`
    ctx = len;
    w0 = A.window > 0 && len - A.window + 1 > 0 ? len - A.window + 1 : 0;
    s_eff = A.n_sink < w0 ? A.n_sink : w0;
    ns = (s_eff + kUnit - 1) / kUnit;
    nw = (len - w0 + kUnit - 1) / kUnit;
    units = ns + nw + (A.fixed > 0 ? 0 : 1);
    nblk = (units + BU - 1) / BU;
  }
  __device__ __forceinline__ int blocks_of(int req) {
    plan(A.fixed > 0 ? A.fixed : A.ctx_len[req]);
    return nblk;
  }
  // Streams per request; entries of each of the current request's in the list.
  __device__ __forceinline__ int streams() const { return A.L * A.Hkv * A.til.sets; }
  __device__ __forceinline__ int entries() const { return uncut ? 1 : nblk + LEAD; }

  __device__ __forceinline__ Walk(const Args &a, int lane) : A(a), uncut(false) {
    int sum = 0, most = 0;
#pragma unroll 1
    for (int r = lane; r < A.n_req; r += 32) {
      sum += blocks_of(r) + LEAD;
      most = nblk > most ? nblk : most;
    }
    sum = (int)__reduce_add_sync(0xffffffffu, (unsigned)sum);
    most = (int)__reduce_max_sync(0xffffffffu, (unsigned)most);
    total = sum * streams();
    groups = (int)(gridDim.x / (unsigned)(A.til.group * A.til.ctas));
    const long long all = (long long)streams() * A.n_req;
    uncut = (all + groups - 1) / groups * (most + LEAD) <= (total + groups - 1) / groups + A.join;
    if (uncut) total = (int)all;
    if (groups > total) groups = total;
    each = total / groups, more = total - each * groups;
    const int at = (int)blockIdx.x / A.til.ctas;
    cg = at / A.til.group;
    slot_in_group = at - cg * A.til.group;
    x = cg < groups ? begin_of(cg) : total;
    x_end = cg < groups ? begin_of(cg + 1) : total;
    // the request of entry x: 32 requests at a time
    b = 0, per_b_base = 0;
    if (x < x_end) {
#pragma unroll 1
      for (int r0 = 0;; r0 += 32) {
        int mine = 0;
        if (r0 + lane < A.n_req) blocks_of(r0 + lane), mine = entries() * streams();
        int upto = mine;
#pragma unroll 1
        for (int w = 1; w < 32; w <<= 1) {
          const int y = __shfl_up_sync(0xffffffffu, upto, w);
          if (lane >= w) upto += y;
        }
        const unsigned past = __ballot_sync(0xffffffffu, per_b_base + upto > x);
        if (past) {
          const int f = __ffs(past) - 1;
          b = r0 + f;
          per_b_base += __shfl_sync(0xffffffffu, upto - mine, f);
          break;
        }
        per_b_base += __shfl_sync(0xffffffffu, upto, 31);
      }
      blocks_of(b);
    }
  }

  // Take the next segment; false at the end of the range.
  __device__ __forceinline__ bool next() {
#pragma unroll 1
    while (x < x_end) {
#pragma unroll 1
      while (x - per_b_base >= entries() * streams()) {
        per_b_base += entries() * streams();
        blocks_of(++b);
      }
      const int in_b = x - per_b_base, s = in_b / entries(), at = x - (in_b - s * entries());
      const int lh = A.til.sets > 1 ? s / A.til.sets : s;
      set = s - lh * A.til.sets;
      l = lh / A.Hkv, h = lh - l * A.Hkv;
      first = uncut ? at : at + LEAD, last = uncut ? at : first + nblk - 1;
      blk0 = uncut || x < first ? 0 : x - first;
      blk1 = uncut || x_end > last ? nblk : x_end - first;
      x = at + entries();
      tile = set * A.til.group + slot_in_group;
      live = tile < A.til.tiles;
      if (blk1 > blk0) return true;  // else the range ends before the stream's blocks
    }
    return false;
  }
  __device__ __forceinline__ int begin_of(int g) const { return g * each + (g < more ? g : more); }
  __device__ __forceinline__ int owner(int at) const {
    const int big = more * (each + 1);
    return at < big ? at / (each + 1) : more + (at - big) / each;
  }
  __device__ __forceinline__ void unit(int u, int &start, bool &tree, int &cnt) const {
    unit_of(*this, A.fixed > 0, A.N, u, start, tree, cnt);
  }
};

}  // namespace cache
}  // namespace lbx
