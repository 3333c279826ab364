// cache_attn.cuh -- attention over a bounded or shared KV cache on the tensor
// cores (sm_103a): the kernel behind lbx_window_attention and
// lbx_prefix_attention.
//
// A stream is one KV head of one layer over one key list, and the query rows
// that read it: a request's (node, head of the group) pairs over its visible
// cache and tree, or, for a shared prefix, the pairs of all requests over the
// prefix.  Rows come in tiles of 128 (the lanes of tensor memory).  Per block
// of 128 keys
//   S = Q K^T          tensor cores, operands in shared memory
//   softmax            online, two threads per row (64 keys each), base 2
//   O += P V           tensor cores, P from tensor memory
// The running reference of a row moves only when a block's maximum exceeds it
// by more than 2^8, so that O is rescaled rarely; the result is the same
// softmax taken from another reference.  Scores, sums, references and O are
// fp32.  P meets V in V's type.  In bf16 it goes as hi + lo, two products
// (2^-17 of a weight): with hi alone the weights' rounding (2^-8 each) would
// add as much error as the rounding of o to bf16, the only one left otherwise.
// In f16 a weight's rounding (2^-11) is as small as that of o in f16, and one
// product serves.
//
// The key list is cut into units of 64 keys from one array: the visible first
// positions before the window, the window, the tree's own keys.  A block is
// two units, one for each of the two threads of a row; the last block may
// have one.  All blocks of all streams form one list (request, layer, KV
// head, block), cut into equal ranges, one per CTA (or per group of CTAs, one
// for each row tile of the stream, which then read the same keys at the same
// time): one CTA per SM, whatever the lengths.  A range's streams that it does
// not cover whole leave partials (m, l, O) in the workspace, at most two per
// CTA, and the last CTA of a row tile to finish joins them.
//
// Per CTA: warps 0-7 softmax, warp 8 issues the MMAs, warp 9 the copies.  K
// and V arrive by TMA in 16 KB pieces (K: 128 keys x 64 columns; V: whole
// rows) through one ring, in the order the MMAs take them, so that all of the
// shared memory next to the Q tile keeps copies in flight.  S of a block and
// its P share one of two 128-column buffers.  Every wait is bounded; a CTA
// whose wait gives up reports LBX_ETIMEOUT, still counts itself in with empty
// partials, drains its copies and frees its tensor memory.
#pragma once

#include <cuda.h>

#include <type_traits>

#include "cache_common.cuh"
#include "cache_ptx.cuh"

namespace lbx {
namespace cache {

constexpr int kRows = 128;         // query rows per tile
constexpr int kUnit = 64;          // keys per unit
constexpr int kPiece = 16 * 1024;  // bytes per ring stage
constexpr int kMaxCtas = 160;      // largest grid (partials in the workspace)
constexpr int kMaxGroup = 8;       // most row tiles that run side by side
constexpr int kSoftmaxThreads = 256;
constexpr int kThreads = kSoftmaxThreads + 64;

// Row tiles of a stream: `sets` sets of up to `group` tiles each.
struct Tiling {
  int rows, tiles, sets, group;
};
inline Tiling tiling(long long rows) {
  Tiling t;
  t.rows = (int)rows;
  t.tiles = (int)((rows + kRows - 1) / kRows);
  t.sets = (t.tiles + kMaxGroup - 1) / kMaxGroup;
  t.group = (t.tiles + t.sets - 1) / t.sets;
  return t;
}

// Floats of one partial: m (base 2) and l per row, then O.
constexpr size_t part_floats(int dh) { return 2 * (size_t)kRows + (size_t)kRows * dh; }

struct AttnMaps {
  CUtensorMap k, v;    // (dh, Hkv, positions, layer x request), boxes of 64 columns
  CUtensorMap kt, vt;  // the tree's
};

struct AttnArgs {
  int L, Hq, Hkv, G;
  int n_req;      // key lists per (layer, KV head): requests, or 1 for the prefix
  int nodes;      // queries per key list and head: N, or all requests' N
  int fixed;      // length of every key list if > 0 (the prefix), else ctx_len
  int Bq, N, T;   // of the batch (its check, the trees)
  int window, n_sink;
  float scale_log2;
  Tiling til;
  const int32_t *ctx_len, *parent;
  const uint16_t *q;
  uint16_t *o;                 // results in the 16-bit type ...
  float *o32, *lse2;           // ... or normalised in fp32 with the base-2 lse (prefix)
  float *lse;                  // natural lse or NULL
  const float *x_o, *x_lse2;   // a prefix's results to join, or NULL
  float *part;
  unsigned int *counters;      // one per (stream, tile)
  int32_t *status;
};

template <int DH>
struct Lay {
  static constexpr int kAtoms = DH / 64;
  static constexpr int kQBytes = kRows * DH * 2;
  static constexpr int kStages = (227 * 1024 - 3072 - kQBytes) / kPiece;
  static constexpr int kVKeys = kPiece / (DH * 2);             // keys per V piece
  static constexpr int kVBox = kVKeys < kUnit ? kVKeys : kUnit;  // rows of a V box
  static constexpr int kVAtom = kVKeys * 128;                  // one 64-column atom of a V piece
  static constexpr int kSmemQ = 0;
  static constexpr int kSmemRing = kSmemQ + kQBytes;
  static constexpr int kSmemRed = kSmemRing + kStages * kPiece;  // float [2][2][128]
  static constexpr int kSmemAnc = kSmemRed + 4 * kRows * 4;      // uint64 [64]
  static constexpr int kSmemMisc = kSmemAnc + kMaxNodes * 8;     // int [8]
  static constexpr int kSmemBars = kSmemMisc + 32;
  static constexpr int kNBars = 2 * kStages + 8;  // full, empty, s[2], p[2], o[2], q, end
  static constexpr int kSmemTotal = kSmemBars + kNBars * 8;
  static_assert(kSmemTotal <= 227 * 1024 && kSmemRing % 1024 == 0, "shared memory");
  static constexpr uint32_t kColO = 0, kColS = 256, kTmemCols = 512;
};

// What joining the pieces of a cut stream costs, in blocks.
constexpr int kJoinBlocks = 3;

// Walks a CTA's range of the block list.  Used by whole warps, each lane alike.
// Where whole streams per group come out within kJoinBlocks of equal ranges of
// blocks, a stream counts as one entry of the list and is not cut.
struct Walk {
  const AttnArgs &A;
  long long total, groups, cg, x, x_end, per_b_base;  // per_b_base: first entry of request b
  bool uncut;
  int slot_in_group, b, nblk, ctx;
  // the current segment
  int l, h, set, tile, blk0, blk1;
  long long first;  // the stream's first entry
  bool live;        // this CTA has a tile of the stream

  // units of a request's key list
  int w0, s_eff, ns, nw, units;

  __device__ __forceinline__ void plan(int len) {  // of length `len`
    ctx = len;
    w0 = A.window > 0 && len - A.window + 1 > 0 ? len - A.window + 1 : 0;
    s_eff = A.n_sink < w0 ? A.n_sink : w0;
    ns = (s_eff + kUnit - 1) / kUnit;
    nw = (len - w0 + kUnit - 1) / kUnit;
    units = ns + nw + (A.fixed > 0 ? 0 : 1);
    nblk = (units + 1) / 2;
  }
  __device__ __forceinline__ int blocks_of(int req) {
    plan(A.fixed > 0 ? A.fixed : A.ctx_len[req]);
    return nblk;
  }
  __device__ __forceinline__ long long streams() const {
    return (long long)A.L * A.Hkv * A.til.sets;
  }

  // Entries of the current request's streams in the list, each.
  __device__ __forceinline__ int entries() const { return uncut ? 1 : nblk; }

  __device__ __forceinline__ Walk(const AttnArgs &a, int lane) : A(a), uncut(false) {
    long long sum = 0;
    int most = 0;
    for (int r = lane; r < A.n_req; r += 32) {
      sum += blocks_of(r);
      most = nblk > most ? nblk : most;
    }
    for (int w = 16; w; w >>= 1) {
      sum += __shfl_xor_sync(0xffffffffu, sum, w);
      const int y = __shfl_xor_sync(0xffffffffu, most, w);
      most = y > most ? y : most;
    }
    total = sum * streams();
    groups = (long long)gridDim.x / A.til.group;
    const long long all = streams() * A.n_req;
    uncut = (all + groups - 1) / groups * most <= (total + groups - 1) / groups + kJoinBlocks;
    if (uncut) total = all;
    if (groups > total) groups = total;
    cg = blockIdx.x / A.til.group;
    slot_in_group = (int)(blockIdx.x - cg * A.til.group);
    x = cg < groups ? total * cg / groups : total;
    x_end = cg < groups ? total * (cg + 1) / groups : total;
    // the request of block x: 32 requests at a time
    b = 0, per_b_base = 0;
    if (x < x_end) {
      for (int r0 = 0;; r0 += 32) {
        long long mine = 0;
        if (r0 + lane < A.n_req) blocks_of(r0 + lane), mine = entries() * streams();
        long long upto = mine;
        for (int w = 1; w < 32; w <<= 1) {
          const long long y = __shfl_up_sync(0xffffffffu, upto, w);
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
    if (x >= x_end) return false;
    while (x - per_b_base >= entries() * streams()) {
      per_b_base += entries() * streams();
      blocks_of(++b);
    }
    const long long in_b = x - per_b_base, s = in_b / entries();
    blk0 = (int)(in_b - s * entries());
    first = x - blk0;
    set = (int)(s % A.til.sets);
    const int lh = (int)(s / A.til.sets);
    l = lh / A.Hkv, h = lh - l * A.Hkv;
    blk1 = uncut || x_end - first >= nblk ? nblk : (int)(x_end - first);
    x = uncut ? x + 1 : first + blk1;
    tile = set * A.til.group + slot_in_group;
    live = tile < A.til.tiles;
    return true;
  }
  __device__ __forceinline__ long long begin_of(long long g) const { return total * g / groups; }
  __device__ __forceinline__ long long owner(long long at) const {
    return ((at + 1) * groups - 1) / total;
  }
  __device__ __forceinline__ int units_in(int blk) const { return 2 * blk + 1 < units ? 2 : 1; }
  // Unit u: the position (or tree node) of its first key, whether it is the
  // tree's, and how many of its keys any query sees.
  __device__ __forceinline__ void unit(int u, int &start, bool &tree, int &cnt) const {
    tree = u >= ns + nw;
    start = u < ns ? u * kUnit : tree ? 0 : w0 + (u - ns) * kUnit;
    const int end = u < ns ? s_eff : tree ? A.N : ctx;
    cnt = end - start < kUnit ? end - start : kUnit;
  }
};

// The low k (0..64) bits.
__device__ __forceinline__ uint64_t low_bits(int k) {
  return k >= 64 ? ~0ull : k <= 0 ? 0ull : (1ull << k) - 1;
}

// Parts of P: f16 once, bf16 hi + lo.
template <bool F16>
constexpr int kParts = F16 ? 1 : 2;

template <bool F16>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  if constexpr (F16) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
  } else {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
  }
}

template <int DH, bool F16>
__global__ void __launch_bounds__(kThreads, 1)
    cache_attn_kernel(const __grid_constant__ AttnMaps maps, const __grid_constant__ AttnArgs A) {
  using Y = Lay<DH>;
  extern __shared__ __align__(1024) unsigned char cache_smem[];
  unsigned char *smem = cache_smem;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  float *red = reinterpret_cast<float *>(smem + Y::kSmemRed);
  uint64_t *anc = reinterpret_cast<uint64_t *>(smem + Y::kSmemAnc);
  // [0] tensor memory base, [1] last of its row tile, [2] a wait gave up
  volatile int *misc = reinterpret_cast<volatile int *>(smem + Y::kSmemMisc);
  uint64_t *full = reinterpret_cast<uint64_t *>(smem + Y::kSmemBars);
  uint64_t *empty = full + Y::kStages, *s_bar = empty + Y::kStages, *p_bar = s_bar + 2;
  uint64_t *o_bar = p_bar + 2, *q_bar = o_bar + 2, *end_bar = q_bar + 1;

  if (batch_bad(A.Bq, A.N, A.T, A.ctx_len, A.parent, nullptr)) {
    if (tid == 0 && A.status) *A.status = LBX_ETREE;
    return;
  }
  if (tid == 0) {
    for (int i = 0; i < Y::kNBars; ++i)
      ptx::mbar_init(full + i, full + i == p_bar || full + i == p_bar + 1 || full + i == q_bar
                                   ? kSoftmaxThreads / 32
                                   : 1);
    ptx::fence_mbar_init();
    misc[2] = 0;
  }
  if (warp == 8) {
    ptx::tmem_alloc(reinterpret_cast<uint32_t *>(smem + Y::kSmemMisc), Y::kTmemCols);
    ptx::tmem_relinquish();
    ptx::tc_fence_before();
  }
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = static_cast<uint32_t>(misc[0]);

  Walk W(A, lane);
  bool bad = false;  // a wait of this thread gave up: it waits no more
  auto wait = [&](uint64_t *bar, uint32_t parity) {
    if (!bad && !ptx::mbar_wait(bar, parity)) bad = true;
    return !bad;
  };
  // V pieces of a block with nu units
  auto v_pieces = [](int nu) { return (nu * kUnit + Y::kVKeys - 1) / Y::kVKeys; };

  if (warp == 9) {
    // ---- copies ----
    long long piece = 0;  // ring position
    while (W.next()) {
      if (!W.live) continue;
      const int nb = W.blk1 - W.blk0;
      const int z = A.fixed > 0 ? W.l : W.l * A.n_req + W.b;
      auto take = [&](uint32_t bytes) -> unsigned char * {
        const int st = (int)(piece % Y::kStages);
        if (piece >= Y::kStages &&
            !wait(&empty[st], (uint32_t)((piece / Y::kStages - 1) & 1)))
          return nullptr;
        ptx::mbar_arrive_expect_tx(&full[st], bytes);
        return smem + Y::kSmemRing + st * kPiece;
      };
      for (int i = 0; i <= nb && !bad && lane == 0; ++i) {
        if (i < nb) {  // K of block i
          const int blk = W.blk0 + i, nu = W.units_in(blk);
          for (int a = 0; a < Y::kAtoms && !bad; ++a) {
            unsigned char *d = take((uint32_t)(nu * kUnit * 128));
            if (!d) break;
            for (int u = 0; u < nu; ++u) {
              int start, cnt;
              bool tree;
              W.unit(2 * blk + u, start, tree, cnt);
              ptx::tma_load_4d(d + u * kUnit * 128, tree ? &maps.kt : &maps.k, a * 64, W.h, start, z,
                               &full[piece % Y::kStages]);
            }
            ++piece;
          }
        }
        if (i > 0 && !bad) {  // V of block i - 1
          const int blk = W.blk0 + i - 1, nu = W.units_in(blk);
          for (int c = 0; c < v_pieces(nu) && !bad; ++c) {
            const int keys = nu * kUnit - c * Y::kVKeys < Y::kVKeys ? nu * kUnit - c * Y::kVKeys
                                                                    : Y::kVKeys;
            unsigned char *d = take((uint32_t)(keys * DH * 2));
            if (!d) break;
            for (int k0 = 0; k0 < keys; k0 += Y::kVBox) {
              const int kk = c * Y::kVKeys + k0;
              int start, cnt;
              bool tree;
              W.unit(2 * blk + kk / kUnit, start, tree, cnt);
              for (int a = 0; a < Y::kAtoms; ++a)
                ptx::tma_load_4d(d + a * Y::kVAtom + k0 * 128, tree ? &maps.vt : &maps.v, a * 64,
                                 W.h, start + kk % kUnit, z, &full[piece % Y::kStages]);
            }
            ++piece;
          }
        }
      }
    }
    if (lane == 0) {
      if (bad) misc[2] = 1;
      // every copy has landed before the CTA may leave (long since, unless a
      // wait gave up)
      bad = false;
      for (long long i = piece > Y::kStages ? piece - Y::kStages : 0; i < piece; ++i)
        (void)ptx::mbar_wait(&full[i % Y::kStages], (uint32_t)((i / Y::kStages) & 1));
    }
  } else if (warp == 8) {
    // ---- MMAs ----
    long long piece = 0, q = 0;
    int seg = 0;
    const uint64_t qdesc = ptx::sdesc_sw128(ptx::smem_u32(smem + Y::kSmemQ));
    const uint64_t kdesc = ptx::sdesc_sw128(ptx::smem_u32(smem + Y::kSmemRing));
    const uint64_t vdesc =
        ptx::sdesc(ptx::smem_u32(smem + Y::kSmemRing), (uint32_t)Y::kVAtom, 1024u, 2u);
    bool issued = false;
    while (W.next()) {
      if (!W.live) continue;
      const int nb = W.blk1 - W.blk0;
      // S of block i into buffer (q + i) & 1
      auto scores = [&](int i) {
        const long long qi = q + i;
        const int nu = W.units_in(W.blk0 + i);
        // the buffer's last P has been multiplied
        if (qi >= 2 && !wait(&o_bar[qi & 1], (uint32_t)(((qi - 2) >> 1) & 1))) return;
        const uint32_t idesc = ptx::idesc_16(F16, kRows, nu * kUnit, false);
        const uint32_t d = tmem + Y::kColS + (uint32_t)(qi & 1) * 128;
        for (int a = 0; a < Y::kAtoms; ++a, ++piece) {
          const int st = (int)(piece % Y::kStages);
          if (!wait(&full[st], (uint32_t)((piece / Y::kStages) & 1))) return;
          ptx::tc_fence_after();
          const uint64_t kd = kdesc + (uint64_t)(st * kPiece >> 4);
          const uint64_t qd = qdesc + (uint64_t)(a * kRows * 128 >> 4);
#pragma unroll
          for (int ks = 0; ks < 4; ++ks)
            ptx::mma_bf16_ss(d, qd + 2 * ks, kd + 2 * ks, idesc, a + ks > 0 ? 1u : 0u);
          ptx::mma_commit(&empty[st]);
        }
        ptx::mma_commit(&s_bar[qi & 1]);
      };
      if (lane == 0) {
        issued = true;
        if (wait(q_bar, (uint32_t)(seg & 1))) scores(0);
        for (int i = 0; i < nb && !bad; ++i) {
          if (i + 1 < nb) scores(i + 1);
          const long long qi = q + i;
          if (!wait(&p_bar[qi & 1], (uint32_t)((qi >> 1) & 1))) break;
          ptx::tc_fence_after();
          const int nu = W.units_in(W.blk0 + i);
          constexpr uint32_t idesc = ptx::idesc_16(F16, kRows, DH, true);
          const uint32_t pc = tmem + Y::kColS + (uint32_t)(qi & 1) * 128;
          for (int c = 0; c < v_pieces(nu); ++c, ++piece) {
            const int st = (int)(piece % Y::kStages);
            if (!wait(&full[st], (uint32_t)((piece / Y::kStages) & 1))) break;
            ptx::tc_fence_after();
            const int keys = nu * kUnit - c * Y::kVKeys < Y::kVKeys ? nu * kUnit - c * Y::kVKeys
                                                                    : Y::kVKeys;
            const uint64_t vd = vdesc + (uint64_t)(st * kPiece >> 4);
            for (int part = 0; part < kParts<F16>; ++part)
              for (int ks = 0; ks < keys / 16; ++ks)
                ptx::mma_bf16_ts(tmem + Y::kColO,
                                 pc + (uint32_t)(part * 64 + c * Y::kVKeys / 2 + ks * 8),
                                 vd + (uint64_t)(ks * 2048 >> 4), idesc,
                                 i + c + part + ks > 0 ? 1u : 0u);
            ptx::mma_commit(&empty[st]);
          }
          ptx::mma_commit(&o_bar[qi & 1]);
        }
      }
      q += nb;
      ++seg;
      if (__shfl_sync(0xffffffffu, (int)bad, 0)) break;
    }
    if (lane == 0 && issued) {
      if (bad) misc[2] = 1;
      ptx::mma_commit(end_bar);
      (void)ptx::mbar_wait(end_bar, 0);
    }
  } else {
    // ---- softmax ----
    const int quad = warp & 3, hf = warp >> 2;
    const uint32_t tq = tmem + ((uint32_t)(quad * 32) << 16);
    const int r = quad * 32 + lane;  // row of the tile
    const float sl2 = A.scale_log2;
    constexpr int kHalf = DH / 2;
    long long q = 0, piece = 0;
    int req = -1;

    // The Q tile of the walk's segment, rows past the stream's zero: a warp
    // per row, 16 bytes per lane, in the swizzled layout of the MMA's operand.
    auto load_q = [&]() {
      constexpr int kPer = DH / 8;  // 16-byte pieces per row
      constexpr int kStep = kSoftmaxThreads / kPer;
      for (int rr = tid / kPer; rr < kRows; rr += kStep) {
        const int row = W.tile * kRows + rr, c = tid % kPer;
        uint4 v = make_uint4(0u, 0u, 0u, 0u);
        if (row < A.til.rows) {
          const int node = row / A.G, hd = row - node * A.G;
          const size_t at = ((size_t)W.l * A.n_req + W.b) * A.nodes + node;
          v = reinterpret_cast<const uint4 *>(A.q)[(at * A.Hq + W.h * A.G + hd) * kPer + c];
        }
        *reinterpret_cast<uint4 *>(smem + Y::kSmemQ + (c / 8) * kRows * 128 + rr * 128 +
                                   ((c & 7) ^ (rr & 7)) * 16) = v;
      }
      ptx::fence_proxy_async();
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(q_bar);
    };
    // The next segment with a tile for this CTA.
    auto advance = [&]() {
      while (W.next())
        if (W.live) return true;
      return false;
    };

    bool have = advance();
    if (have) load_q();
    while (have) {
      const int l = W.l, b = W.b, h = W.h, tile = W.tile, blk0 = W.blk0, blk1 = W.blk1;
      const int nb = blk1 - blk0, ctx = W.ctx;
      const long long first = W.first;
      const int row = tile * kRows + r;
      const bool real = row < A.til.rows;
      const int node = real ? row / A.G : 0;
      // ancestor masks of the request's tree, by doubling
      if (A.fixed <= 0 && b != req) {
        ptx::named_sync(5, kSoftmaxThreads);  // the last request's masks are read
        if (tid < 32) {
          uint64_t m[2];
          int up[2];
          for (int e = 0; e < 2; ++e) {
            const int n = lane + 32 * e;
            up[e] = n < A.N ? A.parent[(size_t)b * A.N + n] : -1;
            m[e] = 1ull << n;
            anc[n] = m[e];
          }
          int *ups = reinterpret_cast<int *>(red);  // not in use between segments
          for (int e = 0; e < 2; ++e) ups[lane + 32 * e] = up[e];
          __syncwarp();
          for (int step = 0; step < 6; ++step) {
            uint64_t add[2];
            int nu[2];
            for (int e = 0; e < 2; ++e) {
              add[e] = up[e] >= 0 ? anc[up[e]] : 0ull;
              nu[e] = up[e] >= 0 ? ups[up[e]] : -1;
            }
            __syncwarp();
            for (int e = 0; e < 2; ++e) {
              m[e] |= add[e], up[e] = nu[e];
              anc[lane + 32 * e] = m[e], ups[lane + 32 * e] = up[e];
            }
            __syncwarp();
          }
        }
        ptx::named_sync(5, kSoftmaxThreads);
        req = b;
      }
      // what this row sees: of the tree as bits, of the cache from lo on
      uint64_t tree_bits = 0;
      int lo = 0;
      if (A.fixed <= 0 && real) {
        tree_bits = anc[node];
        if (A.window > 0) {
          lo = ctx + __popcll(tree_bits) - A.window;  // ctx + depth - window + 1
          uint64_t m = tree_bits;
          for (int pos = ctx; m; ++pos, m &= m - 1)  // nodes of the path, root first
            if (pos < lo && pos >= A.n_sink) tree_bits &= ~(m & (0 - m));
        }
      }

      float m_run = -INFINITY, l_run = 0.f;  // the row's reference (raw); this half's sum
      long long v_piece = 0;                 // ring position of the block's V
      for (int i = 0; i < nb; ++i) {
        const long long qi = q + i;
        const int nu = W.units_in(blk0 + i);
        v_piece = piece + (long long)Y::kAtoms * (i + 1 < nb ? i + 2 : nb) + i * v_pieces(2);
        wait(&s_bar[qi & 1], (uint32_t)((qi >> 1) & 1));
        ptx::tc_fence_after();
        const bool has = hf < nu;  // this half's unit
        float sv[64], mh = -INFINITY;
        const uint32_t sc = tq + Y::kColS + (uint32_t)(qi & 1) * 128;
        if (has) {
          ptx::tmem_ld32(sc + hf * 64, *reinterpret_cast<float(*)[32]>(sv));
          ptx::tmem_ld32(sc + hf * 64 + 32, *reinterpret_cast<float(*)[32]>(sv + 32));
          int start, cnt;
          bool tree;
          W.unit(2 * (blk0 + i) + hf, start, tree, cnt);
          const uint64_t ok = tree ? tree_bits
                                   : low_bits(cnt) & (~low_bits(lo - start) |
                                                      low_bits(A.n_sink - start));
          // values no query sees must not reach O through a zero weight
          if (!tree && cnt < kUnit) {
            // the stage's earlier V has been multiplied, so that its barrier is
            // in the phase that ends with this one's arrival
            if (i > 0) wait(&o_bar[(qi - 1) & 1], (uint32_t)(((qi - 1) >> 1) & 1));
            const int gone = kUnit - cnt;
            for (int idx = tid & 127; idx < gone * (DH / 8); idx += 128) {
              const int key = cnt + idx / (DH / 8), c = idx % (DH / 8);
              const int at = hf * kUnit + key;
              const long long pc = v_piece + at / Y::kVKeys;
              const int st = (int)(pc % Y::kStages);
              wait(&full[st], (uint32_t)((pc / Y::kStages) & 1));
              *reinterpret_cast<uint4 *>(smem + Y::kSmemRing + st * kPiece + (c / 8) * Y::kVAtom +
                                         (at % Y::kVKeys) * 128 + (c & 7) * 16) =
                  make_uint4(0u, 0u, 0u, 0u);
            }
            ptx::fence_proxy_async();
          }
          ptx::tmem_wait_ld();
          if (!__all_sync(0xffffffffu, ok == ~0ull)) {
            const uint32_t ok0 = (uint32_t)ok, ok1 = (uint32_t)(ok >> 32);
#pragma unroll
            for (int e = 0; e < 32; ++e) {
              if (!(ok0 >> e & 1)) sv[e] = -INFINITY;
              if (!(ok1 >> e & 1)) sv[32 + e] = -INFINITY;
            }
          }
          float mx[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) mx[e] = sv[e];
#pragma unroll
          for (int e = 8; e < 64; ++e) mx[e & 7] = fmaxf(mx[e & 7], sv[e]);
          mh = fmaxf(fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])),
                     fmaxf(fmaxf(mx[4], mx[5]), fmaxf(mx[6], mx[7])));
        }
        // (two buffers: the other half may not have read the last block's yet)
        float *max_of = red + (int)(qi & 1) * 2 * kRows;
        max_of[hf * kRows + r] = mh;
        ptx::tc_fence_before();
        ptx::named_sync(1 + quad, 64);  // the row's other half: maxima out, scores read
        ptx::tc_fence_after();
        const float mb = fmaxf(mh, max_of[(1 - hf) * kRows + r]);
        float alpha = 1.f;
        bool need = false;
        if ((mb - m_run) * sl2 > 8.f) {  // the first time too
          alpha = ptx::ex2((m_run - mb) * sl2);
          need = i > 0;
          l_run *= alpha;
          m_run = mb;
        }
        const float ref = m_run == -INFINITY ? 0.f : m_run * sl2;
        if (has) {
          float sum[4] = {0.f, 0.f, 0.f, 0.f};
          uint32_t pk[32];
#pragma unroll
          for (int e = 0; e < 32; ++e) {
            const float p0 = ptx::ex2(fmaf(sv[2 * e], sl2, -ref));
            const float p1 = ptx::ex2(fmaf(sv[2 * e + 1], sl2, -ref));
            sum[e & 3] += p0 + p1;
            pk[e] = pack2<F16>(p0, p1);
            if constexpr (!F16) {  // what bf16 leaves of the weights
              sv[2 * e] = p0 - __uint_as_float(pk[e] << 16);
              sv[2 * e + 1] = p1 - __uint_as_float(pk[e] & 0xffff0000u);
            }
          }
          l_run += (sum[0] + sum[1]) + (sum[2] + sum[3]);
          ptx::tmem_st32(sc + hf * 32, pk);
          if constexpr (!F16) {
#pragma unroll
            for (int e = 0; e < 32; ++e) pk[e] = pack2<false>(sv[2 * e], sv[2 * e + 1]);
            ptx::tmem_st32(sc + 64 + hf * 32, pk);
          }
        }
        // rows whose reference moved rescale their half of O's columns, once
        // the previous product is done
        if (__any_sync(0xffffffffu, need)) {
          wait(&o_bar[(qi - 1) & 1], (uint32_t)(((qi - 1) >> 1) & 1));
          ptx::tc_fence_after();
#pragma unroll 1
          for (int c = 0; c < kHalf / 32; ++c) {
            const uint32_t col = tq + Y::kColO + (uint32_t)(hf * kHalf + 32 * c);
            float ov[32];
            ptx::tmem_ld32(col, ov);
            ptx::tmem_wait_ld();
            uint32_t w[32];
#pragma unroll
            for (int e = 0; e < 32; ++e) w[e] = __float_as_uint(ov[e] * alpha);
            ptx::tmem_st32(col, w);
          }
        }
        ptx::tmem_wait_st();
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(&p_bar[qi & 1]);
      }
      piece = v_piece + v_pieces(W.units_in(blk1 - 1));
      q += nb;
      // the next Q tile goes in while the last product runs: every score
      // product of this segment is done
      const long long c_first = W.owner(first), c_last = W.owner(first + W.entries() - 1);
      const int set = W.set;
      have = advance();
      if (have) load_q();

      // ---- this segment's result: whole, or a partial ----
      wait(&o_bar[(q - 1) & 1], (uint32_t)(((q - 1) >> 1) & 1));
      ptx::tc_fence_after();
      ptx::named_sync(1 + quad, 64);  // the last maxima are read
      red[hf * kRows + r] = l_run;
      if (bad) misc[2] = 1;
      ptx::named_sync(5, kSoftmaxThreads);
      const bool valid = misc[2] == 0;
      float l_sum = red[r] + red[kRows + r], m2 = m_run == -INFINITY ? -INFINITY : m_run * sl2;
      if (!valid) l_sum = 0.f, m2 = -INFINITY;
      // Write C columns of a finished row (its place among all queries), joined
      // with the prefix's if there is one.
      auto emit = [&](auto width, size_t at, int col, const float *acc, float m, float sum) {
        constexpr int C = decltype(width)::value;
        const float own = sum > 0.f ? m + log2f(sum) : -INFINITY;
        float all = own, w = sum > 0.f ? 1.f / sum : 0.f;
        float v[C];
        if (A.x_o) {
          float4 f[C / 4];
          const float4 *xo = reinterpret_cast<const float4 *>(A.x_o + at * DH + col);
#pragma unroll
          for (int e = 0; e < C / 4; ++e) f[e] = __ldcg(xo + e);
          const float x = __ldcg(A.x_lse2 + at), top = fmaxf(own, x);
          float wx = 0.f;
          if (top != -INFINITY) {
            const float eo = exp2f(own - top), ex = exp2f(x - top), inv = 1.f / (eo + ex);
            w *= eo * inv, wx = ex * inv;
            all = top + log2f(eo + ex);
          }
#pragma unroll
          for (int e = 0; e < C / 4; ++e) {
            v[4 * e] = fmaf(acc[4 * e], w, wx * f[e].x);
            v[4 * e + 1] = fmaf(acc[4 * e + 1], w, wx * f[e].y);
            v[4 * e + 2] = fmaf(acc[4 * e + 2], w, wx * f[e].z);
            v[4 * e + 3] = fmaf(acc[4 * e + 3], w, wx * f[e].w);
          }
        } else {
#pragma unroll
          for (int e = 0; e < C; ++e) v[e] = acc[e] * w;
        }
        if (A.o32) {
          float4 *to = reinterpret_cast<float4 *>(A.o32 + at * DH + col);
#pragma unroll
          for (int e = 0; e < C / 4; ++e)
            to[e] = make_float4(v[4 * e], v[4 * e + 1], v[4 * e + 2], v[4 * e + 3]);
        } else {
          uint2 *to = reinterpret_cast<uint2 *>(A.o + at * DH + col);
#pragma unroll
          for (int e = 0; e < C / 4; ++e)
            to[e] = make_uint2(pack2<F16>(v[4 * e], v[4 * e + 1]),
                               pack2<F16>(v[4 * e + 2], v[4 * e + 3]));
        }
        if (col == 0) {
          if (A.lse2) A.lse2[at] = all;
          if (A.lse) A.lse[at] = all * 0.6931471805599453f;
        }
      };
      // The place among all queries of a row of the stream.
      auto place = [&](int rw) {
        const int nd = rw / A.G;
        return (((size_t)l * A.n_req + b) * A.nodes + nd) * A.Hq + h * A.G + (rw - nd * A.G);
      };
      const bool whole = c_first == c_last;
      // this CTA's partial: its first segment's, or its last's
      float *pp = A.part + ((size_t)blockIdx.x * 2 + (W.begin_of(W.cg) >= first ? 0 : 1)) *
                               part_floats(DH);
      if (quad * 32 < A.til.rows - tile * kRows && (whole || valid)) {
#pragma unroll 1
        for (int c = 0; c < kHalf / 32; ++c) {
          const int col = hf * kHalf + 32 * c;
          float ov[32];
          ptx::tmem_ld32(tq + Y::kColO + (uint32_t)col, ov);
          ptx::tmem_wait_ld();
          if (!real) continue;
          if (whole) {
            if (valid) emit(std::integral_constant<int, 32>{}, place(row), col, ov, m2, l_sum);
          } else {
            float4 *to = reinterpret_cast<float4 *>(pp + 2 * kRows + (size_t)r * DH + col);
#pragma unroll
            for (int e = 0; e < 8; ++e)
              to[e] = make_float4(ov[4 * e], ov[4 * e + 1], ov[4 * e + 2], ov[4 * e + 3]);
          }
        }
      }
      if (!whole) {
        if (real && hf == 0) pp[r] = m2, pp[kRows + r] = l_sum;
        __threadfence();
        ptx::named_sync(5, kSoftmaxThreads);
        const size_t counter =
            (((size_t)b * A.L + l) * A.Hkv + h) * A.til.tiles + tile;
        if (tid == 0) {
          const unsigned prev = atomicAdd(&A.counters[counter], 1u);
          misc[1] = (long long)prev == c_last - c_first ? 1 : 0;
          if (misc[1]) A.counters[counter] = 0u;  // for the next call
        }
        ptx::named_sync(5, kSoftmaxThreads);
        // the last CTA joins the pieces: four columns of a row per thread, the
        // pieces' m, l and O of up to eight of them in flight at a time
        // the last CTA joins the pieces: four columns of a row per thread, eight
        // loads of O in flight (of several rows where there are few pieces)
        if (misc[1]) {
          __threadfence();
          const int rows = A.til.rows - tile * kRows < kRows ? A.til.rows - tile * kRows : kRows;
          const int lane_of = tile - set * A.til.group, n_piece = (int)(c_last - c_first) + 1;
          // only a stream's first piece may not be its CTA's first
          const int slot0 = W.begin_of(c_first) < first ? 1 : 0;
          auto join = [&](auto per) {
            constexpr int PP = decltype(per)::value, II = 8 / PP;  // pieces, items at a time
            for (int idx0 = tid; idx0 < rows * (DH / 4); idx0 += II * kSoftmaxThreads) {
              float top[II], sum[II], acc[II][4];
              size_t at[II];  // of the item in a partial's O
#pragma unroll
              for (int i = 0; i < II; ++i) {
                const int idx = idx0 + i * kSoftmaxThreads;
                at[i] = (size_t)(idx < rows * (DH / 4) ? idx : idx0);
                top[i] = -INFINITY, sum[i] = 0.f;
                acc[i][0] = acc[i][1] = acc[i][2] = acc[i][3] = 0.f;
              }
              for (int g0 = 0; g0 < n_piece; g0 += PP) {
                float mg[II][PP], lg[II][PP];
                float4 og[II][PP];
#pragma unroll
                for (int e = 0; e < PP; ++e) {
                  const int g = g0 + e < n_piece ? g0 + e : 0;
                  const float *pg =
                      A.part + ((size_t)((c_first + g) * A.til.group + lane_of) * 2 +
                                (g == 0 ? slot0 : 0)) * part_floats(DH);
#pragma unroll
                  for (int i = 0; i < II; ++i) {
                    const int rr = (int)(at[i] / (DH / 4));
                    mg[i][e] = g0 + e < n_piece ? __ldcg(pg + rr) : -INFINITY;
                    lg[i][e] = __ldcg(pg + kRows + rr);
                    og[i][e] = __ldcg(reinterpret_cast<const float4 *>(pg + 2 * kRows) + at[i]);
                  }
                }
#pragma unroll
                for (int i = 0; i < II; ++i) {
                  float t8 = top[i];
#pragma unroll
                  for (int e = 0; e < PP; ++e) t8 = fmaxf(t8, mg[i][e]);
                  if (t8 == -INFINITY) continue;
                  const float old = ptx::ex2(top[i] - t8);
                  top[i] = t8, sum[i] *= old;
#pragma unroll
                  for (int e = 0; e < 4; ++e) acc[i][e] *= old;
#pragma unroll
                  for (int e = 0; e < PP; ++e) {
                    if (mg[i][e] == -INFINITY) continue;  // an empty piece's O is not read
                    const float w = ptx::ex2(mg[i][e] - t8);
                    sum[i] = fmaf(w, lg[i][e], sum[i]);
                    acc[i][0] = fmaf(w, og[i][e].x, acc[i][0]);
                    acc[i][1] = fmaf(w, og[i][e].y, acc[i][1]);
                    acc[i][2] = fmaf(w, og[i][e].z, acc[i][2]);
                    acc[i][3] = fmaf(w, og[i][e].w, acc[i][3]);
                  }
                }
              }
#pragma unroll
              for (int i = 0; i < II; ++i)
                if (idx0 + i * kSoftmaxThreads < rows * (DH / 4))
                  emit(std::integral_constant<int, 4>{},
                       place(tile * kRows + (int)(at[i] / (DH / 4))),
                       (int)(at[i] % (DH / 4)) * 4, acc[i], top[i], sum[i]);
            }
          };
          if (n_piece <= 2)
            join(std::integral_constant<int, 2>{});
          else
            join(std::integral_constant<int, 8>{});
        }
      }
      ptx::tc_fence_before();
      ptx::named_sync(5, kSoftmaxThreads);  // O and red are free again
    }
    if (bad) misc[2] = 1;
  }

  ptx::tc_fence_before();
  __syncthreads();
  if (tid == 0 && misc[2] && A.status) *A.status = LBX_ETIMEOUT;
  if (warp == 8) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, Y::kTmemCols);
  }
}

// Launches of one head dimension and type (instances in cache_attn_*.cu).
template <int DH>
cudaError_t launch_attn(bool f16, const AttnMaps &maps, const AttnArgs &A, int grid,
                        cudaStream_t stream);
template <int DH, bool F16>
cudaError_t launch_attn_of(const AttnMaps &maps, const AttnArgs &A, int grid,
                           cudaStream_t stream) {
  cudaError_t e = cudaFuncSetAttribute(cache_attn_kernel<DH, F16>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       Lay<DH>::kSmemTotal);
  if (e != cudaSuccess) return e;
  cache_attn_kernel<DH, F16><<<(unsigned)grid, kThreads, Lay<DH>::kSmemTotal, stream>>>(maps, A);
  return cudaGetLastError();
}

}  // namespace cache
}  // namespace lbx
