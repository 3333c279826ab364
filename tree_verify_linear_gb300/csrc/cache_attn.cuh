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
// product serves (the error of o is 1.4 times that of weights in fp32).  f16 ends
// at 2^-25, which many small weights beside one large one add up to: weights are
// taken 2^7 times as large there (2^15 at most), so that what falls below is 2^-32 of
// the reference.
//
// The key list is cut into units of 64 keys from one array: the visible first
// positions before the window, the window, the tree's own keys.  A block is
// two units, one for each of the two threads of a row (one unit, half for
// each, at head dimension 256 in one CTA, where O leaves room for two score
// buffers of 64 columns).  All blocks of all streams form one list (request,
// layer, KV head, block), cut into equal ranges, one per CTA or pair (or per
// group of them, one for each row tile of the stream, which then read the same
// keys at the same time): one CTA per SM, whatever the lengths.  Streams that
// a range does not cover whole leave partials (m, l, O) in the workspace, at
// most two per CTA.  Of two pieces the CTA that finishes last joins both (its own
// from tensor memory).  Of more, the rows are joined in shares, one fewer than pieces:
// the CTAs of all but the last piece, whose ranges end there, wait a little for the
// others (they finish at about the same time) and take a share each; the one that
// finishes last takes what shares are left.  Where other work holds the SMs and CTAs
// of the launch run one after the other, the waits run out and that one takes all:
// no result depends on a CTA that may not be running.
//
// Streams of more than 128 rows (head dimensions 128 and 256) run on pairs of
// CTAs that share one product of 256 rows: each CTA keeps half of the block's
// keys and half of the columns of V, so a block takes half the shared memory
// and half the reads of L2.  Each CTA's copies arrive on its own barriers; the
// follower passes the news on to the leader, whose one thread issues all MMAs.
//
// Per CTA: warps 0-7 softmax, warp 8 issues the MMAs, warp 9 the copies, warp 10
// of a pair brings the Q tiles.  K
// and V arrive by TMA in 16 KB pieces through one ring, in the order the MMAs
// take them, so that all of the shared memory keeps copies in flight.  The Q
// tile sits in tensor memory (in shared memory for a pair, whose 128-key
// blocks need the columns).  S of a block and its P share one of two buffers.
// Every wait is bounded; a CTA whose wait gives up reports LBX_ETIMEOUT, counts
// its segment in with an empty partial, drains its copies, frees its tensor
// memory and leaves.
//
// What bounds it, measured on one GB300 (copies reach 6.77 TB/s).  One row per KV
// head's group, 16 requests of 8001 to 16384 keys, 4 layers, 32/8 heads of dimension
// 128, f16: 500 to 511 us, 92 to 94% of that bandwidth.  Trees of 22 nodes in bf16 at
// 24/4 heads of dimension 256: the tensor pipe, 1.8 us per block and pair for
// Q K^T and two products with V; five requests, 16 layers, 4096 keys each: 322 to 334 us (on
// single CTAs, which read K and V for 128 rows each, 618 us).  Short lists: the
// 7 us that a stream takes to begin and end.
#pragma once

#include "cache_common.cuh"
#include "cache_ptx.cuh"
#include "cache_walk.cuh"

namespace lbx {
namespace cache {

constexpr int kSoftmaxThreads = 256;

// Floats of one partial: m (base 2) and l per row, then O.
constexpr size_t part_floats(int dh) { return 2 * (size_t)kRows + (size_t)kRows * dh; }

struct AttnArgs {
  int L, Hq, Hkv, G;
  int n_req;      // key lists per (layer, KV head): requests, or 1 for the prefix
  int nodes;      // queries per key list and head: N, or all requests' N
  int fixed;      // length of every key list if > 0 (the prefix), else ctx_len
  int Bq, N, T;   // of the batch (its check, the trees)
  int window, n_sink;
  int join;       // what joining the pieces of a cut stream costs, in blocks
  float scale_log2;
  PerGroup per;
  Tiling til;
  const int32_t *ctx_len, *parent;
  const uint16_t *q;
  uint16_t *o;                 // results in the 16-bit type ...
  float *o32, *lse2;           // ... or normalised in fp32 with the base-2 lse
  float *lse;                  // natural lse or NULL
  const float *x_o, *x_lse2;   // the first launch's results to join, or NULL
  float *part;
  // Per CTA, of the stream that begins in its range and ends beyond it (one at most):
  // pieces written, and in the upper half the CTAs that are done with the stream; and,
  // kMaxCtas further on, the shares of its rows that are taken.
  unsigned int *counters;
  int32_t *status;
};

// A segment (a stream's blocks in the CTA's range) as the softmax threads see it:
// one warp walks the list for them and publishes the segments in turn.
struct Seg {
  int have;          // 0: the range is done
  int l, h, b;       // the stream
  int row0;          // its first row of this CTA
  int blk0, nb;      // blocks
  int ctx, w0, s_eff, ns, nw;  // the key list's units
  int slot, late;    // partials of the stream: the first one, and whether it is its CTA's second
  int pieces, mine;  // how many, and which is this CTA's
};

template <int DH, bool PAIR>
struct Lay {
  static constexpr int kCtas = PAIR ? 2 : 1;
  static constexpr bool kQTmem = !PAIR;
  static constexpr int kAtoms = DH / 64;
  static constexpr int kBlkUnits = DH == 256 && !PAIR ? 1 : 2;  // units per block
  static constexpr int kThreads = kSoftmaxThreads + (PAIR ? 96 : 64);
  static constexpr int kBlk = kBlkUnits * kUnit;                 // keys per block
  static constexpr int kMine = kBlk / 2;                         // keys per softmax thread
  // what one CTA holds of a block: kKeys keys of K, kCols columns of V
  static constexpr int kKeys = kBlk / kCtas, kCols = DH / kCtas;
  static constexpr int kPieces = kKeys * DH * 2 / kPiece < 1 ? 1 : kKeys * DH * 2 / kPiece;
  static constexpr int kKAtom = kKeys * 128;           // 64 columns of the K block
  static constexpr int kKAtoms = kPiece / kKAtom;      // such atoms per K piece
  static constexpr int kVKeys = kPiece / (kCols * 2);  // keys per V piece
  static constexpr int kVBox = kVKeys < kUnit ? kVKeys : kUnit;  // rows of a V box
  static constexpr int kVAtom = kVKeys * 128;          // 64 columns of a V piece
  static_assert(kPieces * kVKeys == kBlk && kPieces * kKAtoms * 64 == DH, "pieces");

  static constexpr int kQBytes = kQTmem ? 0 : kRows * DH * 2;
  static constexpr int kStages = (227 * 1024 - 3072 - kQBytes) / kPiece;
  static_assert(kStages > 2 * kPieces, "the next scores do not wait for this block's V");
  static constexpr int kSmemQ = 0;
  static constexpr int kSmemRing = kSmemQ + kQBytes;
  static constexpr int kSmemRed = kSmemRing + kStages * kPiece;  // float [2][2][128]
  static constexpr int kSmemSegs = kSmemRed + 4 * kRows * 4;     // Seg [4]
  static constexpr int kSmemMisc = kSmemSegs + 4 * (int)sizeof(Seg);  // int [8]
  static constexpr int kSmemBars = kSmemMisc + 32;
  // full, empty, peer (of a pair), s[2], p[2], o[2], lo[2], segs[4], q, q here, q free, end
  static constexpr int kNBars = (PAIR ? 3 : 2) * kStages + 16;
  static constexpr int kSmemTotal = kSmemBars + kNBars * 8;
  static_assert(kSmemTotal <= 227 * 1024 && kSmemRing % 1024 == 0, "shared memory");

  // tensor memory: Q (16-bit pairs), two buffers of S / P, O
  static constexpr uint32_t kColQ = 0, kColS = kQTmem ? 128 : 0;
  static constexpr uint32_t kColO = kColS + 2 * kBlk, kTmemCols = 512;
  static_assert(kColO + DH <= kTmemCols && (!kQTmem || DH / 2 <= 128), "tensor memory");
};

// Most rows whose pieces are joined by columns instead of by rows.
constexpr int kFewRows = 32;
// How long a CTA waits for the other pieces of a stream before it leaves them to the
// last: some times the spread of the ends of equal ranges; and an SM that other work
// waits for is kept no longer than that.  (64 requests of one row over 32001 shared keys,
// 16/2 heads of dimension 128: 84 us, 136 us where the last joins alone.)
constexpr uint64_t kJoinWaitNs = 50000;
// In blocks (of 2200 to 3400 cycles): what a stream costs beside its own, and what
// cutting streams and joining the pieces costs, the requests' and a prefix's
// (whose rows are more, and joined with the requests' results too).  Measured
// against 3 for both joins: five requests of 22 nodes, 24/4 heads of dimension
// 256, 2 layers over 1000 shared keys 71 -> 42 us, 4 layers over 4096 118 -> 100 us;
// of 3 nodes, 5 layers of 1024 keys 54 -> 38 us; where they lose, it is up to 5%.
constexpr int kLeadBlocks = 4, kJoinBlocks = 8, kJoinPrefixBlocks = 13;

// Parts of P: f16 once, bf16 hi + lo.
template <bool F16>
constexpr int kParts = F16 ? 1 : 2;

// What f16 weights are raised by, as a power of two.
template <bool F16>
constexpr float kLift = F16 ? 7.f : 0.f;

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

template <int DH, bool F16, bool PAIR>
__global__ void __launch_bounds__(Lay<DH, PAIR>::kThreads, 1)
    cache_attn_kernel(const __grid_constant__ AttnMaps maps, const __grid_constant__ AttnArgs A) {
  using Y = Lay<DH, PAIR>;
  extern __shared__ __align__(1024) unsigned char cache_smem[];
  unsigned char *smem = cache_smem;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  float *red = reinterpret_cast<float *>(smem + Y::kSmemRed);
  Seg *segs = reinterpret_cast<Seg *>(smem + Y::kSmemSegs);
  // [0] tensor memory base, [1] last of its row tile, [2] a wait gave up, [3] one
  // of a softmax thread did
  volatile int *misc = reinterpret_cast<volatile int *>(smem + Y::kSmemMisc);
  uint64_t *full = reinterpret_cast<uint64_t *>(smem + Y::kSmemBars);
  uint64_t *empty = full + Y::kStages, *peer = empty + Y::kStages;
  uint64_t *s_bar = peer + (PAIR ? Y::kStages : 0), *p_bar = s_bar + 2;
  uint64_t *o_bar = p_bar + 2, *lo_bar = o_bar + 2, *seg_bar = lo_bar + 2;
  uint64_t *q_bar = seg_bar + 4, *qh_bar = q_bar + 1, *qf_bar = qh_bar + 1;
  uint64_t *end_bar = qf_bar + 1;

  if (batch_bad(A.Bq, A.N, A.T, A.ctx_len, A.parent, nullptr)) {
    if (tid == 0 && A.status) *A.status = LBX_ETREE;
    return;
  }
  if (tid == 0) {
    for (int i = 0; i < Y::kNBars; ++i)
      ptx::mbar_init(full + i, full + i == p_bar || full + i == p_bar + 1
                                   ? Y::kCtas * kSoftmaxThreads / 32
                               : full + i == q_bar ? (PAIR ? 2 : kSoftmaxThreads / 32)
                                                   : 1);
    ptx::fence_mbar_init();
    misc[2] = misc[3] = 0;
  }
  if (warp == 8) {
    uint32_t *base = reinterpret_cast<uint32_t *>(smem + Y::kSmemMisc);
    if constexpr (PAIR) {
      ptx::tmem_alloc_pair(base, Y::kTmemCols);
    } else {
      ptx::tmem_alloc(base, Y::kTmemCols);
      ptx::tmem_relinquish();
    }
    ptx::tc_fence_before();
  }
  __syncthreads();
  if constexpr (PAIR) ptx::cluster_sync();  // the other CTA's barriers are set up
  ptx::tc_fence_after();
  const uint32_t tmem = static_cast<uint32_t>(misc[0]);

  const int rank = PAIR ? (int)ptx::cluster_rank() : 0;
  // the prefix's launch may take the SMs that this one leaves
  if (A.o32) ptx::launch_dependents();
  using Walker = Walk<Y::kBlkUnits, kLeadBlocks, AttnArgs>;
  bool bad = false;  // a wait of this thread gave up: it waits no more
  auto wait = [&](uint64_t *bar, uint32_t parity) {
    if (!bad && !ptx::mbar_wait(bar, parity)) bad = true;
    return !bad;
  };
  // One arrival of this warp on a barrier of the CTA that issues the MMAs.
  auto tell = [&](uint64_t *bar) {
    __syncwarp();
    if (lane == 0) {
      if constexpr (PAIR) ptx::mbar_arrive_at(bar, 0);
      else ptx::mbar_arrive(bar);
    }
  };
  // Query rows of the walk's tile from this CTA's first on.
  auto first_row = [&](const Walker &W) { return (W.tile * Y::kCtas + rank) * A.til.per_cta; };
  // The place of a row of the stream among all queries: of its first one, and
  // of the row from there.
  auto queries = [&](int l, int b, int h) {
    return (size_t)(l * A.n_req + b) * A.nodes * A.Hq + h * A.G;
  };
  auto query_of = [&](int row) { return row + A.per.node(row) * (A.Hq - A.G); };
  // Without a pair: the segment's queries into L2, ahead of its keys (loads of
  // them would wait for all the copies in flight).  One warp.
  auto prefetch_q = [&](const Walker &W) {
    const int row = first_row(W), left = A.til.rows - row;
    const int rows = left < A.til.per_cta ? left : A.til.per_cta;
    if (rows <= 0) return;
    const uint16_t *q0 = A.q + queries(W.l, W.b, W.h) * DH;
#pragma unroll 1
    for (int n = A.per.node(row) + lane; n <= A.per.node(row + rows - 1); n += 32)
      ptx::prefetch_bytes(q0 + (size_t)n * A.Hq * DH, (uint32_t)(A.G * DH * 2));
  };
  // The next segment with a tile for this CTA.
  auto advance = [&](Walker &W) {
#pragma unroll 1
    while (W.next())
      if (W.live) return true;
    return false;
  };
  // Segment k for the softmax threads.  The warp that does this is at most three
  // segments ahead of them (it has the last one's queries to load first, or its
  // products to issue), so that four places do.
  auto publish = [&](const Walker &W, bool have, uint32_t k) {
    if (lane != 0) return;
    Seg &s = segs[k & 3];
    s.have = have;
    if (have) {
      const int c_first = W.owner(W.first), c_last = W.owner(W.last);
      s.l = W.l, s.h = W.h, s.b = W.b, s.row0 = first_row(W);
      s.blk0 = W.blk0, s.nb = W.blk1 - W.blk0;
      s.ctx = W.ctx, s.w0 = W.w0, s.s_eff = W.s_eff, s.ns = W.ns, s.nw = W.nw;
      s.slot = 2 * ((c_first * A.til.group + W.slot_in_group) * Y::kCtas + rank);
      s.late = W.begin_of(c_first) < W.first;
      s.pieces = c_last - c_first + 1, s.mine = W.cg - c_first;
    }
    ptx::mbar_arrive(&seg_bar[k & 3]);
  };

  if (warp == 9) {
    // ---- copies ----
    Walker W(A, lane);
    Ring<Y::kStages> ring;
    int loads = 0;
    // behind the first Q tile's loads
    if constexpr (!PAIR) ptx::named_sync(6, kSoftmaxThreads + 32);
#pragma unroll 1
    while (advance(W)) {
      if (!PAIR) prefetch_q(W);
      if (lane != 0) continue;
      const int nb = W.blk1 - W.blk0;
      const int z = A.fixed > 0 ? W.l : W.l * A.n_req + W.b;
      auto take = [&]() -> unsigned char * {
        // the first round finds every stage free
        if (!wait(&empty[ring.st], ring.ph ^ 1u)) return nullptr;
        ptx::mbar_arrive_expect_tx(&full[ring.st], (uint32_t)kPiece);
        ++loads;
        return smem + Y::kSmemRing + ring.st * kPiece;
      };
#pragma unroll 1
      for (int i = 0; i <= nb && !bad; ++i) {
        if (i < nb) {  // K of block i
          const int u0 = (W.blk0 + i) * Y::kBlkUnits + rank;
          for (int p = 0; p < Y::kPieces; ++p, ring.step()) {
            unsigned char *d = take();
            if (!d) break;
#pragma unroll
            for (int u = 0; u < Y::kKeys / kUnit; ++u) {
              int start, cnt;
              bool tree;
              W.unit(u0 + u, start, tree, cnt);
#pragma unroll
              for (int a = 0; a < Y::kKAtoms; ++a)
                ptx::tma_load_4d(d + a * Y::kKAtom + u * kUnit * 128, tree ? &maps.kt : &maps.k,
                                 (p * Y::kKAtoms + a) * 64, W.h, start, z,
                                 &full[ring.st]);
            }
          }
        }
        if (i > 0 && !bad) {  // V of block i - 1
          const int u0 = (W.blk0 + i - 1) * Y::kBlkUnits;
          for (int p = 0; p < Y::kPieces; ++p, ring.step()) {
            unsigned char *d = take();
            if (!d) break;
#pragma unroll
            for (int k0 = 0; k0 < Y::kVKeys; k0 += Y::kVBox) {
              const int kk = p * Y::kVKeys + k0;
              int start, cnt;
              bool tree;
              W.unit(u0 + kk / kUnit, start, tree, cnt);
#pragma unroll
              for (int a = 0; a < Y::kCols / 64; ++a)
                ptx::tma_load_4d(d + a * Y::kVAtom + k0 * 128, tree ? &maps.vt : &maps.v,
                                 rank * Y::kCols + a * 64, W.h, start + kk % kUnit, z,
                                 &full[ring.st]);
            }
          }
        }
      }
    }
    if (lane == 0) {
      if (bad) misc[2] = 1;
      // every copy has landed before the CTA may leave (long since, unless a
      // wait gave up)
#pragma unroll 1
      for (int i = loads > Y::kStages ? loads - Y::kStages : 0; i < loads; ++i)
        (void)ptx::mbar_wait(&full[i % Y::kStages], (uint32_t)((i / Y::kStages) & 1));
    }
  } else if (PAIR && warp == 10) {
    // ---- Q tiles of a pair, by tensor copies (nodes past the last read as zeros) ----
    Walker W(A, lane);
    const uint32_t bytes = (uint32_t)(A.til.per_cta * DH * 2);
#pragma unroll 1
    for (uint32_t seg = 0;; ++seg) {
      const bool have = advance(W);
      publish(W, have, seg);
      if (!have) break;
      // the last segment's score products are done
      if (lane == 0 && (seg == 0 || wait(qf_bar, (seg - 1) & 1))) {
        ptx::mbar_arrive_expect_tx(qh_bar, bytes);
#pragma unroll 1
        for (int a = 0; a < Y::kAtoms; ++a)
          ptx::tma_load_4d(smem + Y::kSmemQ + a * kRows * 128, &maps.q, a * 64, W.h * A.G,
                           A.per.node(first_row(W)), A.fixed > 0 ? W.l : W.l * A.n_req + W.b,
                           qh_bar);
        if (wait(qh_bar, seg & 1)) ptx::mbar_arrive_at(q_bar, 0);
      }
      __syncwarp();
      if (A.x_o) {  // what the segment will be joined with, into L2
        ptx::wait_prerequisite_grid();
        const int row = first_row(W), left = A.til.rows - row;
        const int rows = left < A.til.per_cta ? left : A.til.per_cta;
        const size_t rows_all = (size_t)A.n_req * A.til.rows;
        const float4 *x0 = reinterpret_cast<const float4 *>(A.x_o) +
                           (size_t)(W.l * A.Hkv + W.h) * rows_all * (DH / 4) +
                           (size_t)W.b * A.til.rows + row;
#pragma unroll 1
        for (int c = lane; c < DH / 4 && rows > 0; c += 32)
          ptx::prefetch_bytes(x0 + c * rows_all, (uint32_t)(rows * 16));
      }
      if (__any_sync(0xffffffffu, bad)) break;
    }
    if (bad) {
      misc[2] = 1;
      (void)ptx::mbar_wait(qh_bar, 0);  // no copy is left behind
      (void)ptx::mbar_wait(qh_bar, 1);
    }
  } else if (warp == 8 && rank == 1) {
    // ---- the follower tells the leader of each piece that has landed ----
    Walker W(A, lane);
    Ring<Y::kStages> ring;
#pragma unroll 1
    while (W.next()) {
      if (!W.live || lane != 0) continue;
#pragma unroll 1
      for (int n = 2 * Y::kPieces * (W.blk1 - W.blk0); n > 0; --n, ring.step()) {
        if (!wait(&full[ring.st], ring.ph)) break;
        ptx::mbar_arrive_at(&peer[ring.st], 0);
      }
    }
    if (bad) misc[2] = 1;
  } else if (warp == 8) {
    // ---- MMAs: the warp walks and waits as one, one lane issues ----
    Walker W(A, lane);
    Ring<Y::kStages> ring;
    uint32_t q = 0, seg = 0;
    const bool one = ptx::elect_one();
    const uint64_t qdesc = ptx::sdesc_sw128(ptx::smem_u32(smem + Y::kSmemQ));
    const uint64_t kdesc = ptx::sdesc_sw128(ptx::smem_u32(smem + Y::kSmemRing));
    const uint64_t vdesc =
        ptx::sdesc(ptx::smem_u32(smem + Y::kSmemRing), (uint32_t)Y::kVAtom, 1024u, 2u);
    auto commit = [&](uint64_t *bar) {
      if constexpr (PAIR) ptx::mma_commit_pair(bar);
      else ptx::mma_commit(bar);
    };
    // the waits of the whole warp: given up by one lane, given up by all
    auto wait_all = [&](uint64_t *bar, uint32_t parity) {
      bad = !__all_sync(0xffffffffu, wait(bar, parity));
      return !bad;
    };
    // the ring's next piece, here and at the follower
    auto arrived = [&]() {
      return wait_all(&full[ring.st], ring.ph) && (!PAIR || wait_all(&peer[ring.st], ring.ph));
    };
#pragma unroll 1
    while (advance(W)) {
      if (!PAIR) publish(W, true, seg);
      const int nb = W.blk1 - W.blk0;
      // S of block i into buffer (q + i) & 1, once the buffer's last P has been
      // multiplied (the first two blocks find it free).  A pair takes the keys in
      // two halves, the upper half of each CTA's first: its columns held the lo
      // part of P, which is multiplied first (or nothing, in f16), so that they
      // are free while the hi part keeps the tensor cores busy.
      constexpr int kHalves = PAIR ? 2 : 1;
      auto scores = [&](int i) {
        const uint32_t qi = q + i, buf = qi & 1, last = ((qi >> 1) & 1) ^ 1u;
        constexpr uint32_t idesc = ptx::idesc_16(F16, kRows * Y::kCtas, Y::kBlk / kHalves, false);
        const Ring<Y::kStages> ring0 = ring;
#pragma unroll
        for (int half = kHalves - 1; half >= 0; --half) {
          if (half == 1 ? !F16 && !wait_all(&lo_bar[buf], last) : !wait_all(&o_bar[buf], last))
            return;
          const uint32_t d = tmem + Y::kColS + buf * Y::kBlk + half * 64;
          ring = ring0;
#pragma unroll
          for (int p = 0; p < Y::kPieces; ++p, ring.step()) {
            if (half == kHalves - 1 && !arrived()) return;
            ptx::tc_fence_after();
            const uint64_t kd =
                kdesc + (uint64_t)(ring.st * (kPiece >> 4)) + half * (32 * 128 >> 4);
            if (one) {
#pragma unroll
              for (int s = 0; s < 4 * Y::kKAtoms; ++s) {
                const int step = p * 4 * Y::kKAtoms + s;  // 16 columns of Q and K
                const uint64_t kb = kd + (uint64_t)((s >> 2) * Y::kKAtom >> 4) + 2 * (s & 3);
                const uint64_t qa =
                    qdesc + (uint64_t)((step >> 2) * kRows * 128 >> 4) + 2 * (step & 3);
                const uint32_t acc = step > 0 ? 1u : 0u;
                if constexpr (PAIR) ptx::mma_16_ss_pair(d, qa, kb, idesc, acc);
                else ptx::mma_bf16_ts(d, tmem + Y::kColQ + 8u * step, kb, idesc, acc);
              }
              if (half == 0) {
                commit(&empty[ring.st]);
                if (p == Y::kPieces - 1) {
                  commit(&s_bar[buf]);
                  if (PAIR && i == nb - 1) commit(qf_bar);
                }
              }
            }
            __syncwarp();
          }
        }
      };
      if (wait_all(q_bar, seg & 1)) {
        ptx::tc_fence_after();
        scores(0);
      }
#pragma unroll 1
      for (int i = 0; i < nb && !bad; ++i) {
        if (i + 1 < nb) scores(i + 1);
        const uint32_t qi = q + i, buf = qi & 1;
        if (!wait_all(&p_bar[buf], (qi >> 1) & 1)) break;
        ptx::tc_fence_after();
        constexpr uint32_t idesc = ptx::idesc_16(F16, kRows * Y::kCtas, DH, true);
        const uint32_t pc = tmem + Y::kColS + buf * Y::kBlk;
        const uint32_t later = i > 0 ? 1u : 0u;
        const Ring<Y::kStages> ring0 = ring;
#pragma unroll
        for (int part = kParts<F16> - 1; part >= 0; --part) {
          ring = ring0;
#pragma unroll
          for (int p = 0; p < Y::kPieces; ++p, ring.step()) {
            if (part == kParts<F16> - 1 && !arrived()) break;
            ptx::tc_fence_after();
            const uint64_t vd = vdesc + (uint64_t)(ring.st * (kPiece >> 4));
            if (one) {
#pragma unroll
              for (int s = 0; s < Y::kVKeys / 16; ++s) {
                const uint32_t pa =
                    pc + (uint32_t)(part * Y::kBlk / 2 + p * Y::kVKeys / 2 + s * 8);
                const uint64_t vb = vd + (uint64_t)(s * 2048 >> 4);
                const uint32_t acc = part < kParts<F16> - 1 || p + s > 0 ? 1u : later;
                if constexpr (PAIR) ptx::mma_16_ts_pair(tmem + Y::kColO, pa, vb, idesc, acc);
                else ptx::mma_bf16_ts(tmem + Y::kColO, pa, vb, idesc, acc);
              }
              if (part == 0) commit(&empty[ring.st]);
              if (p == Y::kPieces - 1) {
                if (part == 0) commit(&o_bar[buf]);
                else if (PAIR) commit(&lo_bar[buf]);
              }
            }
            __syncwarp();
          }
          if (bad) break;
        }
      }
      q += nb;
      ++seg;
      if (bad) break;
    }
    if (!PAIR) publish(W, false, seg);
    if (one) {
      if (bad) misc[2] = 1;
      commit(end_bar);
      (void)ptx::mbar_wait(end_bar, 0);
    }
  } else {
    // ---- softmax ----
    const int quad = warp & 3, hf = warp >> 2;
    const uint32_t tq = tmem + ((uint32_t)(quad * 32) << 16);
    const int r = quad * 32 + lane;  // row of the tile
    const float sl2 = A.scale_log2;
    constexpr int kHalf = DH / 2;
    uint32_t q = 0, piece = 0;  // blocks and ring pieces so far

    // Without a pair: the Q tile of a segment into tensor memory, half a
    // row per thread, pairs along dh, rows past the stream's zero.  The first
    // tile's loads go ahead of the first copies of K and V.
    bool ahead = !PAIR;
    auto go_ahead = [&]() {
      if (ahead) asm volatile("bar.arrive 6, %0;" ::"n"(kSoftmaxThreads + 32) : "memory");
      ahead = false;
    };
    auto load_q = [&](const volatile Seg &s) {
      constexpr int kPer = DH / 8;  // 16-byte pieces per row
      const int row = s.row0 + r;
      const bool in = row < A.til.rows;
      const uint4 *from = reinterpret_cast<const uint4 *>(A.q);
      if (in) from += (queries(s.l, s.b, s.h) + query_of(row)) * kPer + hf * (kPer / 2);
      constexpr int kC = DH / 4 < 32 ? DH / 4 : 32;  // columns per store
      uint4 v[DH / 16];
#pragma unroll
      for (int e = 0; e < DH / 16; ++e) v[e] = in ? from[e] : make_uint4(0u, 0u, 0u, 0u);
      go_ahead();
#pragma unroll
      for (int c = 0; c < DH / 4; c += kC) {
        uint32_t w[kC];
#pragma unroll
        for (int e = 0; e < kC / 4; ++e) {
          const uint4 f = v[c / 4 + e];
          w[4 * e] = f.x, w[4 * e + 1] = f.y, w[4 * e + 2] = f.z, w[4 * e + 3] = f.w;
        }
        if constexpr (kC == 32) ptx::tmem_st32(tq + Y::kColQ + hf * (DH / 4) + c, w);
        else ptx::tmem_st16(tq + Y::kColQ + hf * (DH / 4) + c, w);
      }
      ptx::tmem_wait_st();
      ptx::tc_fence_before();
      tell(q_bar);
    };
    // What this row sees in a segment: of the tree as bits, of the cache from a
    // position on.  The ancestor masks of the request's tree, by doubling, are one
    // warp's work; they lie where the last maxima were.
    uint64_t next_bits = 0;
    int next_lo = 0;
    int up[2] = {-1, -1};
    auto parents = [&](const volatile Seg &s) {  // ahead of look()
      if (A.fixed > 0 || warp != 0) return;
      const int32_t *parent = A.parent + (size_t)s.b * A.N;
      up[0] = lane < A.N ? parent[lane] : -1, up[1] = lane + 32 < A.N ? parent[lane + 32] : -1;
    };
    auto look = [&](const volatile Seg &s) {
      if (A.fixed > 0) return;
      uint64_t *anc = reinterpret_cast<uint64_t *>(red);
      if (warp == 0) {
        uint64_t m[2] = {1ull << lane, 1ull << (lane + 32)};
#pragma unroll 1
        for (int step = 0; step < 6; ++step) {
          uint64_t add[2];
          int to[2];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int a = up[e] & 31;
            const uint64_t m0 = __shfl_sync(0xffffffffu, m[0], a);
            const uint64_t m1 = __shfl_sync(0xffffffffu, m[1], a);
            const int u0 = __shfl_sync(0xffffffffu, up[0], a);
            const int u1 = __shfl_sync(0xffffffffu, up[1], a);
            add[e] = up[e] < 0 ? 0ull : up[e] < 32 ? m0 : m1;
            to[e] = up[e] < 0 ? -1 : up[e] < 32 ? u0 : u1;
          }
          m[0] |= add[0], m[1] |= add[1], up[0] = to[0], up[1] = to[1];
        }
        anc[lane] = m[0], anc[lane + 32] = m[1];
      }
      ptx::named_sync(5, kSoftmaxThreads);
      const int row = s.row0 + r;
      next_bits = 0, next_lo = 0;
      if (r < A.til.per_cta && row < A.til.rows) {
        next_bits = anc[A.per.node(row)];
        if (A.window > 0) {
          const int ctx = s.ctx;
          next_lo = ctx + __popcll(next_bits) - A.window;  // ctx + depth - window + 1
          uint64_t m = next_bits;
#pragma unroll 1
          for (int pos = ctx; m; ++pos, m &= m - 1)  // nodes of the path, root first
            if (pos < next_lo && pos >= A.n_sink) next_bits &= ~(m & (0 - m));
        }
      }
    };

    // Segment k is published (and the last one's maxima are read); false in all
    // threads if a wait of any of them gave up.
    auto published = [&](uint32_t k) {
      wait(&seg_bar[k & 3], (k >> 2) & 1);
      if (bad) misc[3] = 1;
      ptx::named_sync(5, kSoftmaxThreads);
      return misc[3] == 0;
    };
    uint32_t k = 0;
    const volatile Seg *g = segs;
    bool more = published(0) && g->have;
    if (more) {
      parents(*g);
      if constexpr (!PAIR) load_q(*g);
      look(*g);
      // the masks are read before the first block's maxima take their place (for
      // later segments the barrier at a segment's end sees to it)
      ptx::named_sync(5, kSoftmaxThreads);
    } else {
      go_ahead();
    }
#pragma unroll 1
    while (more) {
      const int nb = g->nb, row = g->row0 + r;
      const bool real = r < A.til.per_cta && row < A.til.rows;
      // the warp has rows
      const bool busy = quad * 32 < A.til.per_cta && row - lane < A.til.rows;
      const uint64_t tree_bits = next_bits;
      const int lo = next_lo;

      float m_run = -INFINITY, l_run = 0.f;  // the row's reference (raw); this half's sum
#pragma unroll 1
      for (int i = 0; i < nb; ++i) {
        const uint32_t qi = q + i;
        wait(&s_bar[qi & 1], (qi >> 1) & 1);
        ptx::tc_fence_after();
        const uint32_t sc = tq + Y::kColS + (qi & 1) * Y::kBlk;
        float sv[Y::kMine], mh = -INFINITY;
        if (busy) {
          // (a pair's columns: the lower halves of both units, then the upper)
          constexpr int kFirst = PAIR ? 32 : Y::kMine, kThen = PAIR ? 64 : 32;
          ptx::tmem_ld32(sc + hf * kFirst, *reinterpret_cast<float(*)[32]>(sv));
          if constexpr (Y::kMine == 64)
            ptx::tmem_ld32(sc + hf * kFirst + kThen, *reinterpret_cast<float(*)[32]>(sv + 32));
        }
        // this thread's unit: its own, or the upper or lower half of the one
        constexpr bool kOne = Y::kBlkUnits == 1;
        int start, cnt;
        bool tree;
        unit_of(*g, A.fixed > 0, A.N, (g->blk0 + i) * Y::kBlkUnits + (kOne ? 0 : hf), start, tree,
                cnt);
        auto clear_unseen = [&]() {
          // values no query sees must not reach O through a zero weight
          if (!tree && cnt > 0 && cnt < kUnit) {
            // the stage's earlier pieces have been multiplied, so that its barrier
            // is in the phase that ends with this one's arrival
            if (i > 0) wait(&o_bar[(qi - 1) & 1], ((qi - 1) >> 1) & 1);
            // V comes after K of the next block; the unit's keys lie in one piece or
            // several, or in a half of one
            const uint32_t v_piece = piece + Y::kPieces * ((i + 1 < nb ? i + 2 : nb) + i);
            constexpr int kWide = Y::kCols / 8, kBy = kOne ? 256 : 128;
            constexpr int kIn = Y::kVKeys < kUnit ? Y::kVKeys : kUnit;  // keys of it in a piece
#pragma unroll
            for (int part = 0; part < kUnit / kIn; ++part) {
              const int at0 = (kOne ? 0 : hf * kUnit) + part * kIn;  // key of the block
              const uint32_t pc = v_piece + at0 / Y::kVKeys, st = pc % Y::kStages;
              const int from = cnt - part * kIn > 0 ? cnt - part * kIn : 0;
              if (from < kIn) wait(&full[st], (pc / Y::kStages) & 1);
              unsigned char *v0 = smem + Y::kSmemRing + st * kPiece + (at0 % Y::kVKeys) * 128;
#pragma unroll 2
              for (int idx = from * kWide + tid % kBy; idx < kIn * kWide; idx += kBy)
                *reinterpret_cast<uint4 *>(v0 + (idx % kWide / 8) * Y::kVAtom +
                                           idx / kWide * 128 + (idx & 7) * 16) =
                    make_uint4(0u, 0u, 0u, 0u);
            }
            ptx::fence_proxy_async();
            if constexpr (PAIR) ptx::fence_cluster();
          }
        };
        if (!busy) {  // no rows: keep step with the others
          clear_unseen();
          tell(&p_bar[qi & 1]);
          continue;
        }
        const uint64_t seen = tree ? tree_bits
                                   : low_bits(cnt) & (~low_bits(lo - start) |
                                                      low_bits(A.n_sink - start));
        const uint64_t ok = (cnt > 0 ? seen : 0ull) >> (kOne ? hf * 32 : 0);
        constexpr uint64_t kAll = Y::kMine == 64 ? ~0ull : 0xffffffffull;
        ptx::tmem_wait_ld();
        if (!__all_sync(0xffffffffu, (ok & kAll) == kAll)) {
#pragma unroll
          for (int e = 0; e < Y::kMine; ++e)
            if (!((uint32_t)(ok >> (e & 32)) >> (e & 31) & 1)) sv[e] = -INFINITY;
        }
        {
          float mx[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) mx[e] = sv[e];
#pragma unroll
          for (int e = 8; e < Y::kMine; ++e) mx[e & 7] = fmaxf(mx[e & 7], sv[e]);
          mh = fmaxf(fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])),
                     fmaxf(fmaxf(mx[4], mx[5]), fmaxf(mx[6], mx[7])));
        }
        // (two buffers: the other half may not have read the last block's yet)
        float *max_of = red + (qi & 1) * 2 * kRows;
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
        const float ref = m_run == -INFINITY ? 0.f : fmaf(m_run, sl2, -kLift<F16>);
        {
          float sum[4] = {0.f, 0.f, 0.f, 0.f};
          uint32_t pk[Y::kMine / 2];
#pragma unroll
          for (int e = 0; e < Y::kMine / 2; ++e) {
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
          auto store = [&](uint32_t col) {
            if constexpr (Y::kMine == 64) ptx::tmem_st32(col, pk);
            else ptx::tmem_st16(col, pk);
          };
          store(sc + hf * (Y::kMine / 2));
          if constexpr (!F16) {
#pragma unroll
            for (int e = 0; e < Y::kMine / 2; ++e) pk[e] = pack2<false>(sv[2 * e], sv[2 * e + 1]);
            store(sc + Y::kMine + hf * (Y::kMine / 2));
          }
        }
        // rows whose reference moved rescale their half of O's columns, once
        // the previous product is done
        if (__any_sync(0xffffffffu, need)) {
          wait(&o_bar[(qi - 1) & 1], ((qi - 1) >> 1) & 1);
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
        clear_unseen();
        ptx::tmem_wait_st();
        ptx::tc_fence_before();
        tell(&p_bar[qi & 1]);
      }
      piece += 2 * Y::kPieces * nb;
      q += nb;
      // what the next segment needs, while the last product runs (every score
      // product of this segment is done: its Q tile may go)
      ++k;
      const volatile Seg *next = &segs[k & 3];
      more = published(k) && next->have;
      if (more) {
        parents(*next);
        if constexpr (!PAIR) load_q(*next);
        look(*next);
      }

      // ---- this segment's result: whole, or a partial ----
      // A finished row of the stream in the first launch's results ([layer, KV head]
      // [DH / 4][all rows] of four columns); the first columns are fetched ahead.
      const int l = g->l, h = g->h, b = g->b, row0 = g->row0;
      const size_t rows_all = (size_t)A.n_req * A.til.rows;
      auto place_x = [&](int rw) {
        return (size_t)(l * A.Hkv + h) * rows_all * (DH / 4) + (size_t)b * A.til.rows + rw;
      };
      float4 x[2][4];
      auto fetch_x = [&](float4(&to)[4], int col) {
        const float4 *from =
            reinterpret_cast<const float4 *>(A.x_o) + place_x(row) + col / 4 * rows_all;
#pragma unroll
        for (int e = 0; e < 4; ++e) to[e] = __ldcg(from + e * rows_all);
      };
      if (A.x_o) ptx::wait_prerequisite_grid();  // that launch is complete
      if (A.x_o && real) fetch_x(x[0], hf * kHalf), fetch_x(x[1], hf * kHalf + 16);
      wait(&o_bar[(q - 1) & 1], ((q - 1) >> 1) & 1);
      ptx::tc_fence_after();
      ptx::named_sync(1 + quad, 64);  // the last maxima are read
      float *sums = red + 2 * kRows;  // clear of the masks
      sums[hf * kRows + r] = l_run;
      if (bad) misc[3] = 1;
      ptx::named_sync(5, kSoftmaxThreads);
      const bool valid = misc[3] == 0;
      float l_sum = sums[r] + sums[kRows + r];
      float m2 = m_run == -INFINITY ? -INFINITY : fmaf(m_run, sl2, -kLift<F16>);
      if (!valid) l_sum = 0.f, m2 = -INFINITY;
      // A finished row's place among all queries, and in the first launch's lse.
      auto place = [&](int rw) { return queries(l, b, h) + query_of(rw); };
      auto place_xl = [&](int rw) {
        return (size_t)(l * A.Hkv + h) * rows_all + (size_t)b * A.til.rows + rw;
      };
      // The factors of this stream's O and of the first launch's o, and the row's lse.
      // (A NaN among a row's scores makes its sum one, and the row with it.)
      auto factors = [&](int rw, float m, float sum, float &w, float &wx) {
        constexpr float kDown = F16 ? 1.f / 128.f : 1.f;  // 2^-kLift
        const float own = sum == 0.f ? -INFINITY : m + kLift<F16> + __log2f(sum * kDown);
        float all = own;
        w = sum == 0.f ? 0.f : __fdividef(1.f, sum), wx = 0.f;
        if (A.x_o) {
          const float x = __ldcg(A.x_lse2 + place_xl(rw)), top = fmaxf(own, x);
          if (own != -INFINITY || x != -INFINITY) {
            const float eo = ptx::ex2(own - top), ex = ptx::ex2(x - top);
            const float inv = __fdividef(1.f, eo + ex);
            w *= eo * inv, wx = ex * inv;
            all = top + __log2f(eo + ex);
          }
        }
        return all;
      };
      auto put_lse = [&](int rw, float all) {
        if (A.lse2) A.lse2[place_xl(rw)] = all;
        if (A.lse) A.lse[place(rw)] = all * 0.6931471805599453f;
      };
      const int n_piece = g->pieces, mine = g->mine;
      const bool whole = n_piece == 1;
      const int left = A.til.rows - row0, rows = left < A.til.per_cta ? left : A.til.per_cta;
      // Partial e of the stream: m and l per row, then O as [DH / 4][128] of
      // four columns.  Each CTA has two: its first segment's, and its last's.
      const size_t by = 2 * (size_t)A.til.group * Y::kCtas * part_floats(DH);
      float *part0 = A.part + (size_t)g->slot * part_floats(DH);
      const int late = g->late ? (int)part_floats(DH) : 0;
      auto partial = [&](int e) { return part0 + e * by + (e == 0 ? late : 0); };
      bool join = false;
      const int counter = g->slot >> 1;
      if (!whole && rows > 0) {
        float4 *to = reinterpret_cast<float4 *>(partial(mine) + 2 * kRows);
        if (busy && valid) {
#pragma unroll 1
          for (int c = 0; c < kHalf / 32; ++c) {
            const int col = hf * kHalf + 32 * c;
            float ov[32];
            ptx::tmem_ld32(tq + Y::kColO + (uint32_t)col, ov);
            ptx::tmem_wait_ld();
            if (real) {
#pragma unroll
              for (int e = 0; e < 8; ++e)
                to[(col / 4 + e) * kRows + r] =
                    make_float4(ov[4 * e], ov[4 * e + 1], ov[4 * e + 2], ov[4 * e + 3]);
            }
          }
        }
        if (real && hf == 0) {
          float *ml = partial(mine);
          ml[r] = m2, ml[kRows + r] = l_sum;
        }
        ptx::named_sync(5, kSoftmaxThreads);
        if (tid == 0) {
          int share = 0;
          __threadfence();  // the CTA's partial, before its arrival
          const unsigned prev = atomicAdd(&A.counters[counter], 1u) & 0xffffu;
          const bool last = prev == (unsigned)n_piece - 1;
          int go = last;
          if (n_piece == 2 && go) A.counters[counter] = 0u;  // for the next call
          if (n_piece > 2) {
            if (!last && mine < n_piece - 1)
              go = ptx::wait_count(&A.counters[counter], (unsigned)n_piece, kJoinWaitNs);
            if (go) share = (int)atomicAdd(&A.counters[kMaxCtas + counter], 1u);
            misc[4] = share, misc[5] = last;
          }
          misc[1] = go;
          __threadfence();
        }
        ptx::named_sync(5, kSoftmaxThreads);
        join = misc[1] != 0;
      }
      if (join && (n_piece > 2 || rows <= kFewRows)) {
        // few rows, or a share of them: the pieces' weights, then four columns of a
        // row per thread; as many rows at a time as `red` holds weights of
        const int shares = n_piece == 2 ? 1 : rows < n_piece - 1 ? rows : n_piece - 1;
        const bool last = n_piece > 2 && misc[5] != 0;
        constexpr int kHeld = (4 * kRows - kFewRows) / 2;
        float *l_of = red + kHeld, *wx_of = l_of + kHeld;
        const int step = kHeld / n_piece < kFewRows ? kHeld / n_piece : kFewRows;
        int share = n_piece > 2 ? misc[4] : 0;
#pragma unroll 1
        while (share < shares) {
          const int from = rows * share / shares, to = rows * (share + 1) / shares;
#pragma unroll 1
          for (int rr0 = from; rr0 < to; rr0 += step) {
            const int here = to - rr0 < step ? to - rr0 : step;
            ptx::named_sync(5, kSoftmaxThreads);  // the last weights are read
            if (tid < here * n_piece) {
              const float *pg = partial(tid / here) + rr0 + tid % here;
              red[tid] = __ldcg(pg), l_of[tid] = __ldcg(pg + kRows);
            }
            ptx::named_sync(5, kSoftmaxThreads);
            if (tid < here) {
              const int rw = row0 + rr0 + tid;
              float top = -INFINITY, sum = 0.f;
#pragma unroll 1
              for (int e = tid; e < here * n_piece; e += here) top = fmaxf(top, red[e]);
              if (top == -INFINITY) top = 0.f;
#pragma unroll 1
              for (int e = tid; e < here * n_piece; e += here) {
                const float w_e = ptx::ex2(red[e] - top);
                red[e] = w_e;
                sum = fmaf(w_e, l_of[e], sum);
              }
              float w, wx;
              put_lse(rw, factors(rw, top, sum, w, wx));
#pragma unroll 1
              for (int e = tid; e < here * n_piece; e += here) red[e] *= w;
              wx_of[tid] = wx;
            }
            ptx::named_sync(5, kSoftmaxThreads);
#pragma unroll 1
            for (int idx = tid; idx < (here + 7) / 8 * 8 * (DH / 4); idx += kSoftmaxThreads) {
              const int rr = idx / (2 * DH) * 8 + idx % 8, c4 = idx / 8 % (DH / 4);
              const int rw = row0 + rr0 + rr;
              if (rr >= here) continue;
              float4 f = make_float4(0.f, 0.f, 0.f, 0.f);
              if (A.x_o) {
                f = __ldcg(reinterpret_cast<const float4 *>(A.x_o) + place_x(rw) + c4 * rows_all);
                const float wx = wx_of[rr];
                f.x *= wx, f.y *= wx, f.z *= wx, f.w *= wx;
              }
              // ten pieces' loads in flight
#pragma unroll 1
              for (int e0 = 0; e0 < n_piece; e0 += 10) {
                float4 y[10];
#pragma unroll
                for (int e = 0; e < 10; ++e)
                  y[e] = __ldcg(reinterpret_cast<const float4 *>(
                                    partial(e0 + e < n_piece ? e0 + e : e0) + 2 * kRows) +
                                c4 * kRows + rr0 + rr);
#pragma unroll
                for (int e = 0; e < 10; ++e) {
                  const float w_e = e0 + e < n_piece ? red[(e0 + e) * here + rr] : 0.f;
                  if (w_e != 0.f)  // (an empty piece's O holds nothing)
                    f.x = fmaf(w_e, y[e].x, f.x), f.y = fmaf(w_e, y[e].y, f.y),
                    f.z = fmaf(w_e, y[e].z, f.z), f.w = fmaf(w_e, y[e].w, f.w);
                }
              }
              if (A.o32)
                reinterpret_cast<float4 *>(A.o32)[place_x(rw) + c4 * rows_all] = f;
              else
                reinterpret_cast<uint2 *>(A.o + place(rw) * DH)[c4] =
                    make_uint2(pack2<F16>(f.x, f.y), pack2<F16>(f.z, f.w));
            }
          }
          if (!last) break;  // those that are left are the last one's
          ptx::named_sync(5, kSoftmaxThreads);  // the share's number is read
          if (tid == 0) misc[4] = (int)atomicAdd(&A.counters[kMaxCtas + counter], 1u);
          ptx::named_sync(5, kSoftmaxThreads);
          share = misc[4];
        }
      } else if (busy && valid && (whole || join)) {
        // a row per two threads; this CTA's piece is still in tensor memory, the
        // other one's columns come ahead
        float top = m2, sum = l_sum, f_it = 0.f, f_mine = 1.f;
        const float *other = partial(join ? 1 - mine : 0);
        float4 y[4];
        auto fetch_y = [&](int col) {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            y[e] = __ldcg(reinterpret_cast<const float4 *>(other + 2 * kRows) +
                          (col / 4 + e) * kRows + r);
        };
        if (join) {
          fetch_y(hf * kHalf);
          const float m_it = __ldcg(other + r), l_it = __ldcg(other + kRows + r);
          top = fmaxf(top, m_it);
          if (top == -INFINITY) top = 0.f;
          f_mine = ptx::ex2(m2 - top), f_it = ptx::ex2(m_it - top);
          // (in the pieces' order, whichever CTA joins them)
          sum = mine == 0 ? fmaf(f_it, l_it, f_mine * l_sum) : fmaf(f_mine, l_sum, f_it * l_it);
        }
        float w = 0.f, wx = 0.f, all = 0.f;
        if (real) all = factors(row, top, sum, w, wx);
        if (real && hf == 0) put_lse(row, all);
        f_mine *= w, f_it *= w;
        // where the four rows of this lane's group of lanes go
        uint64_t to[4] = {};
        if (A.o) {
          const uint64_t mine = real ? reinterpret_cast<uint64_t>(A.o + place(row) * DH) : 0ull;
#pragma unroll
          for (int k = 0; k < 4; ++k) to[k] = __shfl_sync(0xffffffffu, mine, (lane & ~3) + k);
        }
#pragma unroll 1
        for (int c = 0; c < kHalf / 32; ++c) {
          uint32_t pc[4][4];  // 32 columns, 16 at a time
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const int col = hf * kHalf + 32 * c + 16 * j;
            const bool more = j == 0 || c + 1 < kHalf / 32;
            float v[16];
            ptx::tmem_ld16(tq + Y::kColO + (uint32_t)col, v);
            ptx::tmem_wait_ld();
            if (!join) {
#pragma unroll
              for (int e = 0; e < 16; ++e) v[e] *= w;
            }
            auto add = [&](float f, const float4(&z)[4]) {
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                v[4 * e] = fmaf(f, z[e].x, v[4 * e]);
                v[4 * e + 1] = fmaf(f, z[e].y, v[4 * e + 1]);
                v[4 * e + 2] = fmaf(f, z[e].z, v[4 * e + 2]);
                v[4 * e + 3] = fmaf(f, z[e].w, v[4 * e + 3]);
              }
            };
            if (join && real) {
              if (!(f_it > 0.f)) {  // an empty piece's O holds nothing
#pragma unroll
                for (int e = 0; e < 4; ++e) y[e] = make_float4(0.f, 0.f, 0.f, 0.f);
              }
              const float *z = reinterpret_cast<const float *>(y);
              if (mine == 0) {
#pragma unroll
                for (int e = 0; e < 16; ++e) v[e] = fmaf(f_it, z[e], f_mine * v[e]);
              } else {
#pragma unroll
                for (int e = 0; e < 16; ++e) v[e] = fmaf(f_mine, v[e], f_it * z[e]);
              }
              if (more) fetch_y(col + 16);
            }
            if (A.x_o && real) {
              add(wx, x[j]);
              if (c + 1 < kHalf / 32) fetch_x(x[j], col + 32);
            }
            if (A.o32) {
              float4 *at = reinterpret_cast<float4 *>(A.o32) + place_x(row) + col / 4 * rows_all;
              if (real) {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                  at[e * rows_all] = make_float4(v[4 * e], v[4 * e + 1], v[4 * e + 2], v[4 * e + 3]);
              }
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) pc[2 * j + (e >> 2)][e & 3] = pack2<F16>(v[2 * e], v[2 * e + 1]);
          }
          if (A.o) {
            // four lanes exchange 16-byte pieces, so that a store of the warp
            // writes 64 bytes of eight rows instead of 16 of thirty-two
#pragma unroll
            for (int s = 1; s <= 2; s *= 2) {
              const bool up = lane & s;
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                if (k & s) continue;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                  const uint32_t got =
                      __shfl_xor_sync(0xffffffffu, up ? pc[k][e] : pc[k + s][e], s);
                  if (up) pc[k][e] = got;
                  else pc[k + s][e] = got;
                }
              }
            }
#pragma unroll
            for (int k = 0; k < 4; ++k)
              if (to[k])
                reinterpret_cast<uint4 *>(to[k])[(hf * kHalf + 32 * c) / 8 + (lane & 3)] =
                    make_uint4(pc[k][0], pc[k][1], pc[k][2], pc[k][3]);
          }
        }
      }
      if (tid == 0 && rows > 0 && n_piece > 2) {
        // done with the stream's counters; the last that is clears them for the next call
        __threadfence();
        if (atomicAdd(&A.counters[counter], 1u << 16) >> 16 == (unsigned)n_piece - 1)
          A.counters[counter] = A.counters[kMaxCtas + counter] = 0u;
      }
      ptx::tc_fence_before();
      ptx::named_sync(5, kSoftmaxThreads);  // O and red are free again
      g = next;
      more = more && valid;
    }
  }

  ptx::tc_fence_before();
  __syncthreads();
  if constexpr (PAIR) ptx::cluster_sync();  // neither leaves while the other may reach it
  if (tid == 0 && (misc[2] || misc[3]) && A.status) *A.status = LBX_ETIMEOUT;
  if (warp == 8) {
    ptx::tc_fence_after();
    if constexpr (PAIR) ptx::tmem_dealloc_pair(tmem, Y::kTmemCols);
    else ptx::tmem_dealloc(tmem, Y::kTmemCols);
  }
}

// The small kernel of cache_few.cu.
struct FewArgs {
  lbx_attn_cfg c;
  int chunks;  // units a stream can have
  float scale_log2;
  const int32_t *ctx_len, *parent;
  const uint16_t *q, *kp, *vp, *kc, *vc, *kt, *vt;
  uint16_t *o;
  float *lse, *part;
  unsigned int *counters;
  int32_t *status;
};
// Most units of all streams it takes (see few_chunks).
constexpr int kFewUnits = 1024;
// Units per stream, or 0 where the call is not one for the small kernel.
int few_chunks(const lbx_attn_cfg *c);
cudaError_t launch_few(const FewArgs &A, cudaStream_t stream);

// Launches of one head dimension and type (instances in cache_attn_*.cu).
template <int DH>
cudaError_t launch_attn(bool f16, const AttnMaps &maps, const AttnArgs &A, int grid,
                        cudaStream_t stream);
template <int DH, bool F16, bool PAIR>
cudaError_t launch_attn_of(const AttnMaps &maps, const AttnArgs &A, int grid,
                           cudaStream_t stream) {
  auto kernel = cache_attn_kernel<DH, F16, PAIR>;
  constexpr int bytes = Lay<DH, PAIR>::kSmemTotal;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid), cfg.blockDim = dim3(Lay<DH, PAIR>::kThreads);
  cfg.dynamicSmemBytes = bytes, cfg.stream = stream;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = PAIR ? 2 : 1, at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  // the second launch of a call begins where the first one's CTAs end and waits for
  // its results where it joins them
  at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at, cfg.numAttrs = A.x_o ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, maps, A);
}

}  // namespace cache
}  // namespace lbx
