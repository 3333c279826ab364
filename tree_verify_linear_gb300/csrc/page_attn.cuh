// page_attn.cuh -- attention of each request's new tokens over its pages on the
// tensor cores (sm_103a): the kernel behind lbx_paged_attention.
//
// Rows are (token, head of the group) pairs of one KV head, 128 to a subtile.  Per block
// of 128 keys and subtile
//   S = Q K^T          tensor cores, operands in shared memory
//   softmax            online, base 2, statistics in fp32
//   O += P V           tensor cores, P from tensor memory, in V's type
// The running reference of a row moves only when a block's maximum exceeds it by more
// than 2^8, so that O is rescaled rarely; the result is the same softmax taken from
// another reference.  P is rounded to the 16-bit type once (2^-8 of a weight in bf16,
// 2^-11 in f16), which adds about as much error as the rounding of o, or (SPLIT, the
// caller's choice) takes two parts, P rounded and what that loses, each with a product of its
// own: good to 2^-16 and 2^-22.  The second product is half of the tensor cores' work again,
// more than copies hide at head dimension 256: there single tokens over long caches (4 layers, 16
// requests of 8001 to 16384 keys, bf16) take 627 us instead of 481, trees of 22 on 16 layers 258
// instead of 200, five of them on one layer 45.5 instead of 42.7, the chunk below 309 instead of
// 221; at 128 the tokens below 561 instead of 487, the prompts 672 instead of 515.  f16
// weights are taken 2^7 times as large, so that what falls below its range is 2^-32 of
// the reference.
//
// Head dimensions 64 and 128: a CTA holds two subtiles, each with its own four softmax
// warps (a row per thread), so that the tensor cores work on one while the other's softmax
// runs; half of a block's weights are handed on while the others are made.  Head dimension
// 256: O takes half of tensor memory, so that a CTA holds one subtile, with two buffers of
// S and two threads per row, 64 keys each.  Pairs of CTAs (256, and 128 where WIDE) share
// products of 256 rows, each with half of the keys and half of V's columns in its shared
// memory: its operand reads and the copies halve.  P lies over its S.  The products of a CTA
// run in the order they are issued, so that the next block's scores follow the product that
// reads the weights they overwrite without a wait in between.
//
// K and V come by tensor copies of whole page rows (boxes of at most 64 positions of
// one head), a lane per box; a box past the request's last position is aimed outside the
// array, which fills zeros without reading.  Rows of a last page behind the last
// position are cleared before the product with V (a weight of 0 times NaN is NaN).
//
// The work is cut as page_walk.cuh says.  A tile cut into pieces leaves partials (m,
// l, O) in the workspace; the CTA that finishes a tile's last piece joins them in
// the pieces' order.  Few rows over few keys are page_few.cuh's.
//
// Warps 0-7 softmax, 8 issues the products, 9 walks the list and copies K and V, 10
// brings the queries, 11 only gives its registers.  Every wait is bounded; a thread whose wait
// gives up waits no more, the call reports LBX_ETIMEOUT, and the CTA leaves after its copies
// have landed.
//
// What bounds it, measured on one GB300 (copies reach 6.79 TB/s, cuBLAS 1898 TFLOP/s in
// bf16).  A chunk of 2048 tokens over 6144 keys, 24/4 heads of 256: 221 us, 1630 TFLOP/s, the
// tensor pipe.  Prompts of 501 to 6001 tokens, 32/8 heads of 128: 512 us, 1355 TFLOP/s, the chain
// from scores to weights (2900 cycles per block, 2060 of products).  16 requests of one token over
// 8001 to 16384 keys, 4 layers, 32/8 heads of 128 in f16: 485 us, 6.59 TB/s.  Trees of 22, five
// requests of 2049 to 4096 keys, 16 layers, 24/4 heads of 256: 200 us, 5.3 TB/s and what beginning
// and ending a tile takes (7 us).
#pragma once

#include "cache_ptx.cuh"
#include "cache_walk.cuh"
#include "page_few.cuh"
#include "page_walk.cuh"

namespace lbx {
namespace paged {

using cache::Ring;

// Registers per thread: at launch 168 (65536 for 384 threads); softmax takes what the other
// warps give: 256 * 208 + 128 * 80 <= 384 * 168.
constexpr int kSoftmaxRegs = 208, kOtherRegs = 80;
constexpr int kMaxCtas = cache::kMaxCtas;
// Keys of a block whose weights are handed on while the others are still made.
constexpr int kEarly = 64;
// Most rows whose pieces are joined by columns instead of by rows.
constexpr int kFewRows = 32;

// Floats of one partial: m (base 2) and l per row, then O as [dh / 4][128] of four.
__host__ __device__ constexpr size_t part_floats(int dh) { return 2 * kRows + (size_t)kRows * dh; }

struct PageMaps {
  CUtensorMap q, o;  // (dh, Hq, M, L), boxes of 64 columns of whole tokens' heads
  CUtensorMap k, v;  // (dh, Hkv, positions of all layers' pools), boxes of 64 columns
};

// A CTA's share of a tile, as the walking warp publishes it.
struct Seg {
  int have, l, h, b;
  int row0, n, tok0, ctx;  // first row of the request, its tokens, the tile's first token
  int blk0, nb;
  int subs;                // subtiles with rows
  int pieces, mine, owner;
};

template <int DH, bool WIDE>
struct Lay {
  // a pair of CTAs per tile; one subtile per CTA, with two buffers of S and two threads per
  // row, or two subtiles
  static constexpr bool kOne = DH == 256, kPair = kOne || WIDE;
  static_assert(!WIDE || DH == 128, "half of V's columns fills a swizzled row of 64");
  static constexpr int kCtas = kPair ? 2 : 1, kSubs = kOne ? 1 : 2;
  static constexpr int kKeys = kBlk / kCtas, kCols = DH / kCtas;  // of a block, per CTA
  static constexpr int kMine = kOne ? 64 : 128;                   // keys per softmax thread
  static constexpr int kGroup = kOne ? 256 : 128;                 // threads of a subtile
  static constexpr int kOut = kOne ? DH / 2 : DH;                 // O's columns per thread
  static constexpr int kStage = kKeys * DH * 2;
  static_assert(kStage == kBlk * kCols * 2, "K and V take the same place");
  static constexpr int kQSub = kRows * DH * 2, kQBytes = kSubs * kQSub;
  // where whole subtiles' results wait for their copy out (where the ring can spare it)
  static constexpr bool kStaged = DH == 64 || WIDE;
  static constexpr int kOutBytes = kStaged ? kQBytes : 0;
  static constexpr int kStages = (224 * 1024 - kQBytes - kOutBytes) / kStage;  // 3 KB for the rest
  static_assert(kStages >= 4, "the next block's K beside this one's V");
  static constexpr int kSmemOut = kQBytes, kSmemRing = kSmemOut + kOutBytes;
  static constexpr int kSmemRed = kSmemRing + kStages * kStage;  // float [4][128]
  static constexpr int kSmemSegs = kSmemRed + 4 * kRows * 4;     // Seg [4]
  static constexpr int kSmemMisc = kSmemSegs + 4 * (int)sizeof(Seg);  // int [16]
  static constexpr int kSmemBars = kSmemMisc + 64;
  static constexpr int kNBars = 3 * kStages + 20;
  static constexpr int kSmemTotal = kSmemBars + kNBars * 8;
  static_assert(kSmemTotal <= 227 * 1024 && kSmemRing % 1024 == 0 && kSmemBars % 8 == 0, "shared");
  // tensor memory: two buffers of S / P, O of each subtile
  static constexpr uint32_t kColO = 2 * kBlk, kTmemCols = 512;
  static_assert(kColO + kSubs * DH <= kTmemCols, "tensor memory");
};

template <bool F16>
constexpr float kLift = F16 ? 7.f : 0.f;

// Whether p holds in any of the threads that share a named barrier.
__device__ __forceinline__ bool any_of(uint32_t id, uint32_t nthreads, bool p) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %3, 0;\n\t"
      "barrier.cta.red.or.pred q, %1, %2, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(id), "r"(nthreads), "r"((uint32_t)p)
      : "memory");
  return r != 0;
}

// Where a CTA's range of the list begins.
struct Begin {
  Cut cut;
  i64 from, X;  // the range's first entry, that of the tile it lies in
  int lh, b, t;
};

// Requests of a warp's share of the sums, a multiple of the lanes.
__device__ __forceinline__ int share_of(int Bq) {
  return (Bq + kThreads - 1) / kThreads * 32;
}

// Checks the batch and adds up the list's entries of the warp's share of the requests, and
// the units of few rows (`units`: of all requests); the same verdict in every thread
// and every block (after a barrier of the block).
__device__ __forceinline__ int check_batch(const PageArgs &A, i64 *warps, int &units) {
  const lbx_page_cfg &c = A.c;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, share = share_of(c.Bq);
  int *few = reinterpret_cast<int *>(warps + kThreads / 32);
  int bad = A.parent ? trees_bad(c, A.start, A.parent, warp, kThreads / 32) : 0;
  i64 sum = 0;
  int own = 0;
#pragma unroll 1
  for (int b = warp * share + lane; b < (warp + 1) * share && b < c.Bq; b += 32) {
    const int s = A.start[b], e = A.start[b + 1], ctx = A.ctx_len[b];
    if (request_bad(c, b, s, e, ctx, A.parent != nullptr)) {
      bad = 1;
    } else {
      sum += entries_of(A.shape, ctx, e - s);
      own = min(own + min(few_units(A, ctx, e - s), 1 << 20), 1 << 20);
    }
  }
  if (warp * share < c.Bq) {
#pragma unroll
    for (int d = 16; d; d >>= 1) {
      sum += __shfl_xor_sync(0xffffffffu, sum, d);
      own = min(own + __shfl_xor_sync(0xffffffffu, own, d), 1 << 20);
    }
  }
  if (lane == 0) warps[warp] = sum, few[warp] = own;
  const int verdict = __syncthreads_or(bad);
  units = 0;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) units = min(units + few[w], 1 << 20);
  return verdict;
}

// Inclusive sums over the lanes.
__device__ __forceinline__ i64 scan32_wide(i64 v) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int d = 1; d < 32; d *= 2) {
    const i64 o = __shfl_up_sync(0xffffffffu, v, d);
    if (lane >= d) v += o;
  }
  return v;
}

// Finds range `me` of the list for one of `ctas` CTAs (or pairs), by one warp: the warp
// whose share it begins in, the request, the tile. False if there is nothing for it.
__device__ __forceinline__ bool find_begin(const PageArgs &A, int me, int ctas, const i64 *warps,
                                           Window &win, Begin &g) {
  const lbx_page_cfg &c = A.c;
  const int lane = threadIdx.x & 31, share = share_of(c.Bq);
  i64 upto = 0, total = warps[0];
  if (c.Bq > share) {  // more than the first warp's share
    upto = scan32_wide(lane < kThreads / 32 ? warps[lane] : 0);
    total = __shfl_sync(0xffffffffu, upto, 31);
  }
  g.cut = cut_of(total * c.L * c.Hkv, ctas);
  if (total == 0 || me >= g.cut.n) return false;
  g.from = g.cut.at(me);
  g.lh = (int)quot(g.from, total);
  i64 y = g.from - g.lh * total;
  const int w = c.Bq > share ? __popc(__ballot_sync(0xffffffffu, upto <= y)) : 0;
  if (w > 0) y -= __shfl_sync(0xffffffffu, upto, w - 1);
#pragma unroll 1
  for (int b0 = w * share;; b0 += 32) {
    if (b0 != win.b0) win.load(A, b0);
    upto = scan32_wide(entries_of(A.shape, win.ctx, win.n));
    const int k = __popc(__ballot_sync(0xffffffffu, upto <= y));
    if (k < 32) {
      if (k > 0) y -= __shfl_sync(0xffffffffu, upto, k - 1);
      g.b = b0 + k;
      break;
    }
    y -= __shfl_sync(0xffffffffu, upto, 31);
  }
  const int ctx = __shfl_sync(0xffffffffu, win.ctx, g.b - win.b0);
  const int n = __shfl_sync(0xffffffffu, win.n, g.b - win.b0);
  g.t = 0;
  i64 before = 0;
#pragma unroll 1
  for (int size = tiles_of(A.shape, n); size > 1;) {  // the last tile that begins at y or before
    const int step = (size + 31) / 32;
    const bool in = (i64)lane * step < size;
    const i64 e = in ? entries_upto(A.shape, ctx, n, g.t + lane * step) : 0;
    const int k = __popc(__ballot_sync(0xffffffffu, in && e <= y)) - 1;
    before = __shfl_sync(0xffffffffu, e, k);
    g.t += k * step;
    size = size - k * step < step ? size - k * step : step;
  }
  g.X = g.from - (y - before);
  return true;
}

// The largest of three (a NaN is passed over).
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

template <int DH, bool F16, bool WIDE, bool SPLIT>
__global__ void __launch_bounds__(kThreads, 1)
    page_attn_kernel(const __grid_constant__ PageMaps maps, const __grid_constant__ PageArgs A) {
  using Y = Lay<DH, WIDE>;
  constexpr bool PAIR = Y::kPair, ONE = Y::kOne;
  extern __shared__ __align__(1024) unsigned char page_smem[];
  unsigned char *smem = page_smem;
  const lbx_page_cfg &c = A.c;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  float *red = reinterpret_cast<float *>(smem + Y::kSmemRed);
  volatile Seg *segs = reinterpret_cast<volatile Seg *>(smem + Y::kSmemSegs);
  // [0] tensor memory base, [1] a wait gave up, [2] a page outside the pool, [4 + sub]
  // last of its tile's pieces
  volatile int *misc = reinterpret_cast<volatile int *>(smem + Y::kSmemMisc);
  uint64_t *full = reinterpret_cast<uint64_t *>(smem + Y::kSmemBars);
  uint64_t *empty = full + Y::kStages, *peer = empty + Y::kStages;
  uint64_t *s_bar = peer + Y::kStages, *p_bar = s_bar + 2, *p2_bar = p_bar + 2, *o_bar = p2_bar + 2;
  uint64_t *seg_bar = o_bar + 2, *seg_free = seg_bar + 4;
  uint64_t *q_bar = seg_free + 4, *qh_bar = q_bar + 1, *q_free = qh_bar + 1, *end_bar = q_free + 1;

  const int rank = PAIR ? (int)ptx::cluster_rank() : 0;
  const int me = blockIdx.x / Y::kCtas, ctas = gridDim.x / Y::kCtas;
  int units = 0;
  Window win;
  win.load(A, 0);
  if (check_batch(A, reinterpret_cast<i64 *>(red), units)) {
    if (tid == 0 && A.status) *A.status = LBX_ETREE;
    return;
  }
  if ((i64)units * c.L * c.Hkv <= (i64)kFewUnits * gridDim.x) {  // every CTA alike
    if (!few_rows<DH, F16>(A, units, win, smem) && A.status) *A.status = LBX_EINVAL;
    return;
  }
  if (tid == 0) {
    for (int i = 0; i < Y::kNBars; ++i)
      ptx::mbar_init(full + i, full + i >= p_bar && full + i < p_bar + 4
                                   ? Y::kCtas * Y::kGroup / 32
                               : full + i >= seg_free && full + i < seg_free + 4 ? 10
                               : full + i == q_bar ? Y::kCtas
                                                   : 1);
    ptx::fence_mbar_init();
    misc[1] = misc[2] = 0;
  }
  if (tid == 32) {
    ptx::prefetch_map(&maps.q);
    ptx::prefetch_map(&maps.k);
    ptx::prefetch_map(&maps.v);
    if (Y::kStaged) ptx::prefetch_map(&maps.o);
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
  if constexpr (PAIR) ptx::cluster_arrive();  // this CTA's barriers are set up
  ptx::tc_fence_after();
  const uint32_t tmem = static_cast<uint32_t>(misc[0]);

  bool bad = false;  // a wait of this thread gave up: it waits no more
  auto wait = [&](uint64_t *bar, uint32_t parity) {
    if (!bad && !ptx::mbar_wait(bar, parity)) bad = true;
    return !bad;
  };
  // Segment k, for every warp but the walking one; false when the list is done (or a
  // wait gave up).
  auto next_seg = [&](uint32_t k, Seg &s) {
    bool ok = wait(&seg_bar[k & 3], (k >> 2) & 1);
    if (ok) {
      const volatile Seg &f = segs[k & 3];
      s.have = f.have, s.l = f.l, s.h = f.h, s.b = f.b, s.row0 = f.row0, s.n = f.n;
      s.tok0 = f.tok0, s.ctx = f.ctx, s.blk0 = f.blk0, s.nb = f.nb, s.subs = f.subs;
      s.pieces = f.pieces, s.mine = f.mine, s.owner = f.owner;
    }
    __syncwarp();
    if (lane == 0) ptx::mbar_arrive(&seg_free[k & 3]);
    return ok && s.have != 0;
  };

  // (the warps that reach the other CTA wait until its barriers are set up; the walking
  // one does not, and waits at its end)
  if constexpr (PAIR) {
    if (warp != 9) ptx::cluster_wait();
  }
  if (warp == 9) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
    // ---- the walk, and copies of K and V ----
    Begin g;
    bool more = find_begin(A, me, ctas, reinterpret_cast<const i64 *>(red), win, g);
    const Cut cut = g.cut;
    int lh = g.lh, b = g.b, t = g.t, s0 = 0, n = 0, ctx = 0;
    auto request = [&]() {
      if (b < win.b0 || b >= win.b0 + 32) win.load(A, b & ~31);
      s0 = __shfl_sync(0xffffffffu, win.row0, b & 31);
      n = __shfl_sync(0xffffffffu, win.n, b & 31);
      ctx = __shfl_sync(0xffffffffu, win.ctx, b & 31);
    };
    if (more) request();
    i64 X = g.X;
    const i64 to = cut.at(me + 1);
    const int n_lh = c.L * c.Hkv;
    auto step = [&]() {  // to the next tile of the list
      X += kLead + blocks_of(A.shape, ctx, n, t);
      ++t;
#pragma unroll 1
      while (t >= tiles_of(A.shape, n)) {
        t = 0;
        if (++b == c.Bq) {
          b = 0;
          if (++lh == n_lh) return;
        }
        request();
      }
    };
    if (more) {
      const i64 y = g.from - X;
      if (y >= kLead + kLeast && y > kLead + blocks_of(A.shape, ctx, n, t) - kLeast) step();
    }
    // The range's next tile.
    auto advance = [&](Seg &s) {
      Piece p;
      const int nb = more && lh < n_lh ? blocks_of(A.shape, ctx, n, t) : 0;
      s.have = nb > 0 && piece_of(cut, me, g.from, to, X, nb, p);
      if (!s.have) return;
      s.l = lh / c.Hkv, s.h = lh - s.l * c.Hkv, s.b = b, s.row0 = s0, s.n = n, s.ctx = ctx;
      s.tok0 = t * A.shape.W, s.subs = n - s.tok0 > Y::kCtas * A.tp ? 2 : 1;
      s.blk0 = p.blk0, s.nb = p.blk1 - p.blk0;
      s.pieces = p.pieces, s.mine = p.mine, s.owner = p.owner;
      if (p.last) more = false;
      else step();
    };
    auto publish = [&](const Seg &s, uint32_t k) {
      if (k >= 4) wait(&seg_free[k & 3], ((k >> 2) & 1) ^ 1u);
      if (lane == 0) {
        volatile Seg &f = segs[k & 3];
        f.have = s.have;
        f.l = s.l, f.h = s.h, f.b = s.b, f.row0 = s.row0, f.n = s.n, f.ctx = s.ctx;
        f.tok0 = s.tok0, f.subs = s.subs, f.blk0 = s.blk0, f.nb = s.nb;
        f.pieces = s.pieces, f.mine = s.mine, f.owner = s.owner;
        ptx::mbar_arrive(&seg_bar[k & 3]);
      }
      __syncwarp();
    };
    Ring<Y::kStages> ring;
    int loads = 0, outside = 0;
    const uint32_t none = (uint32_t)(c.L * c.n_pages) * (uint32_t)c.page;  // past the pools' end
    Seg s, next;
    advance(s);
    publish(s, 0);
    // (a segment is published before the copies of the one before it, so that its
    // queries can come as soon as their place is free)
#pragma unroll 1
    for (uint32_t k = 0; s.have; ++k, s = next) {
      advance(next);
      if (__any_sync(0xffffffffu, bad)) next.have = 0;
      publish(next, k + 1);
      const int nb = s.nb;
      // Lane e brings box e of a block: `box` positions of one head, 64 columns.
      // The rows of its boxes come from the table one block ahead.
      const int kv_len = s.ctx + s.n;
      constexpr int kKA = DH / 64, kVA = Y::kCols / 64;
      const int k_boxes = Y::kKeys / A.box * kKA, v_boxes = kBlk / A.box * kVA;
      const int32_t *row = A.table + (size_t)s.b * c.max_pages;
      auto place = [&](int blk, int off) -> uint32_t {
        const int pos = blk * kBlk + off;
        if (pos >= kv_len) return none;
        const int id = row[pos >> A.shift];
        if (id < 0 || id >= c.n_pages) {
          outside = 1;
          return none;
        }
        return (uint32_t)(s.l * c.n_pages + id) * (uint32_t)c.page + (uint32_t)(pos & (c.page - 1));
      };
      const int k_off = lane / kKA * A.box + rank * Y::kKeys, v_off = lane / kVA * A.box;
      auto k_row = [&](int blk) { return lane < k_boxes ? place(blk, k_off) : none; };
      auto v_row = [&](int blk) { return lane < v_boxes ? place(blk, v_off) : none; };
      auto take = [&]() {
        // the first round finds every stage free
        const bool ok = __all_sync(0xffffffffu, wait(&empty[ring.st], ring.ph ^ 1u));
        if (ok && lane == 0) ptx::mbar_arrive_expect_tx(&full[ring.st], (uint32_t)Y::kStage);
        __syncwarp();
        loads += ok;
        return ok;
      };
      auto load_k = [&](uint32_t at) {
        if (take() && lane < k_boxes)
          ptx::tma_load_3d(smem + Y::kSmemRing + ring.st * Y::kStage + lane % kKA * (Y::kKeys * 128) +
                               lane / kKA * A.box * 128,
                           &maps.k, lane % kKA * 64, s.h, (int)at, &full[ring.st]);
        ring.step();
      };
      auto load_v = [&](uint32_t at) {
        if (take() && lane < v_boxes)
          ptx::tma_load_3d(smem + Y::kSmemRing + ring.st * Y::kStage + lane % kVA * (kBlk * 128) +
                               lane / kVA * A.box * 128,
                           &maps.v, rank * Y::kCols + lane % kVA * 64, s.h, (int)at, &full[ring.st]);
        ring.step();
      };
      uint32_t k_at = k_row(s.blk0), v_at = v_row(s.blk0);
#pragma unroll 1
      for (int i = 0; i < nb; ++i) {
        // K of block i; V of block i goes before K of block i + 1 where a CTA has two
        // subtiles, else behind it, as the products take them
        const int ahead = s.blk0 + (i + 1 < nb ? i + 1 : i);
        const uint32_t k_next = k_row(ahead), v_next = v_row(ahead);
        if (!ONE || i == 0) load_k(k_at);
        if (ONE && i + 1 < nb) load_k(k_next);
        load_v(v_at);
        k_at = k_next, v_at = v_next;
      }
    }
    if constexpr (PAIR) ptx::cluster_wait();
    outside = __any_sync(0xffffffffu, outside);
    if (lane == 0 && outside) misc[2] = 1;
    if (bad) misc[1] = 1;
    // every copy has landed before the CTA may leave (long since, unless a wait gave up)
    if (lane == 0) {
#pragma unroll 1
      for (int i = loads > Y::kStages ? loads - Y::kStages : 0; i < loads; ++i)
        (void)ptx::mbar_wait(&full[i % Y::kStages], (uint32_t)((i / Y::kStages) & 1));
    }
  } else if (warp == 10) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
    // ---- queries, by tensor copies (tokens past the last row read as zeros) ----
    Seg s;
    uint32_t k = 0;
    uint64_t *here = PAIR ? qh_bar : q_bar;
#pragma unroll 1
    for (; next_seg(k, s); ++k) {
      if (k > 0) wait(q_free, (k - 1) & 1);  // the last segment's score products are done
      if (lane == 0 && !bad) {
        const int live = ONE ? 1 : s.subs;
        ptx::mbar_arrive_expect_tx(here, (uint32_t)(live * A.tp * A.G * DH * 2));
#pragma unroll 1
        for (int e = 0; e < live; ++e)
#pragma unroll 1
          for (int a = 0; a < DH / 64; ++a)
            ptx::tma_load_4d(smem + e * Y::kQSub + a * kRows * 128, &maps.q, a * 64, s.h * A.G,
                             s.row0 + s.tok0 + (e * Y::kCtas + rank) * A.tp, s.l, here);
        if constexpr (PAIR) {
          if (wait(qh_bar, k & 1)) ptx::mbar_arrive_at(q_bar, 0);
        }
      }
      __syncwarp();
    }
    if (bad) misc[1] = 1;
    // no copy is left behind
    if (lane == 0 && k > 0) (void)ptx::mbar_wait(here, (k - 1) & 1);
  } else if (warp == 11) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
  } else if (warp == 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
    // ---- products: the warp waits as one, one lane issues ----
    Ring<Y::kStages> ring;
    uint32_t qs[2] = {0, 0};  // blocks so far, of each subtile (of a pair: in [0])
    const bool one = ptx::elect_one();
    const uint64_t qdesc = ptx::sdesc_sw128(ptx::smem_u32(smem));
    const uint64_t kdesc = ptx::sdesc_sw128(ptx::smem_u32(smem + Y::kSmemRing));
    const uint64_t vdesc = ptx::sdesc(ptx::smem_u32(smem + Y::kSmemRing), kBlk * 128, 1024u, 2u);
    auto commit = [&](uint64_t *bar) {
      if constexpr (PAIR) ptx::mma_commit_pair(bar);
      else ptx::mma_commit(bar);
    };
    auto wait_all = [&](uint64_t *bar, uint32_t parity) {
      bad = !__all_sync(0xffffffffu, wait(bar, parity));
      return !bad;
    };
    // Clear V's rows of the block in `stage` behind the request's last position, up to
    // the end of their box (boxes past it are zeros).
    auto clear = [&](const Seg &s, int blk, int stage) {
      const int from = s.ctx + s.n - blk * kBlk;
      if (from >= kBlk || from % A.box == 0) return;
      const int rows = (from + A.box - 1) / A.box * A.box - from;
      unsigned char *v0 = smem + Y::kSmemRing + stage * Y::kStage + from * 128;
      constexpr int kWide = Y::kCols / 8;  // 16-byte pieces of a row
#pragma unroll 1
      for (int i = lane; i < rows * kWide; i += 32)
        *reinterpret_cast<uint4 *>(v0 + (i % kWide / 8) * (kBlk * 128) + i / kWide * 128 +
                                   (i & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
      ptx::fence_proxy_async();
      if constexpr (PAIR) ptx::fence_cluster();
      __syncwarp();
    };
    Seg s;
    uint32_t k = 0;
    if (rank == 1) {
      // the follower tells the leader of each stage that has landed
#pragma unroll 1
      for (; next_seg(k, s); ++k) {
#pragma unroll 1
        for (int i = 0; i < 2 * s.nb; ++i, ring.step()) {
          // K 0, K 1, V 0, K 2, V 1, .., V nb - 1, or K 0, V 0, K 1, ..
          const bool is_v = ONE ? i == 2 * s.nb - 1 || (i > 0 && i % 2 == 0) : i % 2 == 1;
          if (!wait_all(&full[ring.st], ring.ph)) break;
          if (is_v) clear(s, s.blk0 + (!ONE ? i / 2 : i == 2 * s.nb - 1 ? s.nb - 1 : i / 2 - 1), ring.st);
          if (lane == 0) ptx::mbar_arrive_at(&peer[ring.st], 0);
        }
      }
      if (bad) misc[1] = 1;
    } else {
      constexpr uint32_t idesc_s = ptx::idesc_16(F16, kRows * Y::kCtas, kBlk, false);
      constexpr uint32_t idesc_o = ptx::idesc_16(F16, kRows * Y::kCtas, DH, true);
      auto arrived = [&](const Ring<Y::kStages> &r) {
        const bool ok = wait_all(&full[r.st], r.ph) && (!PAIR || wait_all(&peer[r.st], r.ph));
        ptx::tc_fence_after();
        return ok;
      };
      // S of subtile e (in a pair 0) into buffer `buf`
      auto scores = [&](int e, int buf, int stage) {
        const uint64_t kd = kdesc + (uint64_t)(stage * (Y::kStage >> 4));
        const uint64_t qd = qdesc + (uint64_t)(e * (Y::kQSub >> 4));
        if (one) {
#pragma unroll
          for (int i = 0; i < DH / 16; ++i) {
            const uint64_t qa = qd + (uint64_t)((i >> 2) * (kRows * 128 >> 4) + 2 * (i & 3));
            const uint64_t kb = kd + (uint64_t)((i >> 2) * (Y::kKeys * 128 >> 4) + 2 * (i & 3));
            if constexpr (PAIR) ptx::mma_16_ss_pair(tmem + buf * kBlk, qa, kb, idesc_s, i > 0);
            else ptx::mma_bf16_ss(tmem + buf * kBlk, qa, kb, idesc_s, i > 0);
          }
          commit(&s_bar[buf]);
        }
        __syncwarp();
      };
      // O of subtile e from the weights in `buf`: steps of 16 keys from `i0` on
      auto values = [&](int e, int buf, int stage, int i0, int i1, uint32_t later) {
        const uint64_t vd = vdesc + (uint64_t)(stage * (Y::kStage >> 4));
        if (one) {
#pragma unroll
          for (int part = 0; part < (SPLIT ? 2 : 1); ++part)
#pragma unroll
            for (int i = i0; i < i1; ++i) {
              const uint32_t pa = tmem + buf * kBlk + part * (kBlk / 2) + 8 * i;
              const uint32_t d = tmem + Y::kColO + e * DH;
              const uint64_t vb = vd + (uint64_t)(i * (2048 >> 4));
              const uint32_t acc = i > 0 || part > 0 ? 1u : later;
              if constexpr (PAIR) ptx::mma_16_ts_pair(d, pa, vb, idesc_o, acc);
              else ptx::mma_bf16_ts(d, pa, vb, idesc_o, acc);
            }
          if (i1 == kBlk / 16) commit(&o_bar[ONE ? buf : e]);
        }
        __syncwarp();
      };
      auto done = [&](uint64_t *bar) {
        if (one) commit(bar);
        __syncwarp();
      };
#pragma unroll 1
      for (; !bad && next_seg(k, s); ++k) {
        if (!wait_all(q_bar, k & 1) || !arrived(ring)) break;
        const int live = ONE ? 1 : s.subs;
#pragma unroll 1
        for (int e = 0; e < live; ++e) scores(e, ONE ? qs[0] & 1 : e, ring.st);
        done(&empty[ring.st]);
        if (s.nb == 1) done(q_free);
        ring.step();
#pragma unroll 1
        for (int i = 0; i < s.nb; ++i) {
          const bool next = i + 1 < s.nb;
          if constexpr (ONE) {
            if (next) {
              if (!arrived(ring)) break;
              scores(0, (qs[0] + 1) & 1, ring.st);
              done(&empty[ring.st]);
              if (i + 2 == s.nb) done(q_free);
              ring.step();
            }
            if (!arrived(ring)) break;
            clear(s, s.blk0 + i, ring.st);
            if (!wait_all(&p_bar[qs[0] & 1], (qs[0] >> 1) & 1)) break;
            ptx::tc_fence_after();
            values(0, qs[0] & 1, ring.st, 0, 8, i > 0);
            done(&empty[ring.st]);
            ring.step();
            ++qs[0];
          } else {
            if (!arrived(ring)) break;
            clear(s, s.blk0 + i, ring.st);
            Ring<Y::kStages> ahead = ring;
            ahead.step();
#pragma unroll 1
            for (int e = 0; e < live; ++e) {
              if (!wait_all(&p_bar[e], qs[e] & 1)) break;
              ptx::tc_fence_after();
              values(e, e, ring.st, 0, kEarly / 16, i > 0);
              if (!wait_all(&p2_bar[e], qs[e] & 1)) break;
              ptx::tc_fence_after();
              values(e, e, ring.st, kEarly / 16, 8, 1u);
              if (e == live - 1) done(&empty[ring.st]);
              if (next) {
                if (e == 0 && !arrived(ahead)) break;
                scores(e, e, ahead.st);
              }
              ++qs[e];
            }
            if (bad) break;
            if (next) {
              done(&empty[ahead.st]);
              if (i + 2 == s.nb) done(q_free);
              ring = ahead;
            }
            ring.step();
          }
        }
      }
      if (one) {
        if (bad) misc[1] = 1;
        commit(end_bar);
        (void)ptx::mbar_wait(end_bar, 0);
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
    // ---- softmax ----
    const int quad = warp & 3, hf = warp >> 2;  // hf: the subtile, or a pair's half of the row
    const int sub = ONE ? rank : hf * Y::kCtas + rank;  // subtile of the tile
    const int gt = ONE ? tid : tid & 127;      // thread of the subtile's group
    const uint32_t bar_id = ONE ? 5 : 5 + hf;
    const uint32_t tq = tmem + ((uint32_t)(quad * 32) << 16);
    const uint32_t to = tq + Y::kColO + (ONE ? hf * Y::kOut : hf * DH);  // this thread's O
    constexpr int kTileSubs = Y::kSubs * Y::kCtas;
    const int r = quad * 32 + lane;             // row of the subtile
    const float sl2 = A.scale_log2;
    auto tell = [&](uint64_t *bar) {
      __syncwarp();
      if (lane == 0) {
        if constexpr (PAIR) ptx::mbar_arrive_at(bar, 0);
        else ptx::mbar_arrive(bar);
      }
    };
    uint32_t q = 0, k = 0;
    Seg s;
#pragma unroll 1
    for (;; ++k) {
      // (all of a group's threads go on, or none)
      const bool over = !next_seg(k, s);
      if (any_of(bar_id, Y::kGroup, over)) break;
      if (!ONE && hf >= s.subs) continue;
      const int left = s.n - s.tok0 - sub * A.tp;  // tokens from the subtile's first on
      const int rows = (left < A.tp ? left : A.tp) * A.G;
      const int tok = s.tok0 + sub * A.tp + r / A.G;
      const bool real = r < rows, busy = quad * 32 < rows;
      // what the row sees: positions below `lim`, and of a tree the nodes in `path`
      int lim = real ? s.ctx + tok + 1 : 0x40000000;
      uint64_t path = 0;
      if (A.parent && real) {
        lim = s.ctx;
        const int32_t *up = A.parent + s.row0;
#pragma unroll 1
        for (int m = tok, d = 0; m >= 0 && d < LBX_ATTN_MAX_NODES; ++d) {
          path |= 1ull << m;
          m = up[m];
        }
      }
      float m_run = -INFINITY, l_run = 0.f;
#pragma unroll 1
      for (int i = 0; i < s.nb; ++i, ++q) {
        const int ch = ONE ? (int)(q & 1) : hf;
        const uint32_t ph = ONE ? (q >> 1) & 1 : q & 1;
        wait(&s_bar[ch], ph);
        ptx::tc_fence_after();
        if (!busy) {  // no rows: keep step with the others
          tell(&p_bar[ch]);
          if constexpr (!ONE) tell(&p2_bar[ch]);
          continue;
        }
        const uint32_t sc = tq + ch * kBlk;
        float sv[Y::kMine];
#pragma unroll
        for (int e = 0; e < Y::kMine; e += 32)
          ptx::tmem_ld32(sc + (ONE ? hf * 64 : 0) + e, *reinterpret_cast<float(*)[32]>(sv + e));
        ptx::tmem_wait_ld();
        const int k0 = (s.blk0 + i) * kBlk + (ONE ? hf * 64 : 0);
        if (!__all_sync(0xffffffffu, lim - k0 >= Y::kMine)) {
#pragma unroll
          for (int w = 0; w < Y::kMine / 64; ++w) {
            uint64_t ok = cache::low_bits(lim - k0 - 64 * w);
            const int by = k0 + 64 * w - lim;  // of a tree: the word's first key, from its root
            if (by >= 0) ok |= by < 64 ? path >> by : 0ull;
            else if (by > -64) ok |= path << -by;
#pragma unroll
            for (int e = 0; e < 64; ++e)
              if (!((uint32_t)(ok >> (e & 32)) >> (e & 31) & 1)) sv[64 * w + e] = -INFINITY;
          }
        }
        float mb;
        {
          float mx[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) mx[e] = max3(sv[3 * e], sv[3 * e + 1], sv[3 * e + 2]);
#pragma unroll
          for (int e = 12; e + 1 < Y::kMine; e += 2)
            mx[(e >> 1) & 3] = max3(mx[(e >> 1) & 3], sv[e], sv[e + 1]);
          mb = fmaxf(max3(mx[0], mx[1], mx[2]), mx[3]);
        }
        if constexpr (ONE) {
          // (two buffers: the other half may not have read the last block's yet)
          float *max_of = red + (q & 1) * 2 * kRows;
          max_of[hf * kRows + r] = mb;
          ptx::tc_fence_before();
          ptx::named_sync(1 + quad, 64);  // the row's other half: maxima out, scores read
          ptx::tc_fence_after();
          mb = fmaxf(mb, max_of[(1 - hf) * kRows + r]);
        }
        float alpha = 1.f;
        bool need = false;
        if ((mb - m_run) * sl2 > 8.f) {  // the first time too
          alpha = ptx::ex2((m_run - mb) * sl2);
          need = i > 0 && real;
          l_run *= alpha;
          m_run = mb;
        }
        const float ref = m_run == -INFINITY ? 0.f : fmaf(m_run, sl2, -kLift<F16>);
        // rows whose reference moved rescale O, once the previous product is done
        if (__any_sync(0xffffffffu, need)) {
          if constexpr (ONE) wait(&o_bar[(q - 1) & 1], ((q - 1) >> 1) & 1);
          else wait(&o_bar[hf], (q - 1) & 1);
          ptx::tc_fence_after();
#pragma unroll 1
          for (int e0 = 0; e0 < Y::kOut; e0 += 16) {
            float ov[16];
            uint32_t w[16];
            ptx::tmem_ld16(to + e0, ov);
            ptx::tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 16; ++e) w[e] = __float_as_uint(ov[e] * alpha);
            ptx::tmem_st16(to + e0, w);
          }
        }
        const uint64_t scale2 = both(sl2, sl2), ref2 = both(-ref, -ref);
        uint64_t sum[4] = {0, 0, 0, 0};
#pragma unroll
        for (int e0 = 0; e0 < Y::kMine; e0 += 32) {
          uint32_t pk[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const float2 x = apart2(fma2(both(sv[e0 + 2 * e], sv[e0 + 2 * e + 1]), scale2, ref2));
            const float p0 = ptx::ex2(x.x), p1 = ptx::ex2(x.y);
            sum[e & 3] = add2(sum[e & 3], both(p0, p1));
            pk[e] = pack2<F16>(p0, p1);
            if constexpr (SPLIT) sv[e0 + 2 * e] = p0, sv[e0 + 2 * e + 1] = p1;
          }
          ptx::tmem_st16(sc + (ONE ? hf * 32 : 0) + e0 / 2, pk);
          if constexpr (SPLIT) {  // the second part, over the rest of S
#pragma unroll
            for (int e = 0; e < 16; ++e)
              pk[e] = pack2_rest<F16>(sv[e0 + 2 * e], sv[e0 + 2 * e + 1], pk[e]);
            ptx::tmem_st16(sc + kBlk / 2 + (ONE ? hf * 32 : 0) + e0 / 2, pk);
          }
          if (!ONE && e0 == 32 * (kEarly / 32 - 1)) {  // most of the weights: their product may begin
            ptx::tmem_wait_st();
            ptx::tc_fence_before();
            tell(&p_bar[ch]);
          }
        }
        ptx::tmem_wait_st();
        ptx::tc_fence_before();
        tell(ONE ? &p_bar[ch] : &p2_bar[ch]);
        const float2 s2 = apart2(add2(add2(sum[0], sum[1]), add2(sum[2], sum[3])));
        l_run += s2.x + s2.y;
      }

      // ---- the segment's result: whole, or a partial ----
      if constexpr (ONE) wait(&o_bar[(q - 1) & 1], ((q - 1) >> 1) & 1);
      else wait(&o_bar[hf], (q - 1) & 1);
      ptx::tc_fence_after();
      float l_sum = l_run;
      if constexpr (ONE) {
        ptx::named_sync(1 + quad, 64);  // the last maxima are read
        red[hf * kRows + r] = l_run;
        ptx::named_sync(1 + quad, 64);
        l_sum = red[r] + red[kRows + r];
      }
      const float m2 = m_run == -INFINITY ? -INFINITY : fmaf(m_run, sl2, -kLift<F16>);
      if (Y::kStaged && gt == 0) ptx::bulk_wait_read_all();  // the last copy out has left its place
      const bool valid = !any_of(bar_id, Y::kGroup, bad);
      // A row's place among the outputs, and its lse.  (A NaN among a row's scores makes
      // its sum one, and the row with it.)
      auto place = [&](int rw) {
        const int token = s.tok0 + sub * A.tp + rw / A.G;
        return ((size_t)s.l * c.M + s.row0 + token) * c.Hq + s.h * A.G + rw % A.G;
      };
      auto finish = [&](int rw, float m, float sum) {
        if (A.lse) A.lse[place(rw)] = sum == 0.f ? -INFINITY : (m + log2f(sum)) * 0.6931471805599453f;
      };
      // Piece e > 0 lies at its range's first place, the first piece at its second.
      auto partial = [&](int e) {
        const int at = 2 * (s.owner + e) + (e == 0 ? 1 : 0);
        return A.part + (size_t)(kTileSubs * at + sub) * part_floats(DH);
      };
      constexpr int kCol0 = ONE ? Y::kOut : 0;  // this thread's first column: hf times this
      bool join = false;
      if (s.pieces > 1 && rows > 0) {
        float *mine = partial(s.mine);
        if (busy && valid) {
#pragma unroll 1
          for (int e0 = 0; e0 < Y::kOut; e0 += 32) {
            float ov[32];
            ptx::tmem_ld32(to + e0, ov);
            ptx::tmem_wait_ld();
            if (!real) continue;
            float4 *at = reinterpret_cast<float4 *>(mine + 2 * kRows) + (hf * kCol0 + e0) / 4 * kRows + r;
#pragma unroll
            for (int e = 0; e < 8; ++e)
              at[e * kRows] = make_float4(ov[4 * e], ov[4 * e + 1], ov[4 * e + 2], ov[4 * e + 3]);
          }
          if (real && (!ONE || hf == 0)) mine[r] = m2, mine[kRows + r] = l_sum;
        }
        ptx::named_sync(bar_id, Y::kGroup);
        if (gt == 0) {
          unsigned int *count = A.counters + kTileSubs * s.owner + sub;
          const bool last = arrive_count(count) == (unsigned)s.pieces - 1;
          if (last) *count = 0u;  // for the next call
          misc[4 + sub] = last;
        }
        ptx::named_sync(bar_id, Y::kGroup);
        join = misc[4 + sub] != 0;
      }
      if (join && valid && rows <= kFewRows) {
        // four columns of a row per thread, eight pieces' loads in flight, the reference
        // moving as it does over blocks of keys
#pragma unroll 1
        for (int idx = gt; idx < rows * (DH / 4); idx += Y::kGroup) {
          const int rw = idx % rows, c4 = idx / rows;
          float top = -INFINITY, sum = 0.f;
          float4 f = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
          for (int e0 = 0; e0 < s.pieces; e0 += 8) {
            float4 y[8];
            float m[8], l[8], most = top;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const bool in = e0 + e < s.pieces;
              const float *from = partial(in ? e0 + e : e0);
              m[e] = __ldcg(from + rw), l[e] = __ldcg(from + kRows + rw);
              y[e] = __ldcg(reinterpret_cast<const float4 *>(from + 2 * kRows) + (size_t)c4 * kRows + rw);
              if (!in) m[e] = -INFINITY;
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) most = fmaxf(most, m[e]);
            const float base = most == -INFINITY ? 0.f : most;
            const float old = ptx::ex2(top - base);
            f.x *= old, f.y *= old, f.z *= old, f.w *= old, sum *= old;
            top = most;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const float w = ptx::ex2(m[e] - base);
              sum = fmaf(w, l[e], sum);
              f.x = fmaf(w, y[e].x, f.x), f.y = fmaf(w, y[e].y, f.y);
              f.z = fmaf(w, y[e].z, f.z), f.w = fmaf(w, y[e].w, f.w);
            }
          }
          const float inv = sum == 0.f ? 0.f : 1.f / sum;
          const uint2 u = make_uint2(pack2<F16>(f.x * inv, f.y * inv), pack2<F16>(f.z * inv, f.w * inv));
          reinterpret_cast<uint2 *>(A.o + place(rw) * DH)[c4] = sum == 0.f ? make_uint2(0u, 0u) : u;
          if (c4 == 0) finish(rw, top, sum);
        }
      } else if (Y::kStaged && s.pieces == 1 && valid && rows == A.tp * A.G) {
        // a whole subtile: through shared memory, as the tensor copy reads it (rows of 128
        // bytes, 16-byte pieces swizzled), which runs beside the next tile
        unsigned char *out = smem + Y::kSmemOut + hf * Y::kQSub;
        if (busy) {
          const float w = l_sum == 0.f ? 0.f : 1.f / l_sum;
          if (real) finish(r, m2, l_sum);
#pragma unroll 1
          for (int e0 = 0; e0 < DH; e0 += 32) {
            float v[32];
            ptx::tmem_ld32(to + e0, v);
            ptx::tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              uint32_t u[4];
#pragma unroll
              for (int f = 0; f < 4; ++f)
                u[f] = l_sum == 0.f ? 0u : pack2<F16>(v[8 * e + 2 * f] * w, v[8 * e + 2 * f + 1] * w);
              const int piece = (e0 / 8 + e) & 7;
              *reinterpret_cast<uint4 *>(out + (e0 / 64) * (kRows * 128) + r * 128 +
                                         ((piece ^ (r & 7)) << 4)) = make_uint4(u[0], u[1], u[2], u[3]);
            }
          }
          ptx::fence_proxy_async();
        }
        ptx::named_sync(bar_id, Y::kGroup);
        if (gt == 0) {
#pragma unroll 1
          for (int a = 0; a < DH / 64; ++a)
            ptx::tma_store_4d(&maps.o, a * 64, s.h * A.G, s.row0 + s.tok0 + sub * A.tp, s.l,
                              out + a * kRows * 128);
          ptx::bulk_commit();
        }
      } else if (busy && valid && (s.pieces == 1 || join)) {
        // a row per thread (or half of one); this CTA's piece is still in tensor memory,
        // the others' are added in the pieces' order, whichever CTA joins them
        float top = m2, sum = l_sum;
        if (join) {
          top = -INFINITY, sum = 0.f;
#pragma unroll 1
          for (int e0 = 0; e0 < s.pieces; e0 += 4) {
            float m[4], l[4], most = top;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const bool in = e0 + e < s.pieces;
              const float *from = partial(in ? e0 + e : e0) + r;
              m[e] = __ldcg(from), l[e] = __ldcg(from + kRows);
              if (!in) m[e] = -INFINITY;
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) most = fmaxf(most, m[e]);
            const float base = most == -INFINITY ? 0.f : most;
            sum *= ptx::ex2(top - base);
            top = most;
#pragma unroll
            for (int e = 0; e < 4; ++e) sum = fmaf(ptx::ex2(m[e] - base), l[e], sum);
          }
          if (top == -INFINITY) top = 0.f;
        }
        const float w = sum == 0.f ? 0.f : 1.f / sum;
        if (real && (!ONE || hf == 0)) finish(r, top, sum);
        const float w_own = join ? ptx::ex2(m2 - top) * w : w;
        // where the four rows of this lane's group of lanes go
        uint64_t rows_at[4];
        {
          const uint64_t at = real ? reinterpret_cast<uint64_t>(A.o + place(r) * DH + hf * kCol0) : 0ull;
#pragma unroll
          for (int e = 0; e < 4; ++e) rows_at[e] = __shfl_sync(0xffffffffu, at, (lane & ~3) + e);
        }
#pragma unroll 1
        for (int e0 = 0; e0 < Y::kOut; e0 += 32) {
          float v[32];
          ptx::tmem_ld32(to + e0, v);
          ptx::tmem_wait_ld();
          if (join) {
            float own[32];
#pragma unroll
            for (int e = 0; e < 32; ++e) own[e] = v[e], v[e] = 0.f;
#pragma unroll 1
            for (int e = 0; e < s.pieces; ++e) {
              if (e == s.mine) {
#pragma unroll
                for (int f = 0; f < 32; ++f) v[f] = fmaf(w_own, own[f], v[f]);
              } else if (real) {
                const float *from = partial(e);
                const float w_e = ptx::ex2(__ldcg(from + r) - top) * w;
                const float4 *at = reinterpret_cast<const float4 *>(from + 2 * kRows) +
                                   (hf * kCol0 + e0) / 4 * kRows + r;
                float4 y[8];
#pragma unroll
                for (int f = 0; f < 8; ++f) y[f] = __ldcg(at + f * kRows);
#pragma unroll
                for (int f = 0; f < 8; ++f) {
                  v[4 * f] = fmaf(w_e, y[f].x, v[4 * f]), v[4 * f + 1] = fmaf(w_e, y[f].y, v[4 * f + 1]);
                  v[4 * f + 2] = fmaf(w_e, y[f].z, v[4 * f + 2]), v[4 * f + 3] = fmaf(w_e, y[f].w, v[4 * f + 3]);
                }
              }
            }
          } else {
#pragma unroll
            for (int e = 0; e < 32; ++e) v[e] *= w;
          }
          uint32_t pc[4][4];
#pragma unroll
          for (int e = 0; e < 16; ++e)
            pc[e >> 2][e & 3] = sum == 0.f ? 0u : pack2<F16>(v[2 * e], v[2 * e + 1]);
          // four lanes exchange 16-byte pieces, so that a store of the warp writes 64
          // bytes of eight rows instead of 16 of thirty-two
#pragma unroll
          for (int d = 1; d <= 2; d *= 2) {
            const bool up = lane & d;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              if (e & d) continue;
#pragma unroll
              for (int f = 0; f < 4; ++f) {
                const uint32_t got = __shfl_xor_sync(0xffffffffu, up ? pc[e][f] : pc[e + d][f], d);
                if (up) pc[e][f] = got;
                else pc[e + d][f] = got;
              }
            }
          }
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (rows_at[e])
              reinterpret_cast<uint4 *>(rows_at[e])[e0 / 8 + (lane & 3)] =
                  make_uint4(pc[e][0], pc[e][1], pc[e][2], pc[e][3]);
        }
      }
      ptx::tc_fence_before();
      ptx::named_sync(bar_id, Y::kGroup);  // red is free again
    }
    if (bad) misc[1] = 1;
    if (Y::kStaged && gt == 0) ptx::bulk_wait_all();
  }

  ptx::tc_fence_before();
  __syncthreads();
  if constexpr (PAIR) ptx::cluster_sync();  // neither leaves while the other may reach it
  if (tid == 0 && A.status) {
    if (misc[1]) *A.status = LBX_ETIMEOUT;
    else if (misc[2]) *A.status = LBX_EINVAL;
  }
  if (warp == 8) {
    ptx::tc_fence_after();
    if constexpr (PAIR) ptx::tmem_dealloc_pair(tmem, Y::kTmemCols);
    else ptx::tmem_dealloc(tmem, Y::kTmemCols);
  }
}

// Launches of one head dimension (instances in page_attn_*.cu).
template <int DH, bool WIDE, bool SPLIT>
cudaError_t launch_page_attn(bool f16, const PageMaps &maps, const PageArgs &A, int grid,
                             cudaStream_t stream);
template <int DH, bool F16, bool WIDE, bool SPLIT>
cudaError_t launch_page_attn_of(const PageMaps &maps, const PageArgs &A, int grid,
                                cudaStream_t stream) {
  auto kernel = page_attn_kernel<DH, F16, WIDE, SPLIT>;
  constexpr int bytes = Lay<DH, WIDE>::kSmemTotal;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid), cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = bytes, cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = Lay<DH, WIDE>::kCtas, at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at, cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, maps, A);
}

}  // namespace paged
}  // namespace lbx
