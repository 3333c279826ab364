// cache_mass.cu -- attention weights per key, gathered over the queries of the
// accepted path, on the tensor cores: lbx_attention_mass.
//
//   score[j] += sum over rows r (path node, head of the group) of
//               exp(scale q_r . k_j - lse_r)
//
// The product is taken as S^T = K Q^T: keys are the 128 lanes of tensor memory
// and the path's queries its columns, so that a thread has all weights of its
// key and sums them by itself, in row order: no exchange between threads, no
// maximum (the lse is known), no atomics.  K is read once and the work on it
// is 2 dh operations per row and key, far below what the tensor cores do in
// the time a key takes to arrive: the kernel is bound by reading K.
//
// The tensor cores truncate as they accumulate, about half a unit in the 24th bit
// of the running sum per 16 columns; a weight takes the score's absolute error as
// its relative one.  So parts of the head dimension have accumulators of their own,
// as many as the columns of tensor memory allow, and are added here: four up to 64
// rows per pass, two up to 128, else one.  Error of the path keys' sums against 64 bits
// (2-norms): 0.4e-6 at most with four (dimension 256, where two gave 0.75e-6 and
// operations in fp32 give 0.5e-6), 1.0e-6 with one (dimension 128; fp32: 0.6e-6 to 0.8e-6).
//
// The path's nodes are taken root first, so row d G + h belongs to the node of
// depth d, and the rows that see a key are one range of rows.  Up to 128 rows
// (256 for head dimensions below 256) are multiplied at a time; longer paths
// take further passes over the CTA's keys, each added to the same scores by
// the same threads.  Keys come as blocks of two units (cache_walk.cuh), cut into
// equal ranges, one per CTA; nothing has to be joined.  Warps 0-3 and 4-7 take
// the blocks in turn, each with a score buffer of its own; warp 8 issues the
// MMAs, warp 9 the copies, through a ring of 16 KB pieces (128 keys x 64
// columns).  Waits are bounded as in the attention kernel.
//
// Measured: 16 layers, five requests of 4097 to 8192 keys, paths of 6 nodes, 24/4
// heads of dimension 256: 167 us, 6.2 TB/s (91% of a copy's rate); one layer, one
// token, 3001 keys: 10.3 us, launch and host call.  Paths of 40 nodes at 4 heads per
// group: 74 us, 45%: 160 exponentials per key.
#include "cache_ptx.cuh"
#include "cache_walk.cuh"

namespace lbx {
namespace cache {
namespace {

struct MassArgs {
  int L, Hq, Hkv, G, n_req, fixed, Bq, N, T, window, n_sink;
  int cap, stages;  // rows per pass, ring stages
  static constexpr int join = 0;  // pieces of a stream need no joining
  float scale;
  PerGroup per;
  Tiling til;
  const int32_t *ctx_len, *parent, *accepted;
  const uint16_t *q;
  const float *lse;
  float *score, *score_tree;
  int32_t *status;
};

constexpr int kThreads = 320;
constexpr int kMaxRows = 256;    // rows per pass
constexpr int kMaxStages = 13;
// shared memory after the Q rows and the ring
constexpr int kTailLse = 0;                              // float [256]
constexpr int kTailNodes = kTailLse + kMaxRows * 4;      // int [64]
constexpr int kTailMisc = kTailNodes + kMaxNodes * 4;    // int [4]
constexpr int kTailBars = kTailMisc + 16;                // full, empty, s[2], free[2], q, end
constexpr int kTail = kTailBars + (2 * kMaxStages + 6) * 8;
static_assert(kTail <= 3072, "shared memory");
constexpr int kMostBytes = 227 * 1024;

// Accumulators of a score buffer's 256 columns for a pass of nr rows: parts of the head
// dimension, each with its own.
__device__ __forceinline__ int accumulators(int nr) { return nr <= 64 ? 4 : nr <= 128 ? 2 : 1; }

template <int DH, bool F16>
__global__ void __launch_bounds__(kThreads, 1)
    mass_kernel(const __grid_constant__ AttnMaps maps, const __grid_constant__ MassArgs A) {
  constexpr int kPieces = DH / 64;  // per block of 128 keys
  extern __shared__ __align__(1024) unsigned char cache_smem[];
  unsigned char *ring_mem = cache_smem + A.cap * DH * 2, *tail = ring_mem + A.stages * kPiece;
  float *lse_of = reinterpret_cast<float *>(tail + kTailLse);
  int *nodes = reinterpret_cast<int *>(tail + kTailNodes);
  volatile int *misc = reinterpret_cast<volatile int *>(tail + kTailMisc);  // TMEM base, gave up
  uint64_t *full = reinterpret_cast<uint64_t *>(tail + kTailBars);
  uint64_t *empty = full + kMaxStages, *s_bar = empty + kMaxStages, *free_bar = s_bar + 2;
  uint64_t *q_bar = free_bar + 2, *end_bar = q_bar + 1;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  if (batch_bad(A.Bq, A.N, A.T, A.ctx_len, A.parent, A.accepted)) {
    if (tid == 0 && A.status) *A.status = LBX_ETREE;
    return;
  }
  if (tid == 0) {
#pragma unroll 1
    for (int i = 0; i < 2 * kMaxStages + 6; ++i)
      ptx::mbar_init(full + i, full + i == q_bar                             ? 8
                               : full + i == free_bar || full + i == free_bar + 1 ? 4
                                                                                  : 1);
    ptx::fence_mbar_init();
    misc[1] = 0;
  }
  if (warp == 8) {
    ptx::tmem_alloc(reinterpret_cast<uint32_t *>(tail + kTailMisc), 512);
    ptx::tmem_relinquish();
    ptx::tc_fence_before();
  }
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = static_cast<uint32_t>(misc[0]);
  Walk<2, 3, MassArgs> W(A, lane);
  bool bad = false;  // a wait of this thread gave up: it waits no more
  auto wait = [&](uint64_t *bar, uint32_t parity) {
    if (!bad && !ptx::mbar_wait(bar, parity)) bad = true;
    return !bad;
  };
  int req = -1;
  uint64_t path = 0;
  auto rows_of = [&]() {  // query rows of the walk's request
    if (W.b != req) {
      req = W.b;
      path = warp_path(A.parent + (size_t)req * A.N, A.N, A.accepted[req], lane);
    }
    return __popcll(path) * A.G;
  };

  if (warp == 9) {
    // ---- copies ----
    int st = 0, loads = 0;
    uint32_t ph = 0;
    ptx::named_sync(6, 256 + 32);  // behind the first queries' loads
#pragma unroll 1
    while (W.next()) {
      const int rows = rows_of(), z = W.l * A.n_req + W.b;
      // the segment's queries into L2, ahead of its keys: loads of them would
      // wait for all the copies in flight
#pragma unroll 1
      for (int n = lane; n < A.N; n += 32)
        if (path >> n & 1)
          ptx::prefetch_bytes(A.q + (((size_t)z * A.N + n) * A.Hq + W.h * A.G) * DH,
                              (uint32_t)(A.G * DH * 2));
      __syncwarp();
#pragma unroll 1
      for (int r0 = 0; r0 < rows && lane == 0; r0 += A.cap)
#pragma unroll 1
        for (int blk = W.blk0; blk < W.blk1 && !bad; ++blk) {
          int start[2], cnt;
          bool tree[2];
          W.unit(2 * blk, start[0], tree[0], cnt);
          W.unit(2 * blk + 1, start[1], tree[1], cnt);
#pragma unroll 1
          for (int a = 0; a < kPieces; ++a) {
            if (!wait(&empty[st], ph ^ 1u)) break;
            ptx::mbar_arrive_expect_tx(&full[st], (uint32_t)kPiece);
            unsigned char *d = ring_mem + st * kPiece;
#pragma unroll
            for (int u = 0; u < 2; ++u)
              ptx::tma_load_4d(d + u * kUnit * 128, tree[u] ? &maps.kt : &maps.k, a * 64, W.h,
                               start[u], z, &full[st]);
            ++loads;
            if (++st == A.stages) st = 0, ph ^= 1u;
          }
        }
      __syncwarp();
    }
    if (lane == 0) {
      if (bad) misc[1] = 1;
      // every copy has landed before the CTA may leave
#pragma unroll 1
      for (int i = loads > A.stages ? loads - A.stages : 0; i < loads; ++i)
        (void)ptx::mbar_wait(&full[i % A.stages], (uint32_t)((i / A.stages) & 1));
    }
  } else if (warp == 8) {
    // ---- MMAs: the warp walks and waits as one, one lane issues ----
    int st = 0;
    uint32_t ph = 0, seg = 0, used[2] = {0, 0};
    const bool one = ptx::elect_one();
    const uint64_t kdesc = ptx::sdesc_sw128(ptx::smem_u32(ring_mem));
    const uint64_t qdesc = ptx::sdesc_sw128(ptx::smem_u32(cache_smem));
    auto wait_all = [&](uint64_t *bar, uint32_t parity) {
      bad = !__all_sync(0xffffffffu, wait(bar, parity));
      return !bad;
    };
#pragma unroll 1
    while (!bad && W.next()) {
      const int rows = rows_of();
#pragma unroll 1
      for (int r0 = 0; r0 < rows && !bad; r0 += A.cap, ++seg) {
        const int nr = (rows - r0 < A.cap ? rows - r0 + 31 : A.cap) & ~31;
        const uint32_t idesc = ptx::idesc_16(F16, 128, nr, false);
        const int acc = accumulators(nr), per = DH / 16 / acc;
        if (!wait_all(q_bar, seg & 1)) break;
#pragma unroll 1
        for (int i = 0; i < W.blk1 - W.blk0 && !bad; ++i) {
          const int buf = i & 1;
          if (!wait_all(&free_bar[buf], (used[buf] & 1) ^ 1u)) break;
#pragma unroll 1
          for (int a = 0; a < kPieces; ++a) {
            if (!wait_all(&full[st], ph)) break;
            ptx::tc_fence_after();
            const uint64_t kd = kdesc + (uint64_t)(st * (kPiece >> 4));
            const uint64_t qd = qdesc + (uint64_t)(a * A.cap * (128 >> 4));
            if (one) {
#pragma unroll
              for (int s = 0; s < 4; ++s) {
                const int step = a * 4 + s, at = step / per;
                ptx::mma_bf16_ss(tmem + buf * 256 + at * (256 / acc), kd + 2 * s, qd + 2 * s, idesc,
                                 step > at * per ? 1u : 0u);
              }
              ptx::mma_commit(&empty[st]);
              if (a == kPieces - 1) ptx::mma_commit(&s_bar[buf]);
            }
            __syncwarp();
            if (++st == A.stages) st = 0, ph ^= 1u;
          }
          ++used[buf];
        }
      }
    }
    if (one) {
      if (bad) misc[1] = 1;
      ptx::mma_commit(end_bar);
      (void)ptx::mbar_wait(end_bar, 0);
    }
  } else {
    // ---- Q rows in, weights out ----
    const int wg = warp >> 2;
    const int key = (warp & 3) * 32 + lane;  // of a block: its lane of tensor memory
    const uint32_t tq = tmem + ((uint32_t)((warp & 3) * 32) << 16) + wg * 256;
    uint32_t used = 0;
    bool ahead = true;
    auto go_ahead = [&]() {
      if (ahead) asm volatile("bar.arrive 6, %0;" ::"n"(256 + 32) : "memory");
      ahead = false;
    };
#pragma unroll 1
    while (W.next()) {
      const int rows = rows_of(), len = rows / A.G;
      const size_t lb = (size_t)W.l * A.n_req + W.b, lbg = lb * A.Hkv + W.h;
      if (tid < kMaxNodes && (path >> tid & 1))
        nodes[__popcll(path & ((1ull << tid) - 1))] = tid;
#pragma unroll 1
      for (int r0 = 0; r0 < rows; r0 += A.cap) {
        const int in = rows - r0 < A.cap ? rows - r0 : A.cap, nr = (in + 31) & ~31;
        ptx::named_sync(5, 256);  // nodes are listed; the last pass is done everywhere
        constexpr int kPer = DH / 8;  // 16-byte pieces per row
        auto query = [&](int r) {  // row r of the pass among all queries
          const int d = A.per.node(r0 + r);
          return (lb * A.N + nodes[d]) * A.Hq + W.h * A.G + (r0 + r - d * A.G);
        };
        // all of a thread's loads in flight, the first tile's ahead of the copies
        constexpr int kStep = 256 / kPer, kLoads = (DH == 256 ? 128 : kMaxRows) / kStep;
        const int piece = tid % kPer, r1 = tid / kPer;
        uint4 v[kLoads];
#pragma unroll
        for (int e = 0; e < kLoads; ++e) {
          const int r = r1 + e * kStep;
          v[e] = make_uint4(0u, 0u, 0u, 0u);
          if (r < in) v[e] = reinterpret_cast<const uint4 *>(A.q)[query(r) * kPer + piece];
        }
        go_ahead();
#pragma unroll
        for (int e = 0; e < kLoads; ++e) {
          const int r = r1 + e * kStep;
          if (r < nr)
            *reinterpret_cast<uint4 *>(cache_smem + (piece / 8) * A.cap * 128 + r * 128 +
                                       ((piece & 7) ^ (r & 7)) * 16) = v[e];
        }
        if (tid < nr) {
          // rows past the last, and those without a finite score, weigh nothing
          const float z = tid < in ? A.lse[query(tid)] : -INFINITY;
          lse_of[tid] = z == -INFINITY ? INFINITY : z;
        }
        ptx::fence_proxy_async();
        ptx::named_sync(5, 256);
        if (lane == 0) ptx::mbar_arrive(q_bar);

#pragma unroll 1
        for (int i = wg; i < W.blk1 - W.blk0; i += 2) {
          int start, cnt;
          bool tree;
          W.unit(2 * (W.blk0 + i) + (key >> 6), start, tree, cnt);
          const int off = key & 63;
          // the range of rows that see the key, and where its sum goes
          int lo = 0, hi = rows;
          float *to = nullptr;
          if (off < cnt && !tree) {
            const int j = start + off;
            if (A.window > 0 && j >= A.n_sink) {
              const int d = A.window - W.ctx + j;  // depths below see it
              hi = d >= len ? rows : d > 0 ? d * A.G : 0;
            }
            to = A.score + lbg * A.T + j;
          } else if (off < cnt) {
            const int d = __popcll(path & ((2ull << off) - 1)) - 1;
            lo = d * A.G;
            if (A.window > 0 && W.ctx + d >= A.n_sink && A.window < len - d)
              hi = (d + A.window) * A.G;
            if (!(path >> off & 1)) hi = 0;
            to = A.score_tree + lbg * A.N + off;
          }
          const bool add = to && (!tree || r0 > 0);
          const float before = add ? *to : 0.f;
          lo -= r0, hi -= r0;
          wait(&s_bar[wg], used & 1);
          ++used;
          ptx::tc_fence_after();
          const bool all = __all_sync(0xffffffffu, !to || (lo <= 0 && hi >= in));
          float sum[4] = {0.f, 0.f, 0.f, 0.f};
          // 32 columns at a time, the next ones on their way meanwhile.  The lse
          // is taken off before the change of base: the difference is small where
          // a weight is not, and so is its rounding.
          constexpr float kLog2e = 1.4426950408889634f;
          auto weigh = [&](const float(&s)[32], int c) {
            float p[32];
#pragma unroll
            for (int e = 0; e < 32; e += 4) {
              const float4 z = *reinterpret_cast<const float4 *>(lse_of + c + e);
              p[e] = ptx::ex2(fmaf(s[e], A.scale, -z.x) * kLog2e);
              p[e + 1] = ptx::ex2(fmaf(s[e + 1], A.scale, -z.y) * kLog2e);
              p[e + 2] = ptx::ex2(fmaf(s[e + 2], A.scale, -z.z) * kLog2e);
              p[e + 3] = ptx::ex2(fmaf(s[e + 3], A.scale, -z.w) * kLog2e);
            }
            if (!all) {
#pragma unroll
              for (int e = 0; e < 32; ++e)
                if (c + e < lo || c + e >= hi) p[e] = 0.f;
            }
#pragma unroll
            for (int e = 0; e < 32; ++e) sum[e & 3] += p[e];
          };
          float s0[32], s1[32];
          ptx::tmem_ld32(tq, s0);
          const int acc = accumulators(nr);
          if (acc > 1) {
#pragma unroll 1
            for (int c = 0; c < nr; c += 32) {
              ptx::tmem_ld32(tq + 256 / acc + c, s1);
              ptx::tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < 32; ++e) s1[e] += s0[e];
#pragma unroll 1
              for (int k = 2; k < acc; ++k) {
                ptx::tmem_ld32(tq + k * (256 / acc) + c, s0);
                ptx::tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 32; ++e) s1[e] += s0[e];
              }
              if (c + 32 < nr) ptx::tmem_ld32(tq + c + 32, s0);
              weigh(s1, c);
            }
          } else {
#pragma unroll 1
            for (int c = 0; c < nr; c += 64) {
              ptx::tmem_wait_ld();
              if (c + 32 < nr) ptx::tmem_ld32(tq + c + 32, s1);
              weigh(s0, c);
              if (c + 32 < nr) {
                ptx::tmem_wait_ld();
                if (c + 64 < nr) ptx::tmem_ld32(tq + c + 64, s0);
                weigh(s1, c + 32);
              }
            }
          }
          ptx::tc_fence_before();
          __syncwarp();
          if (lane == 0) ptx::mbar_arrive(&free_bar[wg]);
          if (to && !bad) *to = before + ((sum[0] + sum[1]) + (sum[2] + sum[3]));
        }
      }
      ptx::named_sync(5, 256);  // nodes and lse are read
    }
    go_ahead();
    if (bad) misc[1] = 1;
  }

  ptx::tc_fence_before();
  __syncthreads();
  if (tid == 0 && misc[1] && A.status) *A.status = LBX_ETIMEOUT;
  if (warp == 8) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, 512);
  }
}

template <int DH>
cudaError_t launch_mass(bool f16, const AttnMaps &maps, const MassArgs &A, int grid, int bytes,
                        cudaStream_t stream) {
  auto kernel = f16 ? mass_kernel<DH, true> : mass_kernel<DH, false>;
  // (the same limit for all calls: another host thread may set it before this launch)
  const cudaError_t e =
      cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMostBytes);
  if (e != cudaSuccess) return e;
  kernel<<<(unsigned)grid, kThreads, (size_t)bytes, stream>>>(maps, A);
  return cudaGetLastError();
}

}  // namespace
}  // namespace cache
}  // namespace lbx

extern "C" int lbx_attention_mass(const lbx_attn_cfg *c, const int32_t *ctx_len,
                                  const int32_t *parent, const int32_t *accepted,
                                  const uint16_t *q, const float *lse, const uint16_t *k_cache,
                                  const uint16_t *k_tree, float *score, float *score_tree,
                                  int32_t *d_status, cudaStream_t stream) {
  using namespace lbx::cache;
  if (!cfg_ok(c)) return LBX_EINVAL;
  if (!aligned_to(ctx_len, 4) || !aligned_to(parent, 4) || !aligned_to(accepted, 4) ||
      !aligned_to(q, 16) || !aligned_to(lse, 4) || !aligned_to(k_tree, 16) ||
      !aligned_to(score_tree, 4) || (d_status && !aligned_to(d_status, 4)))
    return LBX_EINVAL;
  if (c->T > 0 && (!aligned_to(k_cache, 16) || !aligned_to(score, 4))) return LBX_EINVAL;
  const int lists = c->L * c->Bq, G = c->Hq / c->Hkv;
  // 32-bit indexes of the block list, and of rows (see PerGroup)
  if ((long long)c->N * G >= (1LL << 32) / G) return LBX_EINVAL;
  if ((long long)lists * c->Hkv >= (1LL << 31) / (c->T / kUnit + 6)) return LBX_EINVAL;
  const int grid = grid_limit();
  if (grid < 1) return LBX_ECUDA;
  AttnMaps maps = {};
  if (!encode_list(&maps.kt, k_tree, c, c->N, lists, kUnit)) return LBX_ECUDA;
  maps.k = maps.kt;  // without a cache: never read
  if (c->T > 0 && !encode_list(&maps.k, k_cache, c, c->T, lists, kUnit)) return LBX_ECUDA;
  MassArgs A = {};
  A.L = c->L, A.Hq = c->Hq, A.Hkv = c->Hkv, A.G = G, A.n_req = c->Bq;
  A.Bq = c->Bq, A.N = c->N, A.T = c->T, A.window = c->window, A.n_sink = c->n_sink;
  A.scale = c->scale;
  A.per = per_group(G);
  A.til = {c->N * G, 1, 1, 1, 1, kRows};
  A.ctx_len = ctx_len, A.parent = parent, A.accepted = accepted, A.q = q, A.lse = lse;
  A.score = score, A.score_tree = score_tree, A.status = d_status;
  // 64 KB of Q rows at most; the ring takes what they leave
  const int most = c->dh == 256 ? 128 : kMaxRows;
  A.cap = c->N * G < most ? (c->N * G + 31) & ~31 : most;
  const int q_bytes = A.cap * c->dh * 2;
  A.stages = (kMostBytes - kTail - q_bytes) / kPiece;
  if (A.stages > kMaxStages) A.stages = kMaxStages;
  const int bytes = q_bytes + A.stages * kPiece + kTail;
  const bool f16 = c->dtype == LBX_F16;
  const cudaError_t e = c->dh == 64    ? launch_mass<64>(f16, maps, A, grid, bytes, stream)
                        : c->dh == 128 ? launch_mass<128>(f16, maps, A, grid, bytes, stream)
                                       : launch_mass<256>(f16, maps, A, grid, bytes, stream);
  return e == cudaSuccess ? LBX_OK : LBX_ECUDA;
}
