// cache_evict.cu -- append the accepted path to the cache and keep the best
// `budget` entries per (layer, request, KV head): lbx_cache_evict.
//
// One CTA per (layer, request, KV head), or a cluster of CTAs that all make the
// same selection and share the moves.  The candidates' scores become 32-bit
// keys of the same order (protected entries above all, NaN below all).  A
// radix selection finds the key of the last entry that stays, eight bits at a
// time: a histogram of the digit among the keys that share the digits found
// so far, then the digit in which the count from the top passes the number
// that stays.  One bit per candidate says whether it stays (equal keys: the
// lowest indexes), with running counts per 64 of them, from which the r-th
// entry to move and the r-th free place follow by a binary search.  Entries
// that move come from at or past min(ctx, size) and go below size into places
// that nothing is read from, so that all rows move at once, in place; only the
// selection has to be done everywhere before the first move.
//
// Measured: 160 lists of 10001 to 16384 entries cut to 2048 (dimension 256): 158 us with
// the copies that put scores and positions back, 4.9 TB/s while rows of 512 bytes
// move, 15 us for the selection; a full cache of 4096 that takes six entries, 64
// lists: 14.3 us, the latency of the selection's passes.
#include <initializer_list>

#include "cache_common.cuh"
#include "cache_ptx.cuh"
#include "cache_walk.cuh"

namespace lbx {
namespace cache {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kBatch = 512;  // rows whose source and place are listed at a time
// keys are kept in shared memory when this many bytes hold them (two CTAs per
// SM, three at 16384 entries), else made again from the scores and positions in each pass
constexpr size_t kKeyBytes = 96 * 1024;
constexpr int kFly = 8;  // 16-byte pieces of rows in flight per thread

// Bytes of the bits and counts of n candidates.
constexpr size_t bit_bytes(size_t n) { return ((n + 63) / 64 * 12 + 15) & ~(size_t)15; }
// The most shared memory a call asks for.
constexpr size_t kMostBytes = bit_bytes((size_t)LBX_EVICT_MAX_T + kMaxNodes);
static_assert(kMostBytes >= kKeyBytes && kMostBytes <= 220 * 1024, "shared memory");

struct Args {
  lbx_attn_cfg c;
  int budget, n_recent, keep_keys, share;  // share: CTAs per selection
  const int32_t *ctx_len, *seen, *parent, *accepted;
  const uint16_t *kt, *vt;
  const float *score_tree;
  uint16_t *kc, *vc;
  float *score;
  int32_t *pos, *ctx_out, *seen_out, *status;
};

// Keys in the order of the scores: NaN, -inf, .., -0 = 0, .., inf.
__device__ __forceinline__ uint32_t key_of(float f) {
  if (f != f) return 0u;
  const uint32_t u = __float_as_uint(f + 0.f);  // -0 + 0 = 0
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}
constexpr uint32_t kSafe = 0xffffffffu;

// Position of the set bit number r (from 0) of w.
__device__ __forceinline__ int nth_bit(uint64_t w, int r) {
  const int c = __popc((uint32_t)w);
  uint32_t h = r < c ? (uint32_t)w : (uint32_t)(w >> 32);
  for (int i = r < c ? 0 : c; i < r; ++i) h &= h - 1;
  return __ffs(h) - 1 + (r < c ? 0 : 32);
}
// The low k (0..63) bits.
__device__ __forceinline__ uint64_t below(int k) { return (1ull << k) - 1; }

__global__ void __launch_bounds__(kThreads) evict_kernel(const Args A) {
  extern __shared__ __align__(16) unsigned char smem[];
  __shared__ uint32_t hist[256], warp_sum[kWarps + 1], found[2];
  __shared__ int src[kBatch], dst[kBatch], node_at[kMaxNodes];
  const lbx_attn_cfg &c = A.c;
  if (batch_bad(c.Bq, c.N, c.T, A.ctx_len, A.parent, A.accepted)) {
    if (threadIdx.x == 0 && A.status) *A.status = LBX_ETREE;
    return;
  }
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = A.share > 1 ? (int)ptx::cluster_rank() : 0;
  const long long lbg = blockIdx.x / A.share;
  const int g = (int)(lbg % c.Hkv);
  const long long lb = lbg / c.Hkv;
  const int b = (int)(lb % c.Bq);
  const int ctx = A.ctx_len[b], seen = A.seen[b];
  const uint64_t path = warp_path(A.parent + (size_t)b * c.N, c.N, A.accepted[b], lane);
  const int n = ctx + __popcll(path), size = n < A.budget ? n : A.budget;
  const int low = ctx < size ? ctx : size;  // entries below do not move
  const int seen_out = seen + n - ctx, recent = seen_out - A.n_recent;
  if (tid < c.N && (path >> tid & 1)) node_at[__popcll(path & ((1ull << tid) - 1))] = tid;
  if (tid == 0 && rank == 0 && lb == b && g == 0) A.ctx_out[b] = size, A.seen_out[b] = seen_out;

  float *score = A.score + lbg * c.T;
  int32_t *pos = A.pos + lbg * c.T;
  const float *score_tree = A.score_tree + lbg * c.N;
  const int words = (n + 63) / 64, cap_words = (c.T + c.N + 63) / 64;
  uint64_t *stay = reinterpret_cast<uint64_t *>(smem);  // one bit per candidate
  uint32_t *before = reinterpret_cast<uint32_t *>(stay + cap_words);  // set in earlier words
  // only with keep_keys
  uint32_t *keys = reinterpret_cast<uint32_t *>(smem + ((cap_words * 12 + 15) & ~15));
  __syncthreads();

  auto rank_of = [&](int p, float s) {
    return p < c.n_sink || p >= recent ? kSafe : key_of(s);
  };
  auto make_key = [&](int i) -> uint32_t {
    return i < ctx ? rank_of(pos[i], score[i])
                   : rank_of(seen + (i - ctx), score_tree[node_at[i - ctx]]);
  };
  auto key = [&](int i) -> uint32_t { return A.keep_keys ? keys[i] : make_key(i); };

  // ---- the key of the last entry that stays, and how many equal ones do ----
  uint32_t last = 0, equal = 0;
  if (n > size) {
    if (A.keep_keys) {
      // four entries at a time where the rows are aligned, then the rest
      const bool wide = ((reinterpret_cast<uintptr_t>(score) | reinterpret_cast<uintptr_t>(pos)) &
                         15) == 0;
      const int quads = wide ? ctx / 4 : 0;
#pragma unroll 4
      for (int i = tid; i < quads; i += kThreads) {
        const int4 p = reinterpret_cast<const int4 *>(pos)[i];
        const float4 s = reinterpret_cast<const float4 *>(score)[i];
        reinterpret_cast<uint4 *>(keys)[i] = make_uint4(rank_of(p.x, s.x), rank_of(p.y, s.y),
                                                        rank_of(p.z, s.z), rank_of(p.w, s.w));
      }
#pragma unroll 2
      for (int i = quads * 4 + tid; i < n; i += kThreads) keys[i] = make_key(i);
    }
    uint32_t want = (uint32_t)size;  // how many of the keys that match so far stay
    for (int shift = 24; shift >= 0; shift -= 8) {
      if (tid < 256) hist[tid] = 0;
      __syncthreads();
      for (int i = tid; i < n; i += kThreads) {
        const uint32_t k = key(i);
        if (shift == 24 || (k >> (shift + 8)) == (last >> (shift + 8)))
          atomicAdd(&hist[(k >> shift) & 255], 1u);
      }
      __syncthreads();
      if (warp == 0) {  // lane holds digits 255 - 8 lane .. 248 - 8 lane
        uint32_t h[8], sum = 0;
        for (int e = 0; e < 8; ++e) sum += h[e] = hist[255 - 8 * lane - e];
        uint32_t upto = sum;
        for (int w = 1; w < 32; w <<= 1) {
          const uint32_t x = __shfl_up_sync(0xffffffffu, upto, w);
          if (lane >= w) upto += x;
        }
        uint32_t above = upto - sum;
        if (above < want && upto >= want)
          for (int e = 0; e < 8; ++e) {
            if (above + h[e] >= want) {
              found[0] = 255 - 8 * lane - e;
              found[1] = want - above;
              break;
            }
            above += h[e];
          }
      }
      __syncthreads();
      last |= found[0] << shift;
      want = found[1];
    }
    equal = want;
  }

  // ---- one bit per candidate; each warp takes consecutive words ----
  const int per = (words + kWarps - 1) / kWarps;
  const int w0 = warp * per, w1 = w0 + per < words ? w0 + per : words;
  uint32_t mine = 0;
  if (n > size) {
    for (int i = w0 * 64 + lane; i < w1 * 64 + lane; i += 32)
      mine += __popc(__ballot_sync(0xffffffffu, i < n && key(i) == last));
  }
  // running sum of `mine` over the warps
  auto scan = [&]() -> uint32_t {
    __syncthreads();
    if (lane == 0) warp_sum[warp] = mine;
    __syncthreads();
    uint32_t s = 0;
    for (int w = 0; w < warp; ++w) s += warp_sum[w];
    return s;
  };
  uint32_t ties = scan();
  mine = 0;
  for (int w = w0; w < w1; ++w) {
    uint64_t bits = 0;
    for (int half = 0; half < 2; ++half) {
      const int i = w * 64 + half * 32 + lane;
      bool in = i < n;
      if (n > size) {
        const uint32_t k = in ? key(i) : 0u;
        const uint32_t eq = __ballot_sync(0xffffffffu, in && k == last);
        in = in && (k > last || (k == last && ties + __popc(eq & ((1u << lane) - 1)) < equal));
        ties += __popc(eq);
      }
      bits |= (uint64_t)__ballot_sync(0xffffffffu, in) << (half * 32);
    }
    if (lane == 0) stay[w] = bits, before[w] = mine;
    mine += __popcll(bits);
  }
  const uint32_t base = scan();
  for (int w = w0 + lane; w < w1; w += 32) before[w] += base;
  __syncthreads();

  // candidates below `low` that stay
  const uint32_t stay_low =
      (low >> 6) >= words ? (uint32_t)size
                          : before[low >> 6] + __popcll(stay[low >> 6] & below(low & 63));
  const int moves = size - (int)stay_low;

  if (A.share > 1) ptx::cluster_sync();  // every score and position is read

  // ---- move: batches of listed rows ----
  const int shift = c.dh == 256 ? 6 : c.dh == 128 ? 5 : 4;  // 16-byte pieces of K and V: 2^shift
  for (int m0 = rank * kBatch; m0 < moves; m0 += A.share * kBatch) {
    const int cnt = moves - m0 < kBatch ? moves - m0 : kBatch;
    for (int t = tid; t < cnt; t += kThreads) {
      const uint32_t rs = stay_low + (uint32_t)(m0 + t);  // number among those that stay
      int a = 0, z = words - 1;
      while (a < z) {  // last word with before <= rs
        const int h = (a + z + 1) >> 1;
        if (before[h] <= rs) a = h;
        else z = h - 1;
      }
      src[t] = a * 64 + nth_bit(stay[a], (int)(rs - before[a]));
      const uint32_t rf = (uint32_t)(m0 + t);  // number among the free places
      auto free_before = [&](int w) -> uint32_t {
        return (uint32_t)(w * 64) - (before[w] < stay_low ? before[w] : stay_low);
      };
      a = 0, z = (size - 1) >> 6;
      while (a < z) {
        const int h = (a + z + 1) >> 1;
        if (free_before(h) <= rf) a = h;
        else z = h - 1;
      }
      uint64_t held = stay[a];  // staying below `low` only
      if (low < a * 64 + 64) held &= low > a * 64 ? below(low - a * 64) : 0ull;
      dst[t] = a * 64 + nth_bit(~held, (int)(rf - free_before(a)));
    }
    __syncthreads();
    for (int t = tid; t < cnt; t += kThreads) {
      const int s = src[t], d = dst[t];
      score[d] = s < ctx ? score[s] : score_tree[node_at[s - ctx]];
      pos[d] = s < ctx ? pos[s] : seen + (s - ctx);
    }
    for (int u0 = tid; u0 < cnt << shift; u0 += kFly * kThreads) {
      uint4 piece[kFly];
      // piece u of the batch: half of a row's are K's, half V's
      auto place = [&](int u, bool from) -> uint4 * {
        const int e = u & ((1 << shift) - 1), half = 1 << (shift - 1), t = u >> shift;
        const int s = src[t], i = from ? s : dst[t];
        const bool is_v = e >= half, old = !from || s < ctx;
        const uint16_t *base = old ? (is_v ? A.vc : A.kc) : (is_v ? A.vt : A.kt);
        const size_t row = old ? (size_t)lb * c.T + i : (size_t)lb * c.N + node_at[s - ctx];
        return reinterpret_cast<uint4 *>(const_cast<uint16_t *>(base)) +
               (row * c.Hkv + g) * half + (e & (half - 1));
      };
#pragma unroll
      for (int k = 0; k < kFly; ++k) {
        const int u = u0 + k * kThreads;
        if (u < cnt << shift) piece[k] = __ldcs(place(u, true));
      }
#pragma unroll
      for (int k = 0; k < kFly; ++k) {
        const int u = u0 + k * kThreads;
        if (u < cnt << shift) *place(u, false) = piece[k];
      }
    }
    __syncthreads();
  }
}

}  // namespace
}  // namespace cache
}  // namespace lbx

extern "C" int lbx_cache_evict(const lbx_attn_cfg *c, int budget, int n_recent,
                               const int32_t *ctx_len, const int32_t *seen, const int32_t *parent,
                               const int32_t *accepted, const uint16_t *k_tree,
                               const uint16_t *v_tree, const float *score_tree, uint16_t *k_cache,
                               uint16_t *v_cache, float *score, int32_t *pos, int32_t *ctx_out,
                               int32_t *seen_out, int32_t *d_status, cudaStream_t stream) {
  using namespace lbx::cache;
  if (!cfg_ok(c) || budget < 1 || budget > c->T || c->T > LBX_EVICT_MAX_T || n_recent < 0)
    return LBX_EINVAL;
  if (!aligned_to(ctx_len, 4) || !aligned_to(seen, 4) || !aligned_to(parent, 4) ||
      !aligned_to(accepted, 4) || !aligned_to(k_tree, 16) || !aligned_to(v_tree, 16) ||
      !aligned_to(score_tree, 4) || !aligned_to(k_cache, 16) || !aligned_to(v_cache, 16) ||
      !aligned_to(score, 4) || !aligned_to(pos, 4) || !aligned_to(ctx_out, 4) ||
      !aligned_to(seen_out, 4) || (d_status && !aligned_to(d_status, 4)))
    return LBX_EINVAL;
  // CTAs read the inputs while one writes the outputs
  const size_t per = (size_t)c->Bq * 4;
  auto apart = [](const void *a, size_t na, const void *b, size_t nb) {
    const uintptr_t x = (uintptr_t)a, y = (uintptr_t)b;
    return x + na <= y || y + nb <= x;
  };
  for (const void *out : {ctx_out, seen_out})
    if (!apart(out, per, ctx_len, per) || !apart(out, per, seen, per) ||
        !apart(out, per, accepted, per) || !apart(out, per, parent, per * c->N))
      return LBX_EINVAL;
  if (!apart(ctx_out, per, seen_out, per)) return LBX_EINVAL;
  const size_t n = (size_t)c->T + c->N, bits = bit_bytes(n);
  const int keep_keys = n * 4 + bits <= kKeyBytes;
  const size_t shared = bits + (keep_keys ? n * 4 : 0);
  // the limit is the function's, not the call's: the same for all, since another host
  // thread may set it between this and the launch
  if (cudaFuncSetAttribute(evict_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           (int)kMostBytes) != cudaSuccess)
    return LBX_ECUDA;
  // A cache larger than its budget may have many rows to move: CTAs share each
  // selection as long as all of them run at once (two waves of clusters would
  // take twice the time).  A full cache moves a few rows per step, and one does.
  const long long lists = (long long)c->L * c->Bq * c->Hkv;
  int share = 1, per_sm = 1;
  if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, evict_kernel, kThreads, shared) !=
      cudaSuccess)
    return LBX_ECUDA;
  if (c->T > budget + c->N)
    while (share < 8 && lists * share * 2 <= (long long)per_sm * grid_limit()) share *= 2;
  const Args A = {*c,     budget, n_recent,   keep_keys, share,   ctx_len, seen, parent,  accepted,
                  k_tree, v_tree, score_tree, k_cache,   v_cache, score,   pos,  ctx_out, seen_out,
                  d_status};
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(lists * share)), cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = shared, cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = (unsigned)share, at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at, cfg.numAttrs = share > 1 ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, evict_kernel, A) == cudaSuccess ? LBX_OK : LBX_ECUDA;
}
