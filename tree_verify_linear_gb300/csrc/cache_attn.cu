// cache_attn.cu -- attention over a bounded or shared KV cache:
// lbx_window_attention and lbx_prefix_attention (host side; the kernel is in
// cache_attn.cuh).
//
// The window call is one launch over the requests' key lists.  The prefix call
// is two: the requests' own keys, whose normalised results and base-2 lse go to
// the workspace in fp32, then the queries of all requests over the prefix, whose
// last step joins the two by their lse.  (In this order because the second's
// streams are the fewer and longer ones, and a stream's end costs 9 us with the
// joining and 3 us without: five requests of 22 nodes over 4096 shared keys take
// 311 us; the other way round cost 14 us more.)  The second launch begins on the SMs that
// the first one's CTAs leave and waits for its results only there.
#include <cudaTypedefs.h>

#include <cstring>
#include <mutex>

#include "cache_attn.cuh"

namespace lbx {
namespace cache {
namespace {

PFN_cuTensorMapEncodeTiled_v12000 g_encode = nullptr;
std::once_flag g_encode_once;

bool have_encode() {
  std::call_once(g_encode_once, [] {
    void *fn = nullptr;
    cudaDriverEntryPointQueryResult qr;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault,
                                         &qr) == cudaSuccess &&
        qr == cudaDriverEntryPointSuccess)
      g_encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
  });
  return g_encode != nullptr;
}

}  // namespace

// Queries as (dh, Hq, nodes, lists); box: 64 columns of a KV head's G heads of as
// many nodes as fit 128 rows.
static bool encode_queries(CUtensorMap *map, const void *base, const lbx_attn_cfg *c, int nodes,
                           int lists) {
  if (!have_encode()) return false;
  const int G = c->Hq / c->Hkv;
  const cuuint64_t row = (cuuint64_t)c->Hq * c->dh * 2;
  const cuuint64_t gdim[4] = {(cuuint64_t)c->dh, (cuuint64_t)c->Hq, (cuuint64_t)nodes,
                              (cuuint64_t)lists};
  const cuuint64_t gstride[3] = {(cuuint64_t)c->dh * 2, row, row * (cuuint64_t)nodes};
  const cuuint32_t box[4] = {64, (cuuint32_t)G, (cuuint32_t)(kRows / G), 1};
  const cuuint32_t estride[4] = {1, 1, 1, 1};
  return g_encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT16, 4, const_cast<void *>(base), gdim, gstride,
                  box, estride, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool encode_list(CUtensorMap *map, const void *base, const lbx_attn_cfg *c, int len, int lists,
                 int keys) {
  if (!have_encode()) return false;
  const cuuint64_t row = (cuuint64_t)c->Hkv * c->dh * 2;
  const cuuint64_t gdim[4] = {(cuuint64_t)c->dh, (cuuint64_t)c->Hkv, (cuuint64_t)len,
                              (cuuint64_t)lists};
  const cuuint64_t gstride[3] = {(cuuint64_t)c->dh * 2, row, row * (cuuint64_t)len};
  const cuuint32_t box[4] = {64, 1, (cuuint32_t)keys, 1};
  const cuuint32_t estride[4] = {1, 1, 1, 1};
  return g_encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT16, 4, const_cast<void *>(base), gdim, gstride,
                  box, estride, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

int grid_limit() {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n < 1)
    return 0;
  return n < kMaxCtas ? n : kMaxCtas;
}

namespace {

size_t up256(size_t n) { return (n + 255) & ~(size_t)255; }

// The workspace: counters, at the same places whatever the configuration, so that
// calls of any kind may take turns on one; then the partials of the requests' launch;
// with a prefix also the prefix launch's, and the first launch's results and lse.
constexpr size_t kCounterBytes = 4 * kFewUnits;
constexpr int kPrefixCounters = 2 * kMaxCtas;  // the first of the prefix launch's
static_assert(2 * kPrefixCounters <= kFewUnits, "counters of two launches, or of the small kernel");
size_t part_bytes(const lbx_attn_cfg *c) {
  return up256((size_t)kMaxCtas * 2 * part_floats(c->dh) * 4);
}
struct Space {
  Tiling own, pre;
  size_t part, pre_part, x_o, x_lse, bytes;  // offsets, and the end
};
Space space_of(const lbx_attn_cfg *c) {
  Space s;
  const long long G = c->Hq / c->Hkv, rows = (long long)c->N * G;
  s.own = tiling(rows, (int)G, c->dh);
  s.pre = tiling(rows * c->Bq, (int)G, c->dh);
  s.part = kCounterBytes;
  s.pre_part = s.x_o = s.x_lse = s.bytes = s.part + part_bytes(c);
  if (c->P > 0) {  // the two launches overlap: nothing is shared
    const size_t queries = (size_t)c->L * c->Bq * c->N * c->Hq;
    s.x_o = s.pre_part + part_bytes(c);
    s.x_lse = s.x_o + up256(queries * c->dh * 4);
    s.bytes = s.x_lse + up256(queries * 4);
  }
  return s;
}

// The block list's indexes are 32-bit.
bool list_ok(const lbx_attn_cfg *c, const Space &s) {
  auto fits = [&](const Tiling &t, long long lists, long long len) {
    return lists * t.sets < (1LL << 31) / (len / kUnit + 3 + kLeadBlocks);
  };
  const long long lists = (long long)c->L * c->Hkv, G = c->Hq / c->Hkv;
  if ((long long)c->Bq * c->N * G >= (1LL << 32) / G) return false;  // see PerGroup
  return fits(s.own, lists * c->Bq, c->T) && fits(s.pre, lists, c->P);
}

int attention(const lbx_attn_cfg *c, const int32_t *ctx_len, const int32_t *parent,
              const uint16_t *q, const uint16_t *kp, const uint16_t *vp, const uint16_t *kc,
              const uint16_t *vc, const uint16_t *kt, const uint16_t *vt, uint16_t *o, float *lse,
              void *ws, size_t ws_bytes, int32_t *status, cudaStream_t stream) {
  if (!aligned_to(ctx_len, 4) || !aligned_to(parent, 4) || !aligned_to(q, 16) ||
      !aligned_to(kt, 16) || !aligned_to(vt, 16) || !aligned_to(o, 16) || !aligned_to(ws, 16))
    return LBX_EINVAL;
  if (c->T > 0 && (!aligned_to(kc, 16) || !aligned_to(vc, 16))) return LBX_EINVAL;
  if (c->P > 0 && (!aligned_to(kp, 16) || !aligned_to(vp, 16))) return LBX_EINVAL;
  if ((lse && !aligned_to(lse, 4)) || (status && !aligned_to(status, 4))) return LBX_EINVAL;
  const Space s = space_of(c);
  if (!list_ok(c, s) || ws_bytes < s.bytes) return LBX_EINVAL;
  unsigned char *base = static_cast<unsigned char *>(ws);
  if (const int chunks = few_chunks(c)) {
    const FewArgs F = {*c, chunks, c->scale * 1.4426950408889634f, ctx_len, parent, q, kp, vp, kc,
                       vc, kt, vt, o, lse, reinterpret_cast<float *>(base + s.part),
                       reinterpret_cast<unsigned int *>(base), status};
    return launch_few(F, stream) == cudaSuccess ? LBX_OK : LBX_ECUDA;
  }

  // rows of a box of V: a piece of it may hold fewer keys than a unit
  static_assert(Lay<128, false>::kVBox == kUnit && Lay<64, false>::kVBox == kUnit &&
                    Lay<128, true>::kVBox == kUnit && Lay<256, true>::kVBox == kUnit,
                "V boxes");
  auto v_box = [&](const Tiling &t) {
    return c->dh == 256 && t.ctas == 1 ? Lay<256, false>::kVBox : kUnit;
  };

  const int nsm = grid_limit();
  if (nsm < 1) return LBX_ECUDA;
  AttnArgs A = {};
  A.L = c->L, A.Hq = c->Hq, A.Hkv = c->Hkv, A.G = c->Hq / c->Hkv;
  A.Bq = c->Bq, A.N = c->N, A.T = c->T;
  A.scale_log2 = c->scale * 1.4426950408889634f;
  A.per = per_group(A.G);
  A.ctx_len = ctx_len, A.parent = parent, A.q = q, A.status = status;
  const bool f16 = c->dtype == LBX_F16;
  auto launch = [&](const AttnMaps &maps) {
    const int by = A.til.group * A.til.ctas;  // at most 16: fewer than SMs
    const int grid = nsm / by * by;
    const cudaError_t e = c->dh == 64    ? launch_attn<64>(f16, maps, A, grid, stream)
                          : c->dh == 128 ? launch_attn<128>(f16, maps, A, grid, stream)
                                         : launch_attn<256>(f16, maps, A, grid, stream);
    return e == cudaSuccess;
  };
  const bool prefix = c->P > 0;
  const int lists = c->L * c->Bq;
  AttnMaps maps;
  std::memset(&maps, 0, sizeof maps);
  // ---- the requests' own keys ----
  if (!encode_list(&maps.kt, kt, c, c->N, lists, kUnit) ||
      !encode_list(&maps.vt, vt, c, c->N, lists, v_box(s.own)))
    return LBX_ECUDA;
  maps.k = maps.kt, maps.v = maps.vt;  // without a cache: never read
  if (c->T > 0 && (!encode_list(&maps.k, kc, c, c->T, lists, kUnit) ||
                   !encode_list(&maps.v, vc, c, c->T, lists, v_box(s.own))))
    return LBX_ECUDA;
  if (s.own.ctas == 2 && !encode_queries(&maps.q, q, c, c->N, lists)) return LBX_ECUDA;
  A.n_req = c->Bq, A.nodes = c->N, A.til = s.own;
  A.window = c->window, A.n_sink = c->n_sink, A.join = kJoinBlocks;
  A.part = reinterpret_cast<float *>(base + s.part);
  A.counters = reinterpret_cast<unsigned int *>(base);
  if (prefix)
    A.o32 = reinterpret_cast<float *>(base + s.x_o), A.lse2 = reinterpret_cast<float *>(base + s.x_lse);
  else
    A.o = o, A.lse = lse;
  if (!launch(maps)) return LBX_ECUDA;
  if (!prefix) return LBX_OK;
  // ---- the prefix, joined with them ----
  if (!encode_list(&maps.k, kp, c, c->P, c->L, kUnit) ||
      !encode_list(&maps.v, vp, c, c->P, c->L, v_box(s.pre)))
    return LBX_ECUDA;
  maps.kt = maps.k, maps.vt = maps.v;  // a prefix has no tree: never read
  if (s.pre.ctas == 2 && !encode_queries(&maps.q, q, c, c->Bq * c->N, c->L)) return LBX_ECUDA;
  A.n_req = 1, A.nodes = c->Bq * c->N, A.fixed = c->P, A.til = s.pre, A.join = kJoinPrefixBlocks;
  A.part = reinterpret_cast<float *>(base + s.pre_part);
  A.counters += kPrefixCounters;
  A.x_o = A.o32, A.x_lse2 = A.lse2, A.o32 = nullptr, A.lse2 = nullptr;
  A.o = o, A.lse = lse;
  return launch(maps) ? LBX_OK : LBX_ECUDA;
}

}  // namespace
}  // namespace cache
}  // namespace lbx

extern "C" size_t lbx_cache_attn_workspace_size(const lbx_attn_cfg *c) {
  using namespace lbx::cache;
  if (!cfg_ok(c)) return 0;
  const Space s = space_of(c);
  return list_ok(c, s) ? s.bytes : 0;
}

extern "C" int lbx_window_attention(const lbx_attn_cfg *c, const int32_t *ctx_len,
                                    const int32_t *parent, const uint16_t *q,
                                    const uint16_t *k_cache, const uint16_t *v_cache,
                                    const uint16_t *k_tree, const uint16_t *v_tree, uint16_t *o,
                                    float *lse, void *workspace, size_t workspace_bytes,
                                    int32_t *d_status, cudaStream_t stream) {
  using namespace lbx::cache;
  if (!cfg_ok(c) || c->P != 0) return LBX_EINVAL;
  return attention(c, ctx_len, parent, q, nullptr, nullptr, k_cache, v_cache, k_tree, v_tree, o,
                   lse, workspace, workspace_bytes, d_status, stream);
}

extern "C" int lbx_prefix_attention(const lbx_attn_cfg *c, const int32_t *ctx_len,
                                    const int32_t *parent, const uint16_t *q,
                                    const uint16_t *k_prefix, const uint16_t *v_prefix,
                                    const uint16_t *k_cache, const uint16_t *v_cache,
                                    const uint16_t *k_tree, const uint16_t *v_tree, uint16_t *o,
                                    float *lse, void *workspace, size_t workspace_bytes,
                                    int32_t *d_status, cudaStream_t stream) {
  using namespace lbx::cache;
  if (!cfg_ok(c) || c->P < 1 || c->window != 0 || c->n_sink != 0) return LBX_EINVAL;
  return attention(c, ctx_len, parent, q, k_prefix, v_prefix, k_cache, v_cache, k_tree, v_tree, o,
                   lse, workspace, workspace_bytes, d_status, stream);
}
