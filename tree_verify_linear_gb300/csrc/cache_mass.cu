// cache_mass.cu -- attention weights per key, gathered over the queries of the
// accepted path: lbx_attention_mass.
#include "cache_common.cuh"

namespace lbx {
namespace cache {
namespace {

struct Args {
  lbx_attn_cfg c;
  const int32_t *ctx_len, *parent, *accepted;
  const uint16_t *q, *kc, *kt;
  const float *lse;
  float *score, *score_tree;
  int32_t *status;
};

constexpr int kWarps = 8;

// One warp per key of a (layer, request, KV head): every query row of the
// accepted path in turn.
__global__ void __launch_bounds__(kWarps * 32) mass_keys_kernel(const Args A) {
  const lbx_attn_cfg &c = A.c;
  if (batch_bad(c.Bq, c.N, c.T, A.ctx_len, A.parent, A.accepted)) {
    if (threadIdx.x == 0 && A.status) *A.status = LBX_ETREE;
    return;
  }
  const long long item = (long long)blockIdx.x * kWarps + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31, keys = c.T + c.N;
  const long long lbg = item / keys;
  if (lbg >= (long long)c.L * c.Bq * c.Hkv) return;
  const int j = (int)(item % keys), g = (int)(lbg % c.Hkv), G = c.Hq / c.Hkv, per = c.dh / 32;
  const long long lb = lbg / c.Hkv;
  const int b = (int)(lb % c.Bq), ctx = A.ctx_len[b];
  const int32_t *parent = A.parent + (size_t)b * c.N;
  const uint64_t path = path_mask(parent, A.accepted[b]);
  const int node = j - c.T;
  if (node < 0 && j >= ctx) return;
  if (node >= 0 && !(path >> node & 1)) {
    if (lane == 0) A.score_tree[lbg * c.N + node] = 0.f;
    return;
  }
  const int at_k = node < 0 ? j : ctx + __popcll(path & ((2ull << node) - 1)) - 1;
  const uint16_t *k = node < 0 ? A.kc + (((size_t)lb * c.T + j) * c.Hkv + g) * c.dh
                               : A.kt + (((size_t)lb * c.N + node) * c.Hkv + g) * c.dh;
  float kf[8], sum = 0.f;
  for (int e = 0; e < per; ++e) kf[e] = to_f32(k[lane * per + e], c.dtype);
  int at = ctx - 1;
  for (int n = 0; n < c.N; ++n) {
    if (!(path >> n & 1)) continue;
    ++at;
    if (at < at_k || !sees(at, at_k, c.window, c.n_sink)) continue;
    for (int h = 0; h < G; ++h) {
      const size_t row = ((size_t)lb * c.N + n) * c.Hq + g * G + h;
      float s = 0.f;
      for (int e = 0; e < per; ++e)
        s = fmaf(to_f32(A.q[row * c.dh + lane * per + e], c.dtype), kf[e], s);
      for (int w = 16; w; w >>= 1) s += __shfl_xor_sync(0xffffffffu, s, w);
      // a query with no finite score (lse = -inf) has no weights to give
      if (A.lse[row] != -INFINITY) sum += expf(s * c.scale - A.lse[row]);
    }
  }
  if (lane == 0) {
    if (node < 0)
      A.score[lbg * c.T + j] += sum;
    else
      A.score_tree[lbg * c.N + node] = sum;
  }
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
  const Args A = {*c,      ctx_len, parent, accepted,   q,       k_cache,
                  k_tree,  lse,     score,  score_tree, d_status};
  const long long items = (long long)c->L * c->Bq * c->Hkv * (c->T + c->N);
  const long long blocks = (items + kWarps - 1) / kWarps;
  if (blocks > 0x7fffffffLL) return LBX_EINVAL;
  mass_keys_kernel<<<(unsigned)blocks, kWarps * 32, 0, stream>>>(A);
  return cudaGetLastError() == cudaSuccess ? LBX_OK : LBX_ECUDA;
}
