// cache_attn.cu -- attention over a bounded or shared KV cache:
// lbx_window_attention and lbx_prefix_attention.
#include "cache_common.cuh"

namespace lbx {
namespace cache {
namespace {

struct Args {
  lbx_attn_cfg c;
  const int32_t *ctx_len, *parent;
  const uint16_t *q, *kp, *vp, *kc, *vc, *kt, *vt;
  uint16_t *o;
  float *lse;
  int32_t *status;
};

constexpr int kWarps = 8;

// One warp per query row: every visible key in turn, a running maximum and sum.
__global__ void __launch_bounds__(kWarps * 32) attn_rows_kernel(const Args A) {
  const lbx_attn_cfg &c = A.c;
  if (batch_bad(c.Bq, c.N, c.T, A.ctx_len, A.parent, nullptr)) {
    if (threadIdx.x == 0 && A.status) *A.status = LBX_ETREE;
    return;
  }
  const long long row = (long long)blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (row >= (long long)c.L * c.Bq * c.N * c.Hq) return;
  const int lane = threadIdx.x & 31;
  const int hq = (int)(row % c.Hq);
  const long long lbn = row / c.Hq;
  const int n = (int)(lbn % c.N);
  const long long lb = lbn / c.N;
  const int l = (int)(lb / c.Bq), b = (int)(lb % c.Bq);
  const int g = hq / (c.Hq / c.Hkv), per = c.dh / 32;
  float q[8], acc[8];
  for (int e = 0; e < per; ++e) {
    q[e] = to_f32(A.q[row * c.dh + lane * per + e], c.dtype) * c.scale;
    acc[e] = 0.f;
  }
  float m = -INFINITY, sum = 0.f;
  auto key = [&](const uint16_t *k, const uint16_t *v, long long at) {
    const size_t off = ((size_t)at * c.Hkv + g) * c.dh + lane * per;
    float s = 0.f;
    for (int e = 0; e < per; ++e) s = fmaf(q[e], to_f32(k[off + e], c.dtype), s);
    for (int w = 16; w; w >>= 1) s += __shfl_xor_sync(0xffffffffu, s, w);
    const float m1 = fmaxf(m, s);
    if (m1 == -INFINITY) return;
    const float old = expf(m - m1), p = expf(s - m1);
    sum = sum * old + p;
    for (int e = 0; e < per; ++e) acc[e] = acc[e] * old + p * to_f32(v[off + e], c.dtype);
    m = m1;
  };
  const uint64_t anc = path_mask(A.parent + (size_t)b * c.N, n);
  const int ctx = A.ctx_len[b], at = ctx + __popcll(anc) - 1;
  for (int j = 0; j < c.P; ++j) key(A.kp, A.vp, (long long)l * c.P + j);
  for (int j = 0; j < ctx; ++j)
    if (sees(at, j, c.window, c.n_sink)) key(A.kc, A.vc, lb * c.T + j);
  int pos = ctx;
  for (int t = 0; t < c.N; ++t)
    if (anc >> t & 1) {
      if (sees(at, pos, c.window, c.n_sink)) key(A.kt, A.vt, lb * c.N + t);
      ++pos;
    }
  for (int e = 0; e < per; ++e)
    A.o[row * c.dh + lane * per + e] = from_f32(sum > 0.f ? acc[e] / sum : 0.f, c.dtype);
  if (A.lse && lane == 0) A.lse[row] = sum > 0.f ? m + logf(sum) : -INFINITY;
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
  if (ws_bytes < lbx_cache_attn_workspace_size(c)) return LBX_EINVAL;
  const Args A = {*c, ctx_len, parent, q, kp, vp, kc, vc, kt, vt, o, lse, status};
  const long long rows = (long long)c->L * c->Bq * c->N * c->Hq;
  attn_rows_kernel<<<(unsigned)((rows + kWarps - 1) / kWarps), kWarps * 32, 0, stream>>>(A);
  return cudaGetLastError() == cudaSuccess ? LBX_OK : LBX_ECUDA;
}

}  // namespace
}  // namespace cache
}  // namespace lbx

extern "C" size_t lbx_cache_attn_workspace_size(const lbx_attn_cfg *c) {
  return lbx::cache::cfg_ok(c) ? 256 : 0;
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
