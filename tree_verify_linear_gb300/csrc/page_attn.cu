// page_attn.cu -- attention of each request's new tokens over its pages:
// lbx_paged_attention.
//
// The simplest form: a warp per (row, query head), the head's dimensions over its
// lanes, one key after another with the running maximum and sum of the softmax.
#include "page_common.cuh"

namespace lbx {
namespace paged {
namespace {

constexpr int kThreads = 256;

struct PlainArgs {
  lbx_page_cfg c;
  int shift;
  const int32_t *start, *ctx_len, *table, *parent;
  const uint16_t *q, *k, *v;
  uint16_t *o;
  float *lse;
  int32_t *status;
};

template <bool F16>
__device__ __forceinline__ float value(uint16_t u) {
  if constexpr (F16) return __half2float(__ushort_as_half(u));
  else return __uint_as_float((uint32_t)u << 16);
}

template <int DH, bool F16>
__global__ void __launch_bounds__(kThreads) plain_kernel(const PlainArgs A) {
  const lbx_page_cfg &c = A.c;
  if (batch_bad(c, A.start, A.ctx_len, A.parent, nullptr)) {
    if (threadIdx.x == 0 && A.status) *A.status = LBX_ETREE;
    return;
  }
  const int lane = threadIdx.x & 31, rows = A.start[c.Bq];
  const long long n = (long long)c.L * rows * c.Hq, warps = (long long)gridDim.x * (kThreads / 32);
#pragma unroll 1
  for (long long w = (long long)blockIdx.x * (kThreads / 32) + threadIdx.x / 32; w < n; w += warps) {
    const int h = (int)(w % c.Hq), r = (int)(w / c.Hq % rows), l = (int)(w / c.Hq / rows);
    int a = 0, z = c.Bq - 1;  // the last request that starts at r or before
    while (a < z) {
      const int m = (a + z + 1) >> 1;
      if (A.start[m] <= r) a = m;
      else z = m - 1;
    }
    const int s = A.start[a], i = r - s, ctx = A.ctx_len[a];
    const int end = A.parent ? ctx + i + 1 : ctx + i + 1;
    const uint64_t path =
        A.parent ? cache::warp_path(A.parent + s, A.start[a + 1] - s, i, lane) : ~0ull;
    const size_t at = ((size_t)l * c.M + r) * c.Hq + h;
    constexpr int kE = DH / 32;
    float q[kE], acc[kE], m = -INFINITY, sum = 0.f;
#pragma unroll
    for (int e = 0; e < kE; ++e) q[e] = value<F16>(A.q[at * DH + lane + 32 * e]), acc[e] = 0.f;
#pragma unroll 1
    for (int p = 0; p < end; ++p) {
      if (A.parent && p >= ctx && !(path >> (p - ctx) & 1)) continue;
      const int id = A.table[(size_t)a * c.max_pages + (p >> A.shift)];
      if (id < 0 || id >= c.n_pages) {
        if (A.status) *A.status = LBX_EINVAL;
        break;
      }
      const size_t row = (((size_t)l * c.n_pages + id) * c.page + (p & (c.page - 1))) * c.Hkv +
                         h / (c.Hq / c.Hkv);
      float x = 0.f;
#pragma unroll
      for (int e = 0; e < kE; ++e) x = fmaf(q[e], value<F16>(A.k[row * DH + lane + 32 * e]), x);
#pragma unroll
      for (int d = 16; d; d >>= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
      x *= c.scale;
      const float top = x > m ? x : m;  // (a NaN stays out of it and reaches the sum)
      const float ref = top == -INFINITY ? 0.f : top;
      const float alpha = expf(m - ref), weight = expf(x - ref);
      m = top;
      sum = fmaf(sum, alpha, weight);
#pragma unroll
      for (int e = 0; e < kE; ++e)
        acc[e] = fmaf(acc[e], alpha, weight * value<F16>(A.v[row * DH + lane + 32 * e]));
    }
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
    for (int e = 0; e < kE; ++e) {
      const float y = sum == 0.f ? 0.f : acc[e] * inv;
      uint16_t u;
      if constexpr (F16) u = __half_as_ushort(__float2half_rn(y));
      else u = __bfloat16_as_ushort(__float2bfloat16_rn(y));
      A.o[at * DH + lane + 32 * e] = u;
    }
    if (lane == 0 && A.lse) A.lse[at] = sum == 0.f ? -INFINITY : m + logf(sum);
  }
}

template <int DH>
void launch(bool f16, const PlainArgs &A, cudaStream_t stream) {
  if (f16) plain_kernel<DH, true><<<152 * 8, kThreads, 0, stream>>>(A);
  else plain_kernel<DH, false><<<152 * 8, kThreads, 0, stream>>>(A);
}

}  // namespace
}  // namespace paged
}  // namespace lbx

extern "C" size_t lbx_paged_workspace_size(const lbx_page_cfg *c) {
  using namespace lbx::paged;
  if (!cfg_ok(c) || c->Hq / c->Hkv > LBX_PAGED_MAX_GROUP) return 0;
  return 256;
}

extern "C" int lbx_paged_attention(const lbx_page_cfg *c, const int32_t *start,
                                   const int32_t *ctx_len, const int32_t *block_table,
                                   const int32_t *parent, const uint16_t *q,
                                   const uint16_t *k_pages, const uint16_t *v_pages, uint16_t *o,
                                   float *lse, void *workspace, size_t workspace_bytes,
                                   int32_t *d_status, cudaStream_t stream) {
  using namespace lbx::paged;
  const size_t need = lbx_paged_workspace_size(c);
  if (need == 0 || workspace_bytes < need) return LBX_EINVAL;
  for (const int32_t *p : {start, ctx_len, block_table})
    if (!aligned_to(p, 4)) return LBX_EINVAL;
  for (const uint16_t *p : {q, k_pages, v_pages, (const uint16_t *)o})
    if (!aligned_to(p, 16)) return LBX_EINVAL;
  if ((parent && !aligned_to(parent, 4)) || (lse && !aligned_to(lse, 4)) ||
      !aligned_to(workspace, 16) || (d_status && !aligned_to(d_status, 4)))
    return LBX_EINVAL;
  PlainArgs A = {*c, 0, start, ctx_len, block_table, parent, q, k_pages, v_pages, o, lse, d_status};
  while (1 << A.shift < c->page) ++A.shift;
  const bool f16 = c->dtype == LBX_F16;
  if (c->dh == 64) launch<64>(f16, A, stream);
  else if (c->dh == 128) launch<128>(f16, A, stream);
  else launch<256>(f16, A, stream);
  return cudaGetLastError() == cudaSuccess ? LBX_OK : LBX_ECUDA;
}
