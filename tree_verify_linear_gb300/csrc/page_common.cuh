// page_common.cuh -- what the operators of the paged KV cache have in common:
// host-side checks of the configuration, the whole-batch check of the lengths
// and trees, and where a position of a request lies.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <initializer_list>

#include "cache_common.cuh"
#include "lbx.h"

namespace lbx {
namespace paged {

using cache::aligned_to;

inline bool cfg_ok(const lbx_page_cfg *c) {
  if (!c || c->L < 1 || c->Bq < 1 || c->Bq > LBX_PAGE_MAX_REQUESTS || c->M < 1) return false;
  if (c->Hkv < 1 || c->Hq < 1 || c->Hq % c->Hkv != 0) return false;
  if (c->dh != 64 && c->dh != 128 && c->dh != 256) return false;
  if (c->page != 16 && c->page != 32 && c->page != 64 && c->page != 128 && c->page != 256)
    return false;
  if (c->n_pages < 1 || c->max_pages < 1) return false;
  if (c->dtype != LBX_BF16 && c->dtype != LBX_F16) return false;
  if (c->weights != LBX_WEIGHTS_ROUNDED && c->weights != LBX_WEIGHTS_SPLIT) return false;
  if (!(c->scale > 0.f) || !isfinite(c->scale)) return false;
  // rows, heads of rows, slots of all layers and positions have 32-bit numbers
  const long long lm = (long long)c->L * c->M, most = 0x7fffffffLL;
  if (lm > most || lm * c->Hq > most) return false;
  if ((long long)c->n_pages * c->page > most / c->L) return false;
  if ((long long)c->max_pages * c->page > (1LL << 30)) return false;
  // and values of a row
  return (long long)c->Hq * c->dh < (1LL << 29) && (long long)c->L * c->Hkv < (1LL << 30);
}

struct Span {
  const void *at;
  size_t bytes;
};
inline bool apart(const Span &a, const Span &b) {
  const uintptr_t x = (uintptr_t)a.at, y = (uintptr_t)b.at;
  return x + a.bytes <= y || y + b.bytes <= x;
}
inline bool all_apart(std::initializer_list<Span> outs, std::initializer_list<Span> ins) {
  for (const Span *o = outs.begin(); o != outs.end(); ++o) {
    for (const Span &i : ins)
      if (!apart(*o, i)) return false;
    for (const Span *p = o + 1; p != outs.end(); ++p)
      if (!apart(*o, *p)) return false;
  }
  return true;
}

// Whether a tree breaks the rules, for warp w of n: requests by warps, nodes by lanes.
// Requests whose rows request_bad refuses are passed over, whatever start holds.
__device__ __forceinline__ int trees_bad(const lbx_page_cfg &c, const int32_t *start,
                                         const int32_t *parent, int w, int n) {
  int bad = 0;
  const int lane = threadIdx.x & 31;
#pragma unroll 4
  for (int b = w; b < c.Bq; b += n) {
    const int s = start[b], e = start[b + 1];
#pragma unroll
    for (int i = lane; i < LBX_ATTN_MAX_NODES; i += 32) {
      if (s < 0 || e < s || e > c.M || i >= e - s) continue;
      const int p = parent[s + i];
      bad |= i == 0 ? p != -1 : (p < 0 || p >= i);
    }
  }
  return bad;
}

// Whether request b's rows and length break the rules.
__device__ __forceinline__ int request_bad(const lbx_page_cfg &c, int b, int s, int e, int ctx,
                                           bool tree) {
  return (b == 0 && s != 0) || s < 0 || e < s || e > c.M || ctx < 0 ||
         (long long)ctx + e - s > (long long)c.max_pages * c.page ||
         (tree && e - s > LBX_ATTN_MAX_NODES);
}

// Two fp32 at a time.
__device__ __forceinline__ uint64_t both(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float2 apart2(uint64_t v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

}  // namespace paged
}  // namespace lbx
