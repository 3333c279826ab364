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
  if (!(c->scale > 0.f) || !isfinite(c->scale)) return false;
  // rows, heads of rows, slots of all layers and positions have 32-bit numbers
  const long long lm = (long long)c->L * c->M, most = 0x7fffffffLL;
  if (lm > most || lm * c->Hq > most) return false;
  if ((long long)c->n_pages * c->page > most / c->L) return false;
  if ((long long)c->max_pages * c->page > (1LL << 30)) return false;
  return (long long)c->Hkv * c->dh * 2 < (1LL << 30) && (long long)c->L * c->Hkv < (1LL << 30);
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

// Whether row r of the trees breaks their rules; start has been found to rise from 0 to
// at most M, or the verdict does not matter.
__device__ __forceinline__ int tree_bad(const lbx_page_cfg &c, const int32_t *start,
                                        const int32_t *parent, int r) {
  int a = 0, z = c.Bq - 1;  // the last request that starts at r or before
  while (a < z) {
    const int h = (a + z + 1) >> 1;
    if (start[h] <= r) a = h;
    else z = h - 1;
  }
  const int p = parent[r], i = r - start[a];
  return i == 0 ? p != -1 : (p < 0 || p >= i);
}

// Whether request b's rows and length break the rules.
__device__ __forceinline__ int request_bad(const lbx_page_cfg &c, int b, int s, int e, int ctx,
                                           bool tree) {
  return (b == 0 && s != 0) || s < 0 || e < s || e > c.M || ctx < 0 ||
         (long long)ctx + e - s > (long long)c.max_pages * c.page ||
         (tree && e - s > LBX_ATTN_MAX_NODES);
}

}  // namespace paged
}  // namespace lbx
