// cache_common.cuh -- what the operators of the bounded, shared KV cache have
// in common: host-side checks of the configuration, the whole-batch check of
// the device-side inputs, the tree's depths and masks, and which positions a
// query sees.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "lbx.h"

namespace lbx {
namespace cache {

constexpr int kMaxNodes = LBX_ATTN_MAX_NODES;

inline bool aligned_to(const void *p, uintptr_t a) {
  return p != nullptr && ((uintptr_t)p & (a - 1)) == 0;
}

// Shapes every operator supports.
inline bool cfg_ok(const lbx_attn_cfg *c) {
  if (!c || c->L < 1 || c->Bq < 1 || c->N < 1 || c->N > kMaxNodes) return false;
  if (c->Hkv < 1 || c->Hq < 1 || c->Hq % c->Hkv != 0) return false;
  if (c->dh != 64 && c->dh != 128 && c->dh != 256) return false;
  if (c->T < 0 || c->P < 0 || c->window < 0 || c->n_sink < 0) return false;
  if (c->dtype != LBX_BF16 && c->dtype != LBX_F16) return false;
  if (!(c->scale > 0.f) || !isfinite(c->scale)) return false;
  const long long lb = (long long)c->L * c->Bq;
  // 32-bit indexes of rows, streams and positions; a request's cache stays
  // below the 2^40 bytes a tensor map's stride can express
  if (lb * c->N > 0x7fffffffLL || lb * c->N * c->Hq > 0x7fffffffLL) return false;
  if (lb * c->Hkv > 0x3fffffffLL) return false;
  if (c->T > (1 << 30) || c->P > (1 << 30)) return false;
  const long long row = (long long)c->Hkv * c->dh * 2;
  const long long longest = c->T > c->P ? c->T : c->P;
  return row < (1LL << 30) && (longest < 1 || row < (1LL << 40) / longest);
}

// 1 in every thread of the block if the batch's trees, context lengths or
// accepted nodes (may be NULL) break the rules; the same verdict in every
// block, so that a bad batch writes nothing at all.
__device__ __forceinline__ int batch_bad(int Bq, int N, int T, const int32_t *ctx_len,
                                         const int32_t *parent, const int32_t *accepted) {
  int bad = 0;
  for (int i = threadIdx.x; i < Bq * N; i += blockDim.x) {
    const int n = i % N, p = parent[i];
    if (n == 0 ? p != -1 : (p < 0 || p >= n)) bad = 1;
  }
  for (int i = threadIdx.x; i < Bq; i += blockDim.x) {
    if (ctx_len[i] < 0 || ctx_len[i] > T) bad = 1;
    if (accepted && (accepted[i] < 0 || accepted[i] >= N)) bad = 1;
  }
  return __syncthreads_or(bad);
}

// The path from the root to `node` as a bit mask (its depth is the number of
// set bits less one).  The warp holds two parents per lane: following them one
// load after the other would take a trip to memory per step.
__device__ __forceinline__ uint64_t warp_path(const int32_t *parent, int N, int node, int lane) {
  const int p0 = lane < N ? parent[lane] : -1, p1 = lane + 32 < N ? parent[lane + 32] : -1;
  uint64_t m = 0;
#pragma unroll 1
  for (int s = 0; s < kMaxNodes && node >= 0; ++s) {
    m |= 1ull << node;
    const int a = __shfl_sync(0xffffffffu, p0, node & 31), b = __shfl_sync(0xffffffffu, p1, node & 31);
    node = node < 32 ? a : b;
  }
  return m;
}

}  // namespace cache
}  // namespace lbx
