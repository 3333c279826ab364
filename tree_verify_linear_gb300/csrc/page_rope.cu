// page_rope.cu -- norms of queries and keys per head, their rotation, and keys and
// values into their pages, in one pass: lbx_qk_norm_rope.
//
// A CTA takes a few rows of one layer.  First the angles: pair i of a row turns by
// pos * inv_freq[i], of which only the fraction of a turn matters.  inv_freq / (2 pi)
// is taken once per pair and CTA as a 64-bit fixed-point fraction of a turn (two
// doubles hold 1 / (2 pi)), times pos in integers modulo 2^64: no position is so far
// that an angle loses digits, as it does in a product of two floats (2^-24 of a
// million radians).  Cosines and sines lie in shared memory for all heads of the row.
// Then the heads, a lane for 16 bytes of one: the sum of squares by shuffles, the
// partners of a pair in halves through the warp's own shared memory (any even rot;
// adjacent pairs lie in one lane), results rounded once.  The next head's load is
// under way while one is worked on.
#include "cache_walk.cuh"
#include "page_common.cuh"

namespace lbx {
namespace paged {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxRows = 8;  // rows of a CTA

struct RopeArgs {
  lbx_page_cfg c;
  lbx_rope_cfg r;
  int half, rows, parts, passes;  // rows per CTA; CTAs that share a row's heads; passes of heads
  const uint4 *qkv;
  const float *qw, *kw, *freq;
  const int32_t *pos, *slot;
  uint4 *q, *k, *v;
  int32_t *status;
};

// f / (2 pi) modulo 1, in units of 2^-64.
__device__ __forceinline__ uint64_t turns_of(float f) {
  const double kHi = 0.15915494309189535, kLo = -9.839338337591243e-18;
  const double x = f, p = x * kHi, rest = fma(x, kLo, fma(x, kHi, -p));
  return __double2ull_rz((p - floor(p)) * 18446744073709551616.0) +
         (uint64_t)__double2ll_rn(rest * 18446744073709551616.0);
}

template <bool F16>
__device__ __forceinline__ void unpack8(const uint4 &u, float (&x)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (F16) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w[i]));
      x[2 * i] = f.x, x[2 * i + 1] = f.y;
    } else {
      x[2 * i] = __uint_as_float(w[i] << 16), x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
}
template <bool F16>
__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (F16) {
      const __half2 h = __floats2half2_rn(x[2 * i], x[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t *>(&h);
    } else {
      const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t *>(&h);
    }
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

template <int DH, bool F16>
__global__ void __launch_bounds__(kThreads) rope_kernel(const RopeArgs A) {
  constexpr int kLanes = DH / 8, kHeads = 32 / kLanes;  // lanes of a head, heads of a pass
  __shared__ float2 turn[kMaxRows][DH / 2];
  __shared__ float stage[kWarps][256];
  __shared__ int slots[kMaxRows];
  const lbx_page_cfg &c = A.c;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int part = blockIdx.x % A.parts, groups = (c.M + A.rows - 1) / A.rows;
  const int group = blockIdx.x / A.parts % groups, l = blockIdx.x / A.parts / groups;
  const int m0 = group * A.rows, rows = c.M - m0 < A.rows ? c.M - m0 : A.rows;
  const int heads = c.Hq + 2 * c.Hkv;
  const uint4 *qkv = A.qkv + (size_t)l * c.M * heads * kLanes;
  const int e = lane % kLanes;  // 16 bytes of the head

  // unit u: a row and `kHeads` of its heads
  const int units = rows * A.passes, step = A.parts * kWarps;
  auto head_of = [&](int u) { return u % A.passes * kHeads + lane / kLanes; };
  auto load = [&](int u) {
    const int h = head_of(u);
    if (u >= units || h >= heads) return make_uint4(0u, 0u, 0u, 0u);
    return __ldcs(qkv + ((size_t)(m0 + u / A.passes) * heads + h) * kLanes + e);
  };
  int u = part * kWarps + warp;
  uint4 next = load(u);

  if (tid < rows) {
    int s = A.slot[m0 + tid];
    if (s >= c.n_pages * c.page) {
      if (A.status) *A.status = LBX_EINVAL;
      s = -1;
    }
    slots[tid] = s;
  }
#pragma unroll 1
  for (int i = tid % (DH / 2); i < A.half; i += DH / 2) {
    int axis = 0, end = A.r.section[0];
    while (i >= end) end += A.r.section[++axis];
    const uint64_t by = turns_of(A.freq[i]);
#pragma unroll 1
    for (int r = tid / (DH / 2); r < rows; r += kThreads / (DH / 2)) {
      const int64_t p = A.pos[(size_t)axis * c.M + m0 + r];
      const int32_t part_of_turn = (int32_t)(((uint64_t)p * by) >> 32);
      float2 cs;
      sincospif((float)part_of_turn * 4.656612873077393e-10f, &cs.y, &cs.x);  // 2^-31
      turn[r][i] = cs;
    }
  }
  __syncthreads();

#pragma unroll 1
  for (; u < units; u += step) {
    const uint4 raw = next;
    next = load(u + step);
    const int r = u / A.passes, h = head_of(u), slot = slots[r], m = m0 + r;
    if (slot < 0) continue;  // the whole warp
    const bool norm_q = h < c.Hq, turns = h < c.Hq + c.Hkv;
    const float *w = norm_q ? A.qw : A.kw;
    uint4 out = raw;
    if (__any_sync(0xffffffffu, turns)) {
      float x[8];
      unpack8<F16>(raw, x);
      float ss = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) ss = fmaf(x[i], x[i], ss);
#pragma unroll
      for (int d = 1; d < kLanes; d *= 2) ss += __shfl_xor_sync(0xffffffffu, ss, d);
      if (w != nullptr && turns) {
        const float inv = 1.f / sqrtf(fmaf(ss, 1.f / DH, A.r.eps));
        const float4 *wv = reinterpret_cast<const float4 *>(w + (size_t)l * DH) + 2 * e;
        const float4 w0 = wv[0], w1 = wv[1];
        x[0] *= inv * w0.x, x[1] *= inv * w0.y, x[2] *= inv * w0.z, x[3] *= inv * w0.w;
        x[4] *= inv * w1.x, x[5] *= inv * w1.y, x[6] *= inv * w1.z, x[7] *= inv * w1.w;
      }
      if (A.r.pairing == LBX_ROPE_ADJACENT) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (4 * e + i >= A.half) break;
          const float2 cs = turn[r][4 * e + i];
          const float a = x[2 * i], b = x[2 * i + 1];
          x[2 * i] = a * cs.x - b * cs.y, x[2 * i + 1] = b * cs.x + a * cs.y;
        }
      } else {
        float *mine = stage[warp] + lane / kLanes * DH;
#pragma unroll
        for (int i = 0; i < 8; ++i) mine[8 * e + i] = x[i];
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int j = 8 * e + i;
          if (j >= 2 * A.half) break;
          const bool second = j >= A.half;
          const float2 cs = turn[r][second ? j - A.half : j];
          const float other = mine[second ? j - A.half : j + A.half];
          x[i] = fmaf(x[i], cs.x, second ? other * cs.y : -other * cs.y);
        }
        __syncwarp();
      }
      if (turns) out = pack8<F16>(x);
    }
    if (h >= heads) continue;
    uint4 *to;
    if (norm_q)
      to = A.q + (((size_t)l * c.M + m) * c.Hq + h) * kLanes;
    else
      to = (turns ? A.k : A.v) + (((size_t)l * c.n_pages * c.page + slot) * c.Hkv +
                                  (turns ? h - c.Hq : h - c.Hq - c.Hkv)) * kLanes;
    to[e] = out;
  }
}

bool rope_ok(const lbx_page_cfg *c, const lbx_rope_cfg *r) {
  if (!r || r->rot < 0 || r->rot % 2 != 0 || r->rot > c->dh) return false;
  if (r->axes < 1 || r->axes > LBX_ROPE_MAX_AXES) return false;
  if (r->pairing != LBX_ROPE_HALVES && r->pairing != LBX_ROPE_ADJACENT) return false;
  if (!(r->eps >= 0.f) || !isfinite(r->eps)) return false;
  long long sum = 0;
  for (int a = 0; a < LBX_ROPE_MAX_AXES; ++a) {
    if (r->section[a] < 0 || (a >= r->axes && r->section[a] != 0)) return false;
    sum += r->section[a];
  }
  return sum == r->rot / 2;
}

template <int DH>
void launch(bool f16, const RopeArgs &A, unsigned grid, cudaStream_t stream) {
  if (f16) rope_kernel<DH, true><<<grid, kThreads, 0, stream>>>(A);
  else rope_kernel<DH, false><<<grid, kThreads, 0, stream>>>(A);
}

}  // namespace
}  // namespace paged
}  // namespace lbx

extern "C" int lbx_qk_norm_rope(const lbx_page_cfg *c, const lbx_rope_cfg *rope,
                                const uint16_t *qkv, const float *q_weight, const float *k_weight,
                                const float *inv_freq, const int32_t *pos, const int32_t *slot,
                                uint16_t *q_out, uint16_t *k_pages, uint16_t *v_pages,
                                int32_t *d_status, cudaStream_t stream) {
  using namespace lbx::paged;
  if (!cfg_ok(c) || !rope_ok(c, rope)) return LBX_EINVAL;
  for (const uint16_t *p : {qkv, (const uint16_t *)q_out, (const uint16_t *)k_pages,
                            (const uint16_t *)v_pages})
    if (!aligned_to(p, 16)) return LBX_EINVAL;
  if ((q_weight && !aligned_to(q_weight, 16)) || (k_weight && !aligned_to(k_weight, 16)) ||
      (rope->rot > 0 && !aligned_to(inv_freq, 4)) || !aligned_to(pos, 4) || !aligned_to(slot, 4) ||
      (d_status && !aligned_to(d_status, 4)))
    return LBX_EINVAL;
  const int heads = c->Hq + 2 * c->Hkv, at_once = 256 / c->dh;
  RopeArgs A = {*c, *rope, rope->rot / 2, 1, 1, (heads + at_once - 1) / at_once,
                reinterpret_cast<const uint4 *>(qkv), q_weight, k_weight, inv_freq, pos, slot,
                reinterpret_cast<uint4 *>(q_out), reinterpret_cast<uint4 *>(k_pages),
                reinterpret_cast<uint4 *>(v_pages), d_status};
  const int nsm = lbx::cache::grid_limit();
  if (nsm < 1) return LBX_ECUDA;
  // Few rows: a CTA per row and eight warps' heads, so that the call is one trip to
  // memory.  Many: several rows share a CTA's fractions of a turn.
  const long long lm = (long long)c->L * c->M;
  while (A.rows < kMaxRows && lm / (2 * A.rows) >= 8LL * nsm) A.rows *= 2;
  if (A.rows == 1 && lm < 4LL * nsm) A.parts = (A.passes + kWarps - 1) / kWarps;
  const long long grid = (long long)c->L * ((c->M + A.rows - 1) / A.rows) * A.parts;
  if (grid > 0x7fffffffLL) return LBX_EINVAL;
  const bool f16 = c->dtype == LBX_F16;
  if (c->dh == 64) launch<64>(f16, A, (unsigned)grid, stream);
  else if (c->dh == 128) launch<128>(f16, A, (unsigned)grid, stream);
  else launch<256>(f16, A, (unsigned)grid, stream);
  return cudaGetLastError() == cudaSuccess ? LBX_OK : LBX_ECUDA;
}
