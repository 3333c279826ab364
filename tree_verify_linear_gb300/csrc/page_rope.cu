// page_rope.cu -- norms of queries and keys per head, their rotation, and keys and
// values into their pages, in one pass: lbx_qk_norm_rope.
//
// A CTA takes a few rows of one layer.  First the angles: pair i of a row turns by
// pos * inv_freq[i], of which only the fraction of a turn matters.  inv_freq / (2 pi)
// is taken once per pair and CTA as a 64-bit fixed-point fraction of a turn (two
// doubles hold 1 / (2 pi)), times pos in integers modulo 2^64: no position is so far
// that an angle loses digits, as it does in a product of two floats (2^-24 of a
// million radians).  Cosines and sines lie in shared memory for all heads of the row,
// and from there in a lane's registers for as long as its warp stays with the row.
// Then the heads, a lane for two 16-byte pieces of one: with pairs in halves those that
// turn with each other (where rot is a multiple of 16; else they meet in shared
// memory), so that all arithmetic but the sum of squares stays in the lane.
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
  int half, rows, share, parts, passes;  // rows per CTA, warps per row, CTAs per row, passes of heads
  const uint4 *qkv;
  const float *qw, *kw, *freq;
  const int32_t *pos, *slot;
  uint4 *q, *k, *v;
  int32_t *status;
};

// Where the partners of a pair are: in a lane's two pieces, next to each other in one, or
// anywhere in the head.
enum { kInLane, kAdjacent, kAnywhere };

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

template <int DH, bool F16, int PAIRS>
__global__ void __launch_bounds__(kThreads) rope_kernel(const RopeArgs A) {
  constexpr int kLanes = DH / 16, kHeads = 32 / kLanes, kPieces = DH / 8;
  __shared__ float2 turn[kMaxRows][DH / 2];
  __shared__ float stage[PAIRS == kAnywhere ? kWarps : 1][512];
  __shared__ int slots[kMaxRows];
  const lbx_page_cfg &c = A.c;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int part = blockIdx.x % A.parts, groups = (c.M + A.rows - 1) / A.rows;
  const int group = blockIdx.x / A.parts % groups, l = blockIdx.x / A.parts / groups;
  const int m0 = group * A.rows, rows = c.M - m0 < A.rows ? c.M - m0 : A.rows;
  const int heads = c.Hq + 2 * c.Hkv;
  const uint4 *qkv = A.qkv + (size_t)l * c.M * heads * kPieces;
  // the lane's two pieces of a head, and whether they turn
  const int e = lane % kLanes, turning = A.half / 8;
  const bool turns = PAIRS != kInLane || e < turning;
  const int p0 = PAIRS != kInLane ? 2 * e : e < turning ? e : 2 * e;
  const int p1 = PAIRS != kInLane ? 2 * e + 1 : e < turning ? e + turning : 2 * e + 1;

  // The warp's rows r0, r0 + by, .. and passes u0, u0 + step, .. of each.
  const int r0 = warp / A.share, by = kWarps / A.share;
  const int u0 = part * A.share + warp % A.share, step = A.parts * A.share;
  auto load = [&](int r, int u, uint4 (&to)[2]) {
    const int h = u * kHeads + lane / kLanes;
    to[0] = to[1] = make_uint4(0u, 0u, 0u, 0u);
    if (r >= rows || u >= A.passes || h >= heads) return;
    const uint4 *from = qkv + ((size_t)(m0 + r) * heads + h) * kPieces;
    to[0] = __ldcs(from + p0), to[1] = __ldcs(from + p1);
  };
  uint4 next[2];
  load(r0, u0, next);
  float qw[16];  // the lane's weights of queries
  auto weights = [&](const float *w, float (&to)[16]) {
    const float4 *from = reinterpret_cast<const float4 *>(w + (size_t)l * DH);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float4 f = __ldg(from + (i < 2 ? 2 * p0 : 2 * p1 - 2) + i);
      to[4 * i] = f.x, to[4 * i + 1] = f.y, to[4 * i + 2] = f.z, to[4 * i + 3] = f.w;
    }
  };
  if (A.qw) weights(A.qw, qw);

  if (tid < rows) {
    int s = A.slot[m0 + tid];
    if (s >= c.n_pages * c.page) {
      if (A.status) *A.status = LBX_EINVAL;
      s = -1;
    }
    slots[tid] = s;
  }
  if (A.half > 0) {
    // a thread per pair, as many rows at a time as there are threads
    const int wide = A.half <= 32 ? 32 : A.half <= 64 ? 64 : 128, i = tid % wide;
    if (i < A.half) {
      int axis = 0, end = A.r.section[0];
      while (i >= end) end += A.r.section[++axis];
      const uint64_t by_pos = turns_of(A.freq[i]);
#pragma unroll 1
      for (int r = tid / wide; r < rows; r += kThreads / wide) {
        const int64_t p = A.pos[(size_t)axis * c.M + m0 + r];
        const int32_t part_of_turn = (int32_t)(((uint64_t)p * by_pos) >> 32);
        float2 cs;
        sincospif((float)part_of_turn * 4.656612873077393e-10f, &cs.y, &cs.x);  // 2^-31
        turn[r][i] = cs;
      }
    }
  }
  __syncthreads();

#pragma unroll 1
  for (int r = r0; r < rows; r += by) {
    const int slot = slots[r], m = m0 + r;
    float2 cs[8];
    if (PAIRS != kAnywhere && turns) {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        cs[i] = 8 * e + i < A.half ? turn[r][8 * e + i] : make_float2(1.f, 0.f);
    }
#pragma unroll 1
    for (int u = u0; u < A.passes; u += step) {
      const uint4 raw[2] = {next[0], next[1]};
      if (u + step < A.passes) load(r, u + step, next);
      else load(r + by, u0, next);
      if (slot < 0) continue;  // the whole warp
      const int h = u * kHeads + lane / kLanes;
      const bool is_q = h < c.Hq, is_v = h >= c.Hq + c.Hkv;
      uint4 out[2] = {raw[0], raw[1]};
      if (__any_sync(0xffffffffu, !is_v)) {
        float x[16], ss = 0.f;
        unpack8<F16>(raw[0], *reinterpret_cast<float(*)[8]>(x));
        unpack8<F16>(raw[1], *reinterpret_cast<float(*)[8]>(x + 8));
#pragma unroll
        for (int i = 0; i < 16; ++i) ss = fmaf(x[i], x[i], ss);
#pragma unroll
        for (int d = 1; d < kLanes; d *= 2) ss += __shfl_xor_sync(0xffffffffu, ss, d);
        const float inv = rsqrtf(fmaf(ss, 1.f / DH, A.r.eps));
        if (is_q ? A.qw != nullptr : A.kw != nullptr && !is_v) {
          if (is_q) {
#pragma unroll
            for (int i = 0; i < 16; ++i) x[i] *= inv * qw[i];
          } else {
            float w[16];
            weights(A.kw, w);
#pragma unroll
            for (int i = 0; i < 16; ++i) x[i] *= inv * w[i];
          }
        }
        if constexpr (PAIRS == kInLane) {
          if (turns) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const float a = x[i], b = x[8 + i];
              x[i] = a * cs[i].x - b * cs[i].y, x[8 + i] = b * cs[i].x + a * cs[i].y;
            }
          }
        } else if constexpr (PAIRS == kAdjacent) {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float a = x[2 * i], b = x[2 * i + 1];
            x[2 * i] = a * cs[i].x - b * cs[i].y, x[2 * i + 1] = b * cs[i].x + a * cs[i].y;
          }
        } else {
          float *mine = stage[warp] + lane / kLanes * DH;
#pragma unroll
          for (int i = 0; i < 4; ++i)
            reinterpret_cast<float4 *>(mine + 16 * e)[i] =
                make_float4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
          __syncwarp();
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const int j = 16 * e + i;
            if (j >= 2 * A.half) break;
            const bool second = j >= A.half;
            const float2 t = turn[r][second ? j - A.half : j];
            const float other = mine[second ? j - A.half : j + A.half];
            x[i] = fmaf(x[i], t.x, second ? other * t.y : -other * t.y);
          }
          __syncwarp();
        }
        if (!is_v) {
          out[0] = pack8<F16>(*reinterpret_cast<float(*)[8]>(x));
          out[1] = pack8<F16>(*reinterpret_cast<float(*)[8]>(x + 8));
        }
      }
      if (h >= heads) continue;
      uint4 *to;
      if (is_q)
        to = A.q + (((size_t)l * c.M + m) * c.Hq + h) * kPieces;
      else
        to = (is_v ? A.v : A.k) + (((size_t)l * c.n_pages * c.page + slot) * c.Hkv +
                                   (is_v ? h - c.Hq - c.Hkv : h - c.Hq)) * kPieces;
      to[p0] = out[0], to[p1] = out[1];
    }
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

template <int DH, bool F16>
void launch(const RopeArgs &A, unsigned grid, cudaStream_t stream) {
  if (A.r.pairing == LBX_ROPE_ADJACENT)
    rope_kernel<DH, F16, kAdjacent><<<grid, kThreads, 0, stream>>>(A);
  else if (A.half % 8 == 0)
    rope_kernel<DH, F16, kInLane><<<grid, kThreads, 0, stream>>>(A);
  else
    rope_kernel<DH, F16, kAnywhere><<<grid, kThreads, 0, stream>>>(A);
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
  const int heads = c->Hq + 2 * c->Hkv, at_once = 512 / c->dh;
  RopeArgs A = {*c, *rope, rope->rot / 2, 1, kWarps, 1, (heads + at_once - 1) / at_once,
                reinterpret_cast<const uint4 *>(qkv), q_weight, k_weight, inv_freq, pos, slot,
                reinterpret_cast<uint4 *>(q_out), reinterpret_cast<uint4 *>(k_pages),
                reinterpret_cast<uint4 *>(v_pages), d_status};
  const int nsm = lbx::cache::grid_limit();
  if (nsm < 1) return LBX_ECUDA;
  // Few rows: a CTA per row and eight warps' heads, so that the call is one trip to
  // memory.  Many: several rows share a CTA's fractions of a turn, a warp per row in the end.
  const long long lm = (long long)c->L * c->M;
  while (A.rows < kMaxRows && lm / (2 * A.rows) >= 4LL * nsm) A.rows *= 2, A.share /= 2;
  if (A.rows == 1 && lm < 4LL * nsm) A.parts = (A.passes + kWarps - 1) / kWarps;
  const long long grid = (long long)c->L * ((c->M + A.rows - 1) / A.rows) * A.parts;
  if (grid > 0x7fffffffLL) return LBX_EINVAL;
  const unsigned n = (unsigned)grid;
  const bool f16 = c->dtype == LBX_F16;
  if (c->dh == 64) f16 ? launch<64, true>(A, n, stream) : launch<64, false>(A, n, stream);
  else if (c->dh == 128) f16 ? launch<128, true>(A, n, stream) : launch<128, false>(A, n, stream);
  else f16 ? launch<256, true>(A, n, stream) : launch<256, false>(A, n, stream);
  return cudaGetLastError() == cudaSuccess ? LBX_OK : LBX_ECUDA;
}
