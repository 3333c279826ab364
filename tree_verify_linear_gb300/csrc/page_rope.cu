// page_rope.cu -- norms of queries and keys per head, their rotation, and keys and
// values into their pages, in one pass: lbx_qk_norm_rope.
//
// A CTA takes a few rows of one layer.  First the angles: pair i of a row turns by
// pos * inv_freq[i], of which only the fraction of a turn matters.  inv_freq / (2 pi)
// is taken once per pair and CTA as a 64-bit fixed-point fraction of a turn, in integers
// (two doubles for 1 / (2 pi) took 1 us more at 5000 rows: an SM does few of them a cycle), times
// pos modulo 2^64: no position is so far that an angle loses digits, as it does in a
// product of two floats (2^-24 of a million radians), and no angle so small.  Cosines and sines lie in shared memory
// for all heads of the row, and from there in a lane's registers for as long as its warp stays
// with the row.  Then the heads, a lane for two 16-byte pieces of one: with pairs in halves
// those that turn with each other (where rot is a multiple of 16; else they meet in shared
// memory), so that all arithmetic but the sum of squares stays in the lane.
//
// What bounds it, measured on one GB300 (copies reach 6.79 TB/s): the instructions of few warps.
// 8052 rows of 24/4 heads of dimension 256 in bf16, 64 dimensions turned in halves: 51 us, 5.1
// TB/s; 16006 rows of 32/8 heads of 128 in f16, all turned, adjacent pairs, three axes: 68 us, 5.8
// TB/s. Halves whose partners meet in shared memory (2 layers of 13728 rows, 20/4 heads of 128 in
// f16): 91 us with 90 dimensions turned, 77 us with 128, whose partners share a lane.  (A lane per
// 16 bytes and all pairs through shared memory: 92 and 107 us for the first two; pieces loaded one
// unit ahead into registers: 56, 76, 107 and 83 us; four CTAs per SM, registers spilled, slower;
// two CTAs with the queries' weights in registers: 53, 72 and 85 us where partners share a lane,
// but 5 us faster where they meet in shared memory, so there alone.)
#include "cache_walk.cuh"
#include "page_common.cuh"
#include "page_turn.cuh"

namespace lbx {
namespace paged {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxRows = 16;  // rows of a CTA

struct RopeArgs {
  lbx_page_cfg c;
  lbx_rope_cfg r;
  int half, rows, parts, passes;  // rows per CTA, CTAs that share a row, passes of heads
  const uint4 *qkv;
  const float *qw, *kw, *freq;
  const int32_t *pos, *slot;
  uint4 *q, *k, *v;
  int32_t *status;
};

// 16 bytes into shared memory, asynchronously.
__device__ __forceinline__ void copy16(uint4 *to, const uint4 *from) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                   (uint32_t)__cvta_generic_to_shared(to)),
               "l"(from)
               : "memory");
}

// Where the partners of a pair are: in a lane's two pieces, next to each other in one, or
// anywhere in the head.
enum { kInLane, kAdjacent, kAnywhere };
constexpr int ctas_per_sm(int pairs) { return pairs == kAnywhere ? 2 : 3; }

// Eight values of a 16-byte piece, two at a time.
template <bool F16>
__device__ __forceinline__ void unpack8(const uint4 &u, uint64_t *x) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (F16) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w[i]));
      x[i] = both(f.x, f.y);
    } else {
      x[i] = both(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
    }
  }
}
template <bool F16>
__device__ __forceinline__ uint4 pack8(const uint64_t *x) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = apart2(x[i]);
    if constexpr (F16) {
      const __half2 h = __floats2half2_rn(f.x, f.y);
      w[i] = *reinterpret_cast<const uint32_t *>(&h);
    } else {
      const __nv_bfloat162 h = __floats2bfloat162_rn(f.x, f.y);
      w[i] = *reinterpret_cast<const uint32_t *>(&h);
    }
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

template <int DH, bool F16, int PAIRS>
__global__ void __launch_bounds__(kThreads, ctas_per_sm(PAIRS))
    rope_kernel(const RopeArgs A) {
  constexpr int kLanes = DH / 16, kHeads = 32 / kLanes, kPieces = DH / 8;
  __shared__ __align__(128) float2 turn[kMaxRows][DH / 2];
  // A head's dimension j lies at j + j / 8 of its kPitch: neighbouring lanes' pieces and heads
  // are nine banks apart.  Behind them a zero (-0: a dimension that does not turn takes it times
  // a sine of 0, which leaves the sign of a zero).
  constexpr int kPitch = 18 * kLanes + (32 - 9 * kLanes % 32) % 32;
  __shared__ float stage[PAIRS == kAnywhere ? kWarps : 1][kHeads * kPitch + 1];
  __shared__ int slots[kMaxRows];
  const lbx_page_cfg &c = A.c;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int part = blockIdx.x % A.parts, groups = (c.M + A.rows - 1) / A.rows;
  const int group = blockIdx.x / A.parts % groups, l = blockIdx.x / A.parts / groups;
  const int m0 = group * A.rows, rows = c.M - m0 < A.rows ? c.M - m0 : A.rows;
  const int heads = c.Hq + 2 * c.Hkv;
  const uint4 *qkv = A.qkv + (size_t)l * c.M * heads * kPieces;
  // the lane's two pieces of a head (neighbouring lanes' lie side by side), and whether
  // they turn
  const int e = lane % kLanes, turning = A.half / 8;
  const bool turns = PAIRS != kInLane || e < turning;
  const int p0 = PAIRS == kInLane && e >= turning ? turning + e : e;
  const int p1 = PAIRS == kInLane && e < turning ? turning + e : kLanes + e;

  // The warp's share of the CTA's (row, pass) units, in order: a .. z - 1.
  const int all = rows * A.passes, warps = A.parts * kWarps, gw = part * kWarps + warp;
  const int a = (int)((long long)all * gw / warps), z = (int)((long long)all * (gw + 1) / warps);
  // This lane's head in pass u is head0 + u * kHeads.
  const int head0 = lane / kLanes;
  // The units' pieces come ahead through shared memory, which costs no registers: each lane
  // reads what it copied itself.  (Of dimension 256 with its stage there is room for one.)
  // On lines of 128 bytes: 16 bytes off them the first measured case takes 55 us.
  constexpr int kAheadUnits = PAIRS != kAnywhere ? 3 : DH == 256 ? 1 : 2;
  __shared__ __align__(128) uint4 ring[kWarps][kAheadUnits][2][32];
  int left = z - a, lu = a % A.passes, at_slot = 0;  // the one to load
  const uint4 *in = qkv + (size_t)(m0 + a / A.passes) * heads * kPieces + head0 * kPieces;
  auto ahead = [&](int to) {
    if (--left >= 0) {
      const int off = lu * (kHeads * kPieces);
      if (head0 + lu * kHeads < heads) {
        copy16(&ring[warp][to][0][lane], in + off + p0);
        copy16(&ring[warp][to][1][lane], in + off + p1);
      }
      if (++lu == A.passes) lu = 0, in += heads * kPieces;
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
#pragma unroll
  for (int k = 0; k < kAheadUnits; ++k) ahead(k);
  auto weights = [&](const float *w, uint64_t (&to)[8]) {
    const float4 *from = reinterpret_cast<const float4 *>(w + (size_t)l * DH);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float4 f = __ldg(from + (i < 2 ? 2 * p0 : 2 * p1 - 2) + i);
      to[2 * i] = both(f.x, f.y), to[2 * i + 1] = both(f.z, f.w);
    }
  };

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
      const uint64_t by_pos = turns_of(__float_as_uint(A.freq[i]));
#pragma unroll 1
      for (int r = tid / wide; r < rows; r += kThreads / wide) {
        float2 cs;
        sincospif(half_turns(A.pos[(size_t)axis * c.M + m0 + r], by_pos), &cs.y, &cs.x);
        turn[r][i] = cs;
      }
    }
  }
  __syncthreads();

  // A row's cosines and sines: of pairs in the lane in twos, else per dimension, the sines
  // with the sign that the other one of the pair takes.
  uint64_t cos2[PAIRS == kInLane ? 4 : 8], sin2[PAIRS == kInLane ? 4 : 8];
  // where the other one of the pair lies, of each dimension: 8 p + i turns with 8 p + i + half or
  // 8 p + i - half, those past the last pair with the zero
  int other[PAIRS == kAnywhere ? 16 : 1];
  const bool second_turns = 2 * A.half > 8 * kLanes;  // any of the lanes' second pieces
  if constexpr (PAIRS == kAnywhere) {
    if (lane == 0) stage[warp][kHeads * kPitch] = -0.f;
    const int full = A.half >> 3, over = A.half & 7;
#pragma unroll
    for (int k = 0; k < 16; ++k) {
      const int p = k < 8 ? p0 : p1, i = k & 7, j = 8 * p + i;
      const int up = 9 * (p + full) + over + i + (i + over >= 8 ? 1 : 0);
      const int down = 9 * (p - full) - over + i - (i < over ? 1 : 0);
      other[k] = j < 2 * A.half ? head0 * kPitch + (j < A.half ? up : down) : kHeads * kPitch;
    }
  }
  // which of the lane's pairs turn: the others' values stay, whatever their neighbours are
  uint32_t turned = 0;
  if constexpr (PAIRS == kAdjacent) {
#pragma unroll
    for (int i = 0; i < 8; ++i) turned |= (uint32_t)((i < 4 ? 4 * p0 + i : 4 * p1 + i - 4) < A.half) << i;
  }
  constexpr bool kKeep = PAIRS == kAnywhere;  // the queries' weights, in registers
  uint64_t wq[8];
  if (kKeep && A.qw) weights(A.qw, wq);
  int slot = -1, r = a / A.passes, u = a % A.passes - 1;
  bool fresh = true;  // the unit begins a row, or the share
  uint4 *q_row = nullptr;
  size_t kv_row = 0;
#pragma unroll 1
  for (int unit = a; unit < z; ++unit) {
    if (++u == A.passes) u = 0, ++r, fresh = true;
    if (fresh) {
      fresh = false;
      slot = slots[r];
      q_row = A.q + ((size_t)l * c.M + m0 + r) * c.Hq * kPieces;
      kv_row = ((size_t)l * c.n_pages * c.page + (slot < 0 ? 0 : slot)) * c.Hkv * kPieces;
      if (turns) {
        auto of = [&](int i) { return i < A.half ? turn[r][i] : make_float2(1.f, 0.f); };
        if constexpr (PAIRS == kInLane) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float2 f = of(8 * e + 2 * i), g = of(8 * e + 2 * i + 1);
            cos2[i] = both(f.x, g.x), sin2[i] = both(f.y, g.y);
          }
        } else if constexpr (PAIRS == kAdjacent) {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float2 f = of(i < 4 ? 4 * p0 + i : 4 * p1 + i - 4);
            cos2[i] = both(f.x, f.x), sin2[i] = both(-f.y, f.y);
          }
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            float2 f[2];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const int j = (i < 4 ? 8 * p0 + 2 * i : 8 * p1 + 2 * i - 8) + k;
              f[k] = j < A.half ? turn[r][j] : j < 2 * A.half ? turn[r][j - A.half] : make_float2(1.f, 0.f);
              if (j < A.half) f[k].y = -f[k].y;
            }
            cos2[i] = both(f[0].x, f[1].x), sin2[i] = both(f[0].y, f[1].y);
          }
        }
      }
    }
    asm volatile("cp.async.wait_group %0;" ::"n"(kAheadUnits - 1) : "memory");
    const uint4 raw[2] = {ring[warp][at_slot][0][lane], ring[warp][at_slot][1][lane]};
    ahead(at_slot);
    if (++at_slot == kAheadUnits) at_slot = 0;
    if (slot < 0) continue;  // the whole warp
    const int h = u * kHeads + head0;
    const bool is_q = h < c.Hq, is_v = h >= c.Hq + c.Hkv;
    uint4 out[2] = {raw[0], raw[1]};
    if (__any_sync(0xffffffffu, !is_v)) {
      uint64_t x[8], s2 = 0;
      unpack8<F16>(raw[0], x);
      unpack8<F16>(raw[1], x + 4);
      const bool norm = is_q ? A.qw != nullptr : A.kw != nullptr && !is_v;
      if (__any_sync(0xffffffffu, norm)) {
#pragma unroll
        for (int i = 0; i < 8; ++i) s2 = fma2(x[i], x[i], s2);
        const float2 f = apart2(s2);
        float ss = f.x + f.y;
#pragma unroll
        for (int d = 1; d < kLanes; d *= 2) ss += __shfl_xor_sync(0xffffffffu, ss, d);
        const float inv = rsqrtf(fmaf(ss, 1.f / DH, A.r.eps));
        const uint64_t inv2 = both(inv, inv);
        if (norm) {
          auto scale = [&](const uint64_t (&w)[8]) {
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = mul2(x[i], mul2(inv2, w[i]));
          };
          if (kKeep && is_q) {
            scale(wq);
          } else {
            uint64_t w[8];
            weights(is_q ? A.qw : A.kw, w);
            scale(w);
          }
        }
      }
      if constexpr (PAIRS == kInLane) {
        if (turns) {
          const uint64_t minus = both(-1.f, -1.f);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint64_t p = x[i], q = x[4 + i];
            x[i] = fma2(mul2(q, minus), sin2[i], mul2(p, cos2[i]));
            x[4 + i] = fma2(p, sin2[i], mul2(q, cos2[i]));
          }
        }
      } else if constexpr (PAIRS == kAdjacent) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float2 f = apart2(x[i]);
          const uint64_t y = fma2(both(f.y, f.x), sin2[i], mul2(x[i], cos2[i]));
          x[i] = turned >> i & 1 ? y : x[i];
        }
      } else {
        float *mine = stage[warp] + head0 * kPitch;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          if (i >= 4 && !second_turns) break;
          const float2 f = apart2(x[i]);
          float *to = mine + (i < 4 ? 9 * p0 + 2 * i : 9 * p1 + 2 * i - 8);
          to[0] = f.x, to[1] = f.y;
        }
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          if (i >= 4 && !second_turns) break;
          x[i] = fma2(both(stage[warp][other[2 * i]], stage[warp][other[2 * i + 1]]), sin2[i],
                      mul2(x[i], cos2[i]));
        }
        __syncwarp();
      }
      if (!is_v) out[0] = pack8<F16>(x), out[1] = pack8<F16>(x + 4);
    }
    if (h >= heads) continue;
    uint4 *to = is_q   ? q_row + h * kPieces
                : is_v ? A.v + kv_row + (h - c.Hq - c.Hkv) * kPieces
                       : A.k + kv_row + (h - c.Hq) * kPieces;
    to[p0] = out[0], to[p1] = out[1];
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

int pairs_of(const RopeArgs &A) {
  if (A.r.pairing == LBX_ROPE_ADJACENT) return kAdjacent;
  return A.half % 8 == 0 ? kInLane : kAnywhere;
}

template <int DH, bool F16>
void launch(const RopeArgs &A, unsigned grid, cudaStream_t stream) {
  switch (pairs_of(A)) {
    case kAdjacent: rope_kernel<DH, F16, kAdjacent><<<grid, kThreads, 0, stream>>>(A); break;
    case kInLane: rope_kernel<DH, F16, kInLane><<<grid, kThreads, 0, stream>>>(A); break;
    default: rope_kernel<DH, F16, kAnywhere><<<grid, kThreads, 0, stream>>>(A);
  }
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
  const size_t head = (size_t)c->L * c->M * c->dh * 2;
  if (!apart({q_out, head * c->Hq}, {qkv, head * heads})) return LBX_EINVAL;
  RopeArgs A = {*c, *rope, rope->rot / 2, 1, 1, (heads + at_once - 1) / at_once,
                reinterpret_cast<const uint4 *>(qkv), q_weight, k_weight, inv_freq, pos, slot,
                reinterpret_cast<uint4 *>(q_out), reinterpret_cast<uint4 *>(k_pages),
                reinterpret_cast<uint4 *>(v_pages), d_status};
  const int nsm = lbx::cache::grid_limit();
  if (nsm < 1) return LBX_ECUDA;
  // Few rows: CTAs of eight warps' heads each, so that the call is one trip to memory.
  // Many: as many rows per CTA as fill whole rounds of the CTAs that the SMs hold.
  const long long lm = (long long)c->L * c->M, slots = (long long)ctas_per_sm(pairs_of(A)) * nsm;
  if (lm >= slots) {
    const long long rounds = (lm + slots * kMaxRows - 1) / (slots * kMaxRows);
    A.rows = (int)((lm + slots * rounds - 1) / (slots * rounds));
  } else {
    const int most = (A.passes + kWarps - 1) / kWarps;
    while (A.parts < most && lm * (A.parts + 1) <= slots) ++A.parts;
  }
  const long long grid = (long long)c->L * ((c->M + A.rows - 1) / A.rows) * A.parts;
  if (grid > 0x7fffffffLL) return LBX_EINVAL;
  const unsigned n = (unsigned)grid;
  const bool f16 = c->dtype == LBX_F16;
  if (c->dh == 64) f16 ? launch<64, true>(A, n, stream) : launch<64, false>(A, n, stream);
  else if (c->dh == 128) f16 ? launch<128, true>(A, n, stream) : launch<128, false>(A, n, stream);
  else f16 ? launch<256, true>(A, n, stream) : launch<256, false>(A, n, stream);
  return cudaGetLastError() == cudaSuccess ? LBX_OK : LBX_ECUDA;
}
