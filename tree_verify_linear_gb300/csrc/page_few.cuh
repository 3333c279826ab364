// page_few.cuh -- the part of lbx_paged_attention for few rows over few keys, where
// latency counts: without tensor memory or copies.
//
// The key lists of all (layer, KV head, request) are cut into units of 128 keys, one CTA
// per unit, 16 keys for each of eight warps.  Keys lie in one page then, and the warp's
// products are 8 (of 16) rows by 16 keys: warp-wide products (mma.sync) whose operands
// come straight from memory, a lane for 16 bytes of a row, with the dimensions in an order of
// their own (of K and Q the same, so that sums do not see it).  The weights of the warp's
// own softmax are an operand of its product with V as they come out of the first: rounded to V's
// type in the upper eight rows, what that loses in the lower eight, so that they are good to
// 2^-16 (f16 2^-22) at no further product.  The
// warps meet in shared memory; lists of more than one unit are joined by the CTA that
// finishes last, in the units' order.  Written for the number of instructions: each is
// fetched once and runs once (on CUDA cores, with several times as many, a call of one token
// over 2001 keys at 24/4 heads of 256 took 18.5 us; here 14.3; in tensor memory 22.5 us).
//
// What bounds it: that call takes 23000 cycles, 2000 for the check of the batch, 2300 to find the
// unit, 5000 for the loads and the scores, 3000 for V, 2200 for the warps' sums, 1500 for the
// arrival and 6000 for the join.
#pragma once

#include "cache_ptx.cuh"
#include "cache_walk.cuh"
#include "page_walk.cuh"

namespace lbx {
namespace paged {

constexpr int kThreads = 384;  // three warpgroups
constexpr int kFewWarps = 8, kFewKeys = 16 * kFewWarps;  // keys of a unit
constexpr int kFewMost = 8;                                // most rows of a list
// Units per CTA, at most: beyond, the tensor-memory kernel's copies are faster (one token over 16000
// keys, 24/4 heads of 64, 128 and 256, 3.3 units per CTA: 29, 38 and 68 us here, 22, 27 and 27 us there).
constexpr int kFewUnits = 2;

struct PageArgs {
  lbx_page_cfg c;
  int G, tp, box, shift;  // heads per group, tokens per subtile, positions per box
  Shape shape;
  float scale_log2;
  const int32_t *start, *ctx_len, *table, *parent;
  const uint16_t *q, *k, *v;
  uint16_t *o;
  float *lse, *part;
  // per CTA and subtile: pieces of the tile that begins its cut there; of few rows: per
  // list (at its first unit), its units
  unsigned int *counters;
  int32_t *status;
};

template <bool F16>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  if constexpr (F16) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
  } else {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
  }
}

template <bool F16>
__device__ __forceinline__ float2 unpack2(uint32_t v) {
  if constexpr (F16) return __half22float2(*reinterpret_cast<const __half2 *>(&v));
  else return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u));
}
// What a and b lose in pack2, rounded in its turn.
template <bool F16>
__device__ __forceinline__ uint32_t pack2_rest(float a, float b, uint32_t packed) {
  const float2 f = unpack2<F16>(packed);
  return pack2<F16>(a - f.x, b - f.y);
}

// One arrival that others of the GPU see after what this block has written before its last
// barrier; what they wrote before theirs is seen after it.
__device__ __forceinline__ unsigned arrive_count(unsigned int *count) {
  unsigned old;
  asm volatile("atom.acq_rel.gpu.global.add.u32 %0, [%1], 1;" : "=r"(old) : "l"(count) : "memory");
  return old;
}

// Units of a request's list, or very many where its rows are too many.
__device__ __forceinline__ int few_units(const PageArgs &A, int ctx, int n) {
  if (n > kFewMost / A.G) return 1 << 20;
  return n > 0 ? (ctx + n + kFewKeys - 1) / kFewKeys : 0;
}

// Rows and lengths of 32 requests from b0 on, one per lane: a warp that walks the list reads
// them once (a load takes thousands of cycles while other CTAs' copies are in flight).
struct Window {
  int b0, row0, n, ctx;
  __device__ __forceinline__ void load(const PageArgs &A, int from) {
    const int b = from + (threadIdx.x & 31);
    b0 = from;
    row0 = b < A.c.Bq ? A.start[b] : 0;
    n = b < A.c.Bq ? A.start[b + 1] - row0 : 0;
    ctx = b < A.c.Bq ? A.ctx_len[b] : 0;
  }
};

__device__ __forceinline__ int scan32(int v) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int d = 1; d < 32; d *= 2) {
    const int o = __shfl_up_sync(0xffffffffu, v, d);
    if (lane >= d) v += o;
  }
  return v;
}

// D (16 x 8, fp32) += A (16 x 16) B (16 x 8) of 16-bit values; a0 and a2 are the lane's of A's
// rows 0-7, a1 and a3 of rows 8-15.
template <bool F16>
__device__ __forceinline__ void mma_16rows(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                           uint32_t a3, uint32_t b0, uint32_t b1) {
  if constexpr (F16)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Floats of a unit's partial: a row's sums over V, then m (base 2) and l of the rows.
template <int DH>
constexpr int kFewPart = kFewMost * DH + 2 * kFewMost;

// All units of this CTA; `units`: of one (layer, KV head).  False where a page lies
// outside the pool.
template <int DH, bool F16>
__device__ __forceinline__ bool few_rows(const PageArgs &A, int units, Window win,
                                         unsigned char *smem) {
  constexpr int kWarps = kFewWarps;
  constexpr float kUp = F16 ? 7.f : 0.f;  // f16 weights are taken 2^7 times as large
  const lbx_page_cfg &c = A.c;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, j = lane & 3;
  constexpr int kPitch = DH + 4;                      // of a row, so that fewer share a bank
  float *sums = reinterpret_cast<float *>(smem);      // [warp][row][DH]
  float *m_of = sums + kWarps * kFewMost * kPitch, *l_of = m_of + kWarps * kFewMost;  // [warp][row]
  // last of the list's pieces; behind all that the join keeps (m and l of every piece, the rows'
  // sums), which it begins to write while warps still read the flag
  constexpr int kMet = kWarps * kFewMost * (kPitch + 2);
  constexpr int kJoined = (2 * kFewUnits * cache::kMaxCtas + 1) * kFewMost;
  int *flag = reinterpret_cast<int *>(sums + (kMet > kJoined ? kMet : kJoined));
  const float sl2 = A.scale_log2;
  bool inside = true;
#pragma unroll 1
  for (int u = blockIdx.x; u < units * c.L * c.Hkv; u += gridDim.x) {
    const int lh = u / units, l = lh / c.Hkv, h = lh - l * c.Hkv;
    int chunk = u - lh * units, b = 0, n = 0, ctx = 0;
    int row0 = 0;
#pragma unroll 1
    for (int b0 = 0;; b0 += 32) {
      if (b0 != win.b0) win.load(A, b0);
      const int mine = few_units(A, win.ctx, win.n), upto = scan32(mine);
      const int k = __popc(__ballot_sync(0xffffffffu, upto <= chunk));
      if (k < 32) {
        chunk -= __shfl_sync(0xffffffffu, upto - mine, k);
        b = b0 + k;
        row0 = __shfl_sync(0xffffffffu, win.row0, k);
        ctx = __shfl_sync(0xffffffffu, win.ctx, k), n = __shfl_sync(0xffffffffu, win.n, k);
        break;
      }
      chunk -= __shfl_sync(0xffffffffu, upto, 31);
    }
    const int rows = n * A.G, kv_len = ctx + n, pieces = few_units(A, ctx, n);
    auto place = [&](int r) {
      return ((size_t)l * c.M + row0 + r / A.G) * c.Hq + h * A.G + r % A.G;
    };
    const int first = chunk * kFewKeys + 16 * warp;  // the warp's keys, all in one page
    if (warp < kWarps) {
      int id = -1;
      if (first < kv_len) {
        id = A.table[(size_t)b * c.max_pages + (first >> A.shift)];
        if (id < 0 || id >= c.n_pages) inside = false, id = -1;
      }
      const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
      uint4 q[DH / 32], kx[2][DH / 32];
      {
        const uint4 *from = reinterpret_cast<const uint4 *>(A.q + place(g < rows ? g : 0) * DH) + j;
#pragma unroll
        for (int s = 0; s < DH / 32; ++s) q[s] = g < rows ? from[4 * s] : zero;
      }
      const size_t by_key = (size_t)c.Hkv * (DH / 8);  // from a key to the next, in 16 bytes
      const size_t at = ((((size_t)l * c.n_pages + (id < 0 ? 0 : id)) * c.page + (first & (c.page - 1))) *
                             c.Hkv + h) * (DH / 8);
      const uint4 *k0 = reinterpret_cast<const uint4 *>(A.k) + at;
      const uint4 *v0 = reinterpret_cast<const uint4 *>(A.v) + at;
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        const bool live = id >= 0 && first + 8 * t + g < kv_len;
#pragma unroll
        for (int s = 0; s < DH / 32; ++s)
          kx[t][s] = live ? k0[(8 * t + g) * by_key + 4 * s + j] : zero;
      }
      // V's rows 2 j, 2 j + 1, 2 j + 8, 2 j + 9, 16 bytes of 64 dimensions at a time
      auto load_v = [&](int d0, uint4 (&v)[4]) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int key = 2 * j + (e & 1) + 8 * (e >> 1);
          v[e] = id >= 0 && first + key < kv_len ? v0[key * by_key + d0 / 8 + g] : zero;
        }
      };
      // (the first half ahead of the scores, the rest as soon as K's registers are free)
      constexpr int kWide = DH / 64, kAhead = kWide < 2 ? 1 : 2;
      uint4 v[kWide][4];
#pragma unroll
      for (int d = 0; d < kAhead; ++d) load_v(64 * d, v[d]);
      // what the lane's row sees
      const int tok = g / A.G;
      int lim = id < 0 || g >= rows ? 0 : ctx + tok + 1;
      uint64_t path = 0;
      if (A.parent && lim > 0) {
        lim = ctx;
        for (int m = tok, d = 0; m >= 0 && d < LBX_ATTN_MAX_NODES; ++d)
          path |= 1ull << m, m = A.parent[row0 + m];
      }
      float x[2][4] = {};
#pragma unroll
      for (int s = 0; s < DH / 32; ++s)
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          mma_16rows<F16>(x[t], q[s].x, 0u, q[s].y, 0u, kx[t][s].x, kx[t][s].y);
          mma_16rows<F16>(x[t], q[s].z, 0u, q[s].w, 0u, kx[t][s].z, kx[t][s].w);
        }
#pragma unroll
      for (int d = kAhead; d < kWide; ++d) load_v(64 * d, v[d]);
      float m = -INFINITY, sum = 0.f;
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int pos = first + 8 * t + 2 * j + e, by = pos - ctx;
          const bool sees = pos < lim || (by >= 0 && by < 64 && (path >> by & 1));
          x[t][e] = sees ? x[t][e] * sl2 : -INFINITY;
          m = fmaxf(m, x[t][e]);
        }
      m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
      m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
      const float ref = m == -INFINITY ? 0.f : m - kUp;
      uint32_t p[2], rest[2];
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        const float p0 = ptx::ex2(x[t][0] - ref), p1 = ptx::ex2(x[t][1] - ref);
        sum += p0 + p1;
        p[t] = pack2<F16>(p0, p1), rest[t] = pack2_rest<F16>(p0, p1, p[t]);
      }
      sum += __shfl_xor_sync(0xffffffffu, sum, 1);
      sum += __shfl_xor_sync(0xffffffffu, sum, 2);
      if (j == 0) m_of[warp * kFewMost + g] = ref, l_of[warp * kFewMost + g] = sum;
      float *to = sums + (warp * kFewMost + g) * kPitch + 16 * j;
#pragma unroll
      for (int d = 0; d < kWide; ++d) {
        // product t: dimension 8 n + t of the 64 is column n
        float y[16];
#pragma unroll
        for (int t = 0; t < 8; ++t) {
          auto word = [&](int e) {
            return t < 2 ? v[d][e].x : t < 4 ? v[d][e].y : t < 6 ? v[d][e].z : v[d][e].w;
          };
          const uint32_t half = t & 1 ? 0x7632u : 0x5410u;
          float f[4] = {};
          mma_16rows<F16>(f, p[0], rest[0], p[1], rest[1], __byte_perm(word(0), word(1), half),
                          __byte_perm(word(2), word(3), half));
          y[t] = f[0] + f[2], y[8 + t] = f[1] + f[3];
        }
#pragma unroll
        for (int e = 0; e < 4; ++e)
          reinterpret_cast<float4 *>(to + 64 * d)[e] =
              make_float4(y[4 * e], y[4 * e + 1], y[4 * e + 2], y[4 * e + 3]);
      }
    }
    __syncthreads();

    // the warps' sums together; a sum of nothing has l = 0, one with a NaN is a NaN
    auto write = [&](int r, int c4, float4 f, float l_sum) {
      const float w = l_sum == 0.f ? 0.f : 1.f / l_sum;
      const uint2 to = l_sum == 0.f ? make_uint2(0u, 0u)
                                    : make_uint2(pack2<F16>(f.x * w, f.y * w), pack2<F16>(f.z * w, f.w * w));
      reinterpret_cast<uint2 *>(A.o + place(r) * DH)[c4] = to;
    };
    auto finish = [&](int r, float top, float l_sum) {
      if (A.lse)
        A.lse[place(r)] = l_sum == 0.f ? -INFINITY : (top + log2f(l_sum)) * 0.6931471805599453f;
    };
    float *part = A.part + (size_t)u * kFewPart<DH>;
#pragma unroll 1
    for (int idx = tid; idx < rows * (DH / 4); idx += kThreads) {
      const int r = idx / (DH / 4), c4 = idx % (DH / 4);
      float top = -INFINITY, l_sum = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w)
        if (l_of[w * kFewMost + r] != 0.f) top = fmaxf(top, m_of[w * kFewMost + r]);
      const float base = top == -INFINITY ? 0.f : top;
      float4 f = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float l_w = l_of[w * kFewMost + r];
        if (l_w == 0.f) continue;
        const float by = ptx::ex2(m_of[w * kFewMost + r] - base);
        const float4 y = reinterpret_cast<const float4 *>(sums + (w * kFewMost + r) * kPitch)[c4];
        l_sum = fmaf(by, l_w, l_sum);
        f.x = fmaf(by, y.x, f.x), f.y = fmaf(by, y.y, f.y);
        f.z = fmaf(by, y.z, f.z), f.w = fmaf(by, y.w, f.w);
      }
      if (pieces == 1) {
        write(r, c4, f, l_sum);
        if (c4 == 0) finish(r, top, l_sum);
      } else {
        reinterpret_cast<float4 *>(part + r * DH)[c4] = f;
        if (c4 == 0) part[kFewMost * DH + r] = top, part[kFewMost * DH + kFewMost + r] = l_sum;
      }
    }
    __syncthreads();
    if (pieces == 1) continue;
    if (tid == 0) {
      unsigned int *count = A.counters + (u - chunk);
      const bool last = arrive_count(count) == (unsigned)pieces - 1;
      if (last) *count = 0u;  // for the next call
      *flag = last;
    }
    __syncthreads();
    if (*flag) {
      // m and l of all pieces and rows; then a warp per row turns m into the piece's weight
      const float *part0 = A.part + (size_t)(u - chunk) * kFewPart<DH>;
      float *m_all = sums, *l_all = sums + pieces * kFewMost;  // [piece][row]
      float *inv_of = l_all + pieces * kFewMost;               // [row]
      float got[2][4];
#pragma unroll 1
      for (int i0 = tid; i0 < pieces * kFewMost; i0 += 4 * kThreads) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int at = i0 + i * kThreads;
          if (at >= pieces * kFewMost || at % kFewMost >= rows) continue;
          const float *from = part0 + (size_t)(at / kFewMost) * kFewPart<DH> + kFewMost * DH + at % kFewMost;
          got[0][i] = __ldcg(from), got[1][i] = __ldcg(from + kFewMost);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int at = i0 + i * kThreads;
          if (at < pieces * kFewMost) m_all[at] = got[0][i], l_all[at] = got[1][i];
        }
      }
      __syncthreads();
      if (warp < rows) {
        float top = -INFINITY, l_sum = 0.f;
        for (int e = lane; e < pieces; e += 32) top = fmaxf(top, m_all[e * kFewMost + warp]);
#pragma unroll
        for (int d = 16; d; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
        const float base = top == -INFINITY ? 0.f : top;
        for (int e = lane; e < pieces; e += 32) {
          const float by = ptx::ex2(m_all[e * kFewMost + warp] - base);
          m_all[e * kFewMost + warp] = by;
          l_sum = fmaf(by, l_all[e * kFewMost + warp], l_sum);
        }
#pragma unroll
        for (int d = 16; d; d >>= 1) l_sum += __shfl_xor_sync(0xffffffffu, l_sum, d);
        if (lane == 0) inv_of[warp] = l_sum, finish(warp, top, l_sum);
      }
      __syncthreads();
#pragma unroll 1
      for (int idx = tid; idx < rows * (DH / 4); idx += kThreads) {
        const int r = idx / (DH / 4), c4 = idx % (DH / 4);
        float4 f = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
        for (int e0 = 0; e0 < pieces; e0 += 16) {  // sixteen loads in flight
          float4 y[16];
#pragma unroll
          for (int e = 0; e < 16; ++e)
            y[e] = __ldcg(reinterpret_cast<const float4 *>(
                              part0 + (size_t)(e0 + e < pieces ? e0 + e : e0) * kFewPart<DH> + r * DH) + c4);
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const float by = e0 + e < pieces ? m_all[(e0 + e) * kFewMost + r] : 0.f;
            f.x = fmaf(by, y[e].x, f.x), f.y = fmaf(by, y[e].y, f.y);
            f.z = fmaf(by, y[e].z, f.z), f.w = fmaf(by, y[e].w, f.w);
          }
        }
        write(r, c4, f, inv_of[r]);
      }
    }
    __syncthreads();
  }
  return inside;
}

}  // namespace paged
}  // namespace lbx
