// cache_few.cu -- attention of a few rows over short key lists: what
// lbx_window_attention and lbx_prefix_attention run when a call is too small
// to pay for the tensor-memory kernel's set-up (cache_attn.cuh).
//
// The smallest calls (one layer's decode step) read a few megabytes at most, less
// than a microsecond's worth: what counts is the chain from launch to result.
// So every unit of 64 keys of every (layer, request, KV head) stream gets a CTA
// of its own, which brings its K and V at once (cp.async, unseen rows as zeros),
// multiplies with mma.sync (16 rows at most: one tile, no tensor memory to
// allocate, no barriers to set up), and leaves a partial (m, l, O) that the
// stream's last CTA to finish joins with the others in their order.  A shared
// prefix is read by each request for itself, out of L2, in the same launch.
// The loops stay rolled: code that runs once costs more to fetch than to
// execute.  Weights are split for bf16 as in cache_attn.cuh.
#include "cache_attn.cuh"

namespace lbx {
namespace cache {
namespace {

constexpr int kFewThreads = 256;
constexpr int kTile = 16;  // rows

template <int DH>
struct Few {
  static constexpr int kStride = DH * 2 + 16;  // bytes per row of Q, K, V (conflict-free)
  static constexpr int kPStride = kUnit * 2 + 16;
  static constexpr int kQ = 0;
  static constexpr int kK = kQ + kTile * kStride;
  static constexpr int kV = kK + kUnit * kStride;
  static constexpr int kP = kV + kUnit * kStride;       // hi, lo
  static constexpr int kRed = kP + 2 * kTile * kPStride;  // float [2][8][16]
  static constexpr int kSees = kRed + 2 * 8 * kTile * 4;  // uint64 [16]
  static constexpr int kBytes = kSees + kTile * 8;
};

__device__ __forceinline__ void copy16(void *dst, const void *src, bool in) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(ptx::smem_u32(dst)), "l"(src),
               "r"(in ? 16 : 0)
               : "memory");
}
template <int X, bool TRANS>
__device__ __forceinline__ void load_tiles(uint32_t (&r)[X], uint32_t at) {
  if constexpr (X == 4)
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(at)
                 : "memory");
  else if constexpr (TRANS)
    asm volatile("ldmatrix.sync.aligned.m8n8.x2.trans.shared.b16 {%0, %1}, [%2];"
                 : "=r"(r[0]), "=r"(r[1])
                 : "r"(at)
                 : "memory");
  else
    asm volatile("ldmatrix.sync.aligned.m8n8.x2.shared.b16 {%0, %1}, [%2];"
                 : "=r"(r[0]), "=r"(r[1])
                 : "r"(at)
                 : "memory");
}
template <bool F16>
__device__ __forceinline__ void mma16(float (&c)[4], const uint32_t (&a)[4],
                                      const uint32_t (&b)[2]) {
  if constexpr (F16)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
}

// Floats of a partial: m (base 2) and l per row, then O [16][DH].
constexpr size_t few_floats(int dh) { return 2 * (size_t)kTile + (size_t)kTile * dh; }

template <int DH, bool F16>
__global__ void __launch_bounds__(kFewThreads) few_rows_kernel(const FewArgs A) {
  using Y = Few<DH>;
  extern __shared__ __align__(16) unsigned char few_smem[];
  unsigned char *smem = few_smem;
  __shared__ int last;
  const lbx_attn_cfg &c = A.c;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int G = c.Hq / c.Hkv, rows = c.N * G;
  const int stream = blockIdx.x / A.chunks, chunk = blockIdx.x - stream * A.chunks;
  const int h = stream % c.Hkv, lb = stream / c.Hkv, l = lb / c.Bq, b = lb - l * c.Bq;

  // ---- the key list, as in Walk, behind the prefix ----
  const int ctx = A.ctx_len[b], pre = (c.P + kUnit - 1) / kUnit;
  const int w0 = c.window > 0 && ctx - c.window + 1 > 0 ? ctx - c.window + 1 : 0;
  const int s_eff = c.n_sink < w0 ? c.n_sink : w0;
  const int ns = (s_eff + kUnit - 1) / kUnit, nw = (ctx - w0 + kUnit - 1) / kUnit;
  const int units = pre + ns + nw + 1;
  if (batch_bad(c.Bq, c.N, c.T, A.ctx_len, A.parent, nullptr)) {
    if (tid == 0 && A.status) *A.status = LBX_ETREE;
    return;
  }
  if (chunk >= units) return;
  const int u = chunk - pre;
  const bool in_pre = u < 0, tree = u == ns + nw;
  const int start = in_pre ? chunk * kUnit : u < ns ? u * kUnit : tree ? 0 : w0 + (u - ns) * kUnit;
  const int end = in_pre ? c.P : u < ns ? s_eff : tree ? c.N : ctx;
  const int cnt = end - start < kUnit ? end - start : kUnit;

  // ---- K, V and Q in, 16 bytes per thread and copy ----
  constexpr int kPer = DH / 8;
  const size_t first = (in_pre ? (size_t)l * c.P : tree ? (size_t)lb * c.N : (size_t)lb * c.T) + start;
  const uint16_t *kg = (in_pre ? A.kp : tree ? A.kt : A.kc) + (first * c.Hkv + h) * DH;
  const uint16_t *vg = (in_pre ? A.vp : tree ? A.vt : A.vc) + (first * c.Hkv + h) * DH;
#pragma unroll 2
  for (int i = tid; i < kUnit * kPer; i += kFewThreads) {
    const int key = i / kPer, p = i % kPer;
    const bool in = key < cnt;
    const size_t off = in ? (size_t)key * c.Hkv * DH + p * 8 : 0;
    copy16(smem + Y::kK + key * Y::kStride + p * 16, kg + off, in);
  }
#pragma unroll 1
  for (int i = tid; i < kTile * kPer; i += kFewThreads) {
    const int r = i / kPer, p = i % kPer, node = r / G;
    const bool in = r < rows;
    const size_t q = ((size_t)lb * c.N + node) * c.Hq + h * G + (r - node * G);
    copy16(smem + Y::kQ + r * Y::kStride + p * 16, A.q + (in ? q * DH + p * 8 : 0), in);
  }
  asm volatile("cp.async.commit_group;" ::: "memory");
#pragma unroll 2
  for (int i = tid; i < kUnit * kPer; i += kFewThreads) {
    const int key = i / kPer, p = i % kPer;
    const bool in = key < cnt;
    const size_t off = in ? (size_t)key * c.Hkv * DH + p * 8 : 0;
    copy16(smem + Y::kV + key * Y::kStride + p * 16, vg + off, in);
  }
  asm volatile("cp.async.commit_group;" ::: "memory");

  // ---- which keys of the unit each row sees ----
  uint64_t *sees = reinterpret_cast<uint64_t *>(smem + Y::kSees);
  if (warp == 0) {
    uint64_t bits = low_bits(cnt);
    const int node = lane < rows ? lane / G : 0;  // rows past the last: as the root's
    if (!in_pre) {
      uint64_t anc = 0;
      for (int n = node; n >= 0; n = A.parent[(size_t)b * c.N + n]) anc |= 1ull << n;
      const int at = ctx + __popcll(anc) - 1, lo = c.window > 0 ? at - c.window + 1 : 0;
      if (!tree) {
        bits &= ~low_bits(lo - start) | low_bits(c.n_sink - start);
      } else {
        bits = anc;
        uint64_t m = anc;
#pragma unroll 1
        for (int pos = ctx; m; ++pos, m &= m - 1)  // nodes of the path, root first
          if (pos < lo && pos >= c.n_sink) bits &= ~(m & (0 - m));
      }
    }
    if (lane < kTile) sees[lane] = bits;
  }
  asm volatile("cp.async.wait_group 1;" ::: "memory");
  __syncthreads();

  // ---- S: a warp per eight keys ----
  const uint32_t base = ptx::smem_u32(smem);
  float s[4] = {0.f, 0.f, 0.f, 0.f};
  {
    const uint32_t qa = base + Y::kQ + (lane & 15) * Y::kStride + (lane >> 4) * 16;
    const uint32_t kb = base + Y::kK + (warp * 8 + (lane & 7)) * Y::kStride + (lane >> 3 & 1) * 16;
#pragma unroll 4
    for (int k = 0; k < DH * 2; k += 32) {
      uint32_t a[4], w[2];
      load_tiles<4, false>(a, qa + k);
      load_tiles<2, false>(w, kb + k);
      mma16<F16>(s, a, w);
    }
  }
  // rows lane / 4 and + 8, keys 8 warp + 2 (lane % 4) and + 1
  const int row = lane >> 2, col = warp * 8 + (lane & 3) * 2;
  float *m_of = reinterpret_cast<float *>(smem + Y::kRed), *l_of = m_of + 8 * kTile;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const bool ok = sees[row + (e >> 1) * 8] >> (col + (e & 1)) & 1;
    s[e] = ok ? s[e] * A.scale_log2 : -INFINITY;
  }
  float m[2] = {fmaxf(s[0], s[1]), fmaxf(s[2], s[3])};
#pragma unroll
  for (int w = 1; w < 4; w *= 2)
    m[0] = fmaxf(m[0], __shfl_xor_sync(0xffffffffu, m[0], w)),
    m[1] = fmaxf(m[1], __shfl_xor_sync(0xffffffffu, m[1], w));
  if ((lane & 3) == 0) m_of[warp * kTile + row] = m[0], m_of[warp * kTile + row + 8] = m[1];
  __syncthreads();
  float sum[2];
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    m[e] = -INFINITY;
#pragma unroll
    for (int w = 0; w < 8; ++w) m[e] = fmaxf(m[e], m_of[w * kTile + row + e * 8]);
    const float ref = m[e] == -INFINITY ? 0.f : m[e];
    const float p0 = ptx::ex2(s[2 * e] - ref), p1 = ptx::ex2(s[2 * e + 1] - ref);
    sum[e] = p0 + p1;
    sum[e] += __shfl_xor_sync(0xffffffffu, sum[e], 1);
    sum[e] += __shfl_xor_sync(0xffffffffu, sum[e], 2);
    const uint32_t hi = pack2<F16>(p0, p1);
    unsigned char *to = smem + Y::kP + (row + e * 8) * Y::kPStride + col * 2;
    *reinterpret_cast<uint32_t *>(to) = hi;
    if constexpr (!F16)
      *reinterpret_cast<uint32_t *>(to + kTile * Y::kPStride) =
          pack2<false>(p0 - __uint_as_float(hi << 16), p1 - __uint_as_float(hi & 0xffff0000u));
  }
  if ((lane & 3) == 0) l_of[warp * kTile + row] = sum[0], l_of[warp * kTile + row + 8] = sum[1];
  asm volatile("cp.async.wait_group 0;" ::: "memory");
  __syncthreads();

  // ---- O: a warp per DH / 8 columns ----
  constexpr int kTiles = DH / 64;
  float o[kTiles][4];
#pragma unroll
  for (int t = 0; t < kTiles; ++t) o[t][0] = o[t][1] = o[t][2] = o[t][3] = 0.f;
#pragma unroll 1
  for (int k = 0; k < kUnit; k += 16) {
#pragma unroll
    for (int part = kParts<F16> - 1; part >= 0; --part) {
      uint32_t a[4];
      load_tiles<4, false>(a, base + Y::kP + part * kTile * Y::kPStride +
                                  (lane & 15) * Y::kPStride + (lane >> 4) * 16 + k * 2);
#pragma unroll
      for (int t = 0; t < kTiles; ++t) {
        uint32_t w[2];
        load_tiles<2, true>(w, base + Y::kV + (k + (lane & 15)) * Y::kStride +
                                   (warp * kTiles + t) * 16);
        mma16<F16>(o[t], a, w);
      }
    }
  }
  float total[2] = {0.f, 0.f};
#pragma unroll
  for (int w = 0; w < 8; ++w)
    total[0] += l_of[w * kTile + row], total[1] += l_of[w * kTile + row + 8];

  // ---- the result, or a partial of it ----
  auto query = [&](int r) {
    const int node = r / G;
    return ((size_t)lb * c.N + node) * c.Hq + h * G + (r - node * G);
  };
  auto put_lse = [&](int r, float m2, float sum1) {
    if (A.lse) A.lse[query(r)] = sum1 == 0.f ? -INFINITY : (m2 + __log2f(sum1)) * 0.6931471805599453f;
  };
  if (units == 1) {
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int r = row + e * 8;
      if (r >= rows) continue;
      const float w = total[e] == 0.f ? 0.f : __fdividef(1.f, total[e]);
#pragma unroll
      for (int t = 0; t < kTiles; ++t)
        reinterpret_cast<uint32_t *>(A.o + query(r) * DH)[(warp * kTiles + t) * 4 + (lane & 3)] =
            pack2<F16>(o[t][2 * e] * w, o[t][2 * e + 1] * w);
      if (warp == 0 && (lane & 3) == 0) put_lse(r, m[e], total[e]);
    }
    return;
  }
  float *part = A.part + ((size_t)stream * A.chunks + chunk) * few_floats(DH);
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const int r = row + e * 8;
    if (r >= rows) continue;
    if (warp == 0 && (lane & 3) == 0) part[r] = m[e], part[kTile + r] = total[e];
#pragma unroll
    for (int t = 0; t < kTiles; ++t)
      reinterpret_cast<float2 *>(part + 2 * kTile + r * DH)[(warp * kTiles + t) * 4 + (lane & 3)] =
          make_float2(o[t][2 * e], o[t][2 * e + 1]);
  }
  __syncthreads();
  if (tid == 0) {
    __threadfence();  // the CTA's partial, before its arrival
    last = atomicAdd(&A.counters[stream], 1u) == (unsigned)units - 1;
    if (last) A.counters[stream] = 0u;  // for the next call
    __threadfence();
  }
  __syncthreads();
  if (!last) return;

  // ---- join: the partials' weights (in K's place), then four columns per thread ----
  float *w_of = reinterpret_cast<float *>(smem + Y::kK), *s_of = w_of + units * kTile;
  const float *part0 = A.part + (size_t)stream * A.chunks * few_floats(DH);
#pragma unroll 2
  for (int i = tid; i < units * kTile; i += kFewThreads) {
    const float *from = part0 + (i / kTile) * few_floats(DH) + i % kTile;
    if (i % kTile < rows) w_of[i] = __ldcg(from), s_of[i] = __ldcg(from + kTile);
  }
  __syncthreads();
  if (tid < rows) {
    float top = -INFINITY, sum1 = 0.f;
#pragma unroll 2
    for (int i = tid; i < units * kTile; i += kTile) top = fmaxf(top, w_of[i]);
    const float ref = top == -INFINITY ? 0.f : top;
#pragma unroll 2
    for (int i = tid; i < units * kTile; i += kTile) {
      const float w = ptx::ex2(w_of[i] - ref);
      w_of[i] = w, sum1 = fmaf(w, s_of[i], sum1);
    }
    put_lse(tid, ref, sum1);
    s_of[tid] = sum1 == 0.f ? 0.f : __fdividef(1.f, sum1);
  }
  __syncthreads();
#pragma unroll 1
  for (int i = tid; i < rows * (DH / 4); i += kFewThreads) {
    const int r = i / (DH / 4), c4 = i % (DH / 4);
    float4 f = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
    for (int e = 0; e < units; ++e) {
      const float w = w_of[e * kTile + r];
      const float4 y = __ldcg(
          reinterpret_cast<const float4 *>(part0 + e * few_floats(DH) + 2 * kTile + r * DH) + c4);
      f.x = fmaf(w, y.x, f.x), f.y = fmaf(w, y.y, f.y);
      f.z = fmaf(w, y.z, f.z), f.w = fmaf(w, y.w, f.w);
    }
    const float w = s_of[r];
    reinterpret_cast<uint2 *>(A.o + query(r) * DH)[c4] =
        make_uint2(pack2<F16>(f.x * w, f.y * w), pack2<F16>(f.z * w, f.w * w));
  }
}

template <int DH>
cudaError_t launch(bool f16, const FewArgs &A, int grid, cudaStream_t stream) {
  auto kernel = f16 ? few_rows_kernel<DH, true> : few_rows_kernel<DH, false>;
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             Few<DH>::kBytes);
  if (e != cudaSuccess) return e;
  kernel<<<(unsigned)grid, kFewThreads, Few<DH>::kBytes, stream>>>(A);
  return cudaGetLastError();
}

}  // namespace

int few_chunks(const lbx_attn_cfg *c) {
  const long long rows = (long long)c->N * (c->Hq / c->Hkv);
  if (rows > kTile) return 0;
  auto units = [](long long n) { return (n + kUnit - 1) / kUnit; };
  // the most a request can have, over all context lengths up to T: once the
  // context is as long as the window its first position is on its own, W - 1
  // cached positions are in the window and the others, up to n_sink, before it
  const long long W = c->window, before = c->T - (W - 1);
  const long long own = W > 0 && before > 0
                            ? units(W - 1) + units(c->n_sink < before ? c->n_sink : before)
                            : units(c->T);
  const long long n = units(c->P) + own + 1, all = n * c->L * c->Bq * c->Hkv;
  // Up to about one wave of CTAs it is the faster one, beyond the other is (at
  // dimensions 64 and 128, whose units are smaller, some way beyond): us per call here /
  // there, bf16, 24 query heads over 4 of dimension 256,
  //   9 units per stream, 4 streams    9.3 / 15.4
  //   17 units, 16 streams            13.1 / 17.6
  //   64 units, 4 streams             21.9 / 28.5
  //   42 units, 12 streams            24.7 / 21.3
  //   64 units, 8 streams             28.4 / 23.4
  // and, with a prefix (two launches there),
  //   21 units, 20 streams            20.3 / 26.4
  //   29 units, 32 streams (dh 128)   17.4 / 23.5
  //   63 units, 16 streams            37.8 / 42.8
  //   32 units, 32 streams            31.7 / 30.6
  // Four heads per KV head, one token, from a graph (dimension 64 f16; 128 bf16; 256 f16):
  //   24 units, 4 streams              9.9 / 14.5     8.9 / 16.7    10.0 / 21.1
  //   62 units, 4 streams             18.7 / 18.2    16.2 / 20.9    18.9 / 31.7
  //   24 units, 16 streams            11.7 / 15.7    11.3 / 17.8    18.3 / 19.9
  //   12 units, 32 streams            10.0 / 14.1    10.6 / 16.7    17.1 / 18.8
  //   48 units, 16 streams            18.9 / 17.2    18.2 / 19.8    28.5 / 24.2
  //   12 units, 64 streams            12.1 / 14.4    15.0 / 16.9    23.7 / 23.3
  // and, with a prefix,
  //   20 units, 16 streams            10.8 / 18.1    11.1 / 22.6    15.2 / 25.0
  //   60 units, 16 streams            22.0 / 22.1    21.7 / 24.9    33.6 / 40.9
  //   32 units, 32 streams            17.1 / 22.5    18.2 / 24.7    29.0 / 33.3
  // The join's weights fit in K's place up to 64 units.
  return n <= 64 && all <= (c->P > 0 ? kFewUnits : kFewUnits * 3 / 8) ? (int)n : 0;
}

cudaError_t launch_few(const FewArgs &A, cudaStream_t stream) {
  const int grid = A.c.L * A.c.Bq * A.c.Hkv * A.chunks;
  const bool f16 = A.c.dtype == LBX_F16;
  return A.c.dh == 64    ? launch<64>(f16, A, grid, stream)
         : A.c.dh == 128 ? launch<128>(f16, A, grid, stream)
                         : launch<256>(f16, A, grid, stream);
}

}  // namespace cache
}  // namespace lbx
