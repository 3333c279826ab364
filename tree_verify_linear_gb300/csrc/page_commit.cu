// page_commit.cu -- keep the verified path of each request's tree in a paged
// cache: lbx_page_commit.
//
// A CTA takes 16-byte columns of one request's and layer's rows.  The i-th node of
// the path moves to place i; its index m_i is at least i, and m_j > m_i >= i for
// every later node, so that no move overwrites what a later one reads: each thread
// takes its column of the path's rows in order, eight loads in flight.
//
// What bounds it: copies of scattered rows.  64 requests, paths of 40 nodes, 16 layers,
// 8 heads of dimension 128: 59 us, 5.5 TB/s read and written (copies reach 6.79 TB/s); five
// paths of 6 nodes, 16 layers, 4 heads of 256: 3.5 us in a captured graph, the trips to memory.
#include "page_common.cuh"

namespace lbx {
namespace paged {
namespace {

constexpr int kThreads = 256;
constexpr int kFly = 8;

struct CommitArgs {
  lbx_page_cfg c;
  int shift, cols, parts;  // 16-byte columns of a row, CTAs per request and layer
  const int32_t *start, *ctx_len, *table, *parent, *accepted;
  uint4 *k, *v;
  int32_t *ctx_out, *status;
};

__global__ void __launch_bounds__(kThreads) page_commit_kernel(const CommitArgs A) {
  const lbx_page_cfg &c = A.c;
  __shared__ int place[LBX_ATTN_MAX_NODES], from[LBX_ATTN_MAX_NODES], len;
  const int tid = threadIdx.x;
  int bad = trees_bad(c, A.start, A.parent, tid >> 5, kThreads / 32);
  for (int b = tid; b < c.Bq; b += kThreads) {
    const int s = A.start[b], e = A.start[b + 1];
    bad |= request_bad(c, b, s, e, A.ctx_len[b], true);
    if (e > s) bad |= A.accepted[b] < 0 || A.accepted[b] >= e - s;
  }
  if (__syncthreads_or(bad)) {
    if (tid == 0 && A.status) *A.status = LBX_ETREE;
    return;
  }
  const int part = blockIdx.x % A.parts, lb = blockIdx.x / A.parts;
  const int b = lb % c.Bq, l = lb / c.Bq;
  const int s = A.start[b], n = A.start[b + 1] - s, ctx = A.ctx_len[b];
  if (n == 0) {
    if (lb < c.Bq && part == 0 && tid == 0) A.ctx_out[b] = ctx;
    return;
  }
  if (tid < 32) {
    // The path's nodes as bits, by doubling: after step k a lane has its two nodes' nearest
    // 2^k ancestors and the one behind them.
    const int acc = A.accepted[b];
    int up[2] = {tid < n ? A.parent[s + tid] : -1, tid + 32 < n ? A.parent[s + tid + 32] : -1};
    uint64_t anc[2] = {1ull << tid, 1ull << (tid + 32)};
#pragma unroll
    for (int k = 0; k < 6; ++k) {
      uint64_t add[2];
      int to[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const uint64_t a0 = __shfl_sync(0xffffffffu, anc[0], up[e] & 31);
        const uint64_t a1 = __shfl_sync(0xffffffffu, anc[1], up[e] & 31);
        const int u0 = __shfl_sync(0xffffffffu, up[0], up[e] & 31);
        const int u1 = __shfl_sync(0xffffffffu, up[1], up[e] & 31);
        add[e] = up[e] < 0 ? 0ull : up[e] < 32 ? a0 : a1;
        to[e] = up[e] < 0 ? -1 : up[e] < 32 ? u0 : u1;
      }
      anc[0] |= add[0], anc[1] |= add[1], up[0] = to[0], up[1] = to[1];
    }
    const uint64_t m0 = __shfl_sync(0xffffffffu, anc[0], acc & 31);
    const uint64_t m1 = __shfl_sync(0xffffffffu, anc[1], acc & 31);
    const uint64_t m = acc < 32 ? m0 : m1;
    const int count = __popcll(m);
    int outside = 0;
    auto slot = [&](int p) {
      const int id = A.table[(size_t)b * c.max_pages + (p >> A.shift)];
      if (id < 0 || id >= c.n_pages) outside = 1;
      return outside ? 0 : id * c.page + (p & (c.page - 1));
    };
#pragma unroll
    for (int node = tid; node < LBX_ATTN_MAX_NODES; node += 32) {
      if (!(m >> node & 1)) continue;
      const int i = __popcll(m & ((1ull << node) - 1));
      place[i] = slot(ctx + i), from[i] = slot(ctx + node);
    }
    outside = __any_sync(0xffffffffu, outside);
    if (tid == 0) {
      len = outside ? 0 : count;
      if (outside && A.status) *A.status = LBX_EINVAL;
      if (lb < c.Bq && part == 0) A.ctx_out[b] = ctx + count;
    }
  }
  __syncthreads();
  const int end = len, col = part * kThreads + tid;
  if (col >= 2 * A.cols) return;
  uint4 *base = (col < A.cols ? A.k + col : A.v + col - A.cols) +
                (size_t)l * c.n_pages * c.page * A.cols;
#pragma unroll 1
  for (int i0 = 1; i0 < end; i0 += kFly) {
    uint4 x[kFly];
#pragma unroll
    for (int i = 0; i < kFly; ++i)
      if (i0 + i < end) x[i] = base[(size_t)from[i0 + i] * A.cols];
#pragma unroll
    for (int i = 0; i < kFly; ++i)
      if (i0 + i < end && place[i0 + i] != from[i0 + i]) base[(size_t)place[i0 + i] * A.cols] = x[i];
  }
}

}  // namespace
}  // namespace paged
}  // namespace lbx

extern "C" int lbx_page_commit(const lbx_page_cfg *c, const int32_t *start,
                               const int32_t *ctx_len, const int32_t *block_table,
                               const int32_t *parent, const int32_t *accepted, uint16_t *k_pages,
                               uint16_t *v_pages, int32_t *ctx_out, int32_t *d_status,
                               cudaStream_t stream) {
  using namespace lbx::paged;
  if (!cfg_ok(c)) return LBX_EINVAL;
  for (const int32_t *p : {start, ctx_len, block_table, parent, accepted, (const int32_t *)ctx_out})
    if (!aligned_to(p, 4)) return LBX_EINVAL;
  if (!aligned_to(k_pages, 16) || !aligned_to(v_pages, 16) || (d_status && !aligned_to(d_status, 4)))
    return LBX_EINVAL;
  const size_t per = (size_t)c->Bq * 4;
  if (!all_apart({{ctx_out, per}}, {{start, per + 4}, {ctx_len, per}, {accepted, per},
                                    {block_table, per * c->max_pages}, {parent, (size_t)c->M * 4}}))
    return LBX_EINVAL;
  CommitArgs A = {*c, 0, c->Hkv * c->dh / 8, 0, start, ctx_len, block_table, parent, accepted,
                  reinterpret_cast<uint4 *>(k_pages), reinterpret_cast<uint4 *>(v_pages), ctx_out,
                  d_status};
  while (1 << A.shift < c->page) ++A.shift;
  A.parts = (2 * A.cols + kThreads - 1) / kThreads;
  const long long grid = (long long)c->L * c->Bq * A.parts;
  if (grid > 0x7fffffffLL) return LBX_EINVAL;
  page_commit_kernel<<<(unsigned)grid, kThreads, 0, stream>>>(A);
  return cudaGetLastError() == cudaSuccess ? LBX_OK : LBX_ECUDA;
}
