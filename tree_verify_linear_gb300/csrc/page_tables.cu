// page_tables.cu -- block tables and slot maps of a step from the requests'
// lengths: lbx_page_tables.
//
// Every CTA makes the same running sums over the requests (new tokens, pages to
// give back, pages to take) in shared memory, and with them the same verdict on
// the batch; then each takes its share of the requests, whose pages it moves, and
// of the rows, whose request it finds by a binary search.  No CTA reads what another
// one writes: a page that is given back and taken again in one call is read from
// the table of the request that gives it, not from the stack.
#include "cache_walk.cuh"
#include "page_common.cuh"

namespace lbx {
namespace paged {
namespace {

constexpr int kThreads = 512;
constexpr int kMost = LBX_PAGE_MAX_REQUESTS;
constexpr int kPer = kMost / kThreads;  // requests per thread, at most
constexpr int kRowsPerCta = 512;        // rows of a CTA's share

struct TableArgs {
  int Bq, M, page, shift, n_pages, max_pages;
  const int32_t *ctx_len, *new_len, *held, *n_free;
  int32_t *table, *stack, *held_out, *n_free_out, *start, *slot, *pos, *status;
};

// Inclusive sums over the block's threads, three at a time; totals in `all`.
__device__ __forceinline__ void scan3(long long (&v)[3], long long (&all)[3],
                                      long long (*warps)[3]) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int k = 0; k < 3; ++k)
#pragma unroll
    for (int s = 1; s < 32; s *= 2) {
      const long long o = __shfl_up_sync(0xffffffffu, v[k], s);
      if (lane >= s) v[k] += o;
    }
  if (lane == 31)
    for (int k = 0; k < 3; ++k) warps[warp][k] = v[k];
  __syncthreads();
#pragma unroll
  for (int k = 0; k < 3; ++k) {
    long long before = 0;
    all[k] = 0;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) {
      if (w < warp) before += warps[w][k];
      all[k] += warps[w][k];
    }
    v[k] += before;
  }
}

__global__ void __launch_bounds__(kThreads) page_tables_kernel(const TableArgs A) {
  __shared__ int first[kMost], back[kMost], taken[kMost];  // before each request
  __shared__ long long warps[kThreads / 32][3];
  const int tid = threadIdx.x;
  const int n_free = A.n_free[0];
  const int per = (A.Bq + kThreads - 1) / kThreads;

  int bad = n_free < 0 || n_free > A.n_pages;
  long long own[kPer][3], sum[3] = {0, 0, 0}, all[3];
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    own[i][0] = own[i][1] = own[i][2] = 0;
    const int b = tid * per + i;
    if (i >= per || b >= A.Bq) continue;
    const int ctx = A.ctx_len[b], n = A.new_len[b], h = A.held[b];
    if (ctx < 0 || n < 0 || h < 0 || h > A.max_pages ||
        (long long)ctx + n > (long long)A.max_pages * A.page) {
      bad = 1;
      continue;
    }
    const int want = (ctx + n + A.page - 1) >> A.shift;
    own[i][0] = n, own[i][1] = h > want ? h - want : 0, own[i][2] = want > h ? want - h : 0;
    for (int k = 0; k < 3; ++k) sum[k] += own[i][k];
  }
  long long upto[3] = {sum[0], sum[1], sum[2]};
  scan3(upto, all, warps);
  bad |= all[0] > A.M || n_free + all[1] > A.n_pages;
  bad = __syncthreads_or(bad);
  const bool short_of = n_free + all[1] < all[2];
  if (bad || short_of) {
    if (tid == 0 && A.status) *A.status = bad ? LBX_EINVAL : LBX_EPAGES;
    return;
  }
  const int rows = (int)all[0], top = n_free + (int)all[1];
#pragma unroll
  for (int k = 0; k < 3; ++k) upto[k] -= sum[k];
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int b = tid * per + i;
    if (i >= per || b >= A.Bq) continue;
    first[b] = (int)upto[0], back[b] = (int)upto[1], taken[b] = (int)upto[2];
    for (int k = 0; k < 3; ++k) upto[k] += own[i][k];
  }
  __syncthreads();

  // the last request whose sum is at most x
  auto find = [&](const int *sums, int x) {
    int a = 0, z = A.Bq - 1;
    while (a < z) {
      const int h = (a + z + 1) >> 1;
      if (sums[h] <= x) a = h;
      else z = h - 1;
    }
    return a;
  };
  auto wanted = [&](int b) { return (A.ctx_len[b] + A.new_len[b] + A.page - 1) >> A.shift; };
  // page j of request b, as this call leaves it
  auto page_of = [&](int b, int held, int j) {
    if (j < held) return A.table[(size_t)b * A.max_pages + j];
    const int at = top - 1 - taken[b] - (j - held);
    if (at < n_free) return A.stack[at];
    const int g = find(back, at - n_free);
    return A.table[(size_t)g * A.max_pages + wanted(g) + at - n_free - back[g]];
  };

  const int warp = tid >> 5, lane = tid & 31;
#pragma unroll 1
  for (int b = blockIdx.x * (kThreads / 32) + warp; b < A.Bq; b += gridDim.x * (kThreads / 32)) {
    const int held = A.held[b], want = wanted(b);
    int32_t *row = A.table + (size_t)b * A.max_pages;
#pragma unroll 1
    for (int j = want + lane; j < held; j += 32) A.stack[n_free + back[b] + j - want] = row[j];
#pragma unroll 1
    for (int j = held + lane; j < want; j += 32) row[j] = page_of(b, held, j);
    if (lane == 0) A.held_out[b] = want, A.start[b] = first[b];
  }
  if (blockIdx.x == 0 && tid == 0)
    A.start[A.Bq] = rows, A.n_free_out[0] = top - (int)all[2];

  int outside = 0;
#pragma unroll 1
  for (uint32_t i = blockIdx.x * kThreads + tid; i < (uint32_t)A.M; i += gridDim.x * kThreads) {
    const int r = (int)i;
    int slot = -1, p = -1;
    if (r < rows) {
      const int b = find(first, r);
      p = A.ctx_len[b] + r - first[b];
      const int id = page_of(b, A.held[b], p >> A.shift);
      if (id >= 0 && id < A.n_pages) slot = id * A.page + (p & (A.page - 1));
      else outside = 1;
    }
    A.slot[r] = slot, A.pos[r] = p;
  }
  if (outside && A.status) *A.status = LBX_EINVAL;
}

}  // namespace
}  // namespace paged
}  // namespace lbx

extern "C" int lbx_page_tables(const lbx_page_cfg *c, const int32_t *ctx_len,
                               const int32_t *new_len, const int32_t *held, const int32_t *n_free,
                               int32_t *block_table, int32_t *free_list, int32_t *held_out,
                               int32_t *n_free_out, int32_t *start, int32_t *slot, int32_t *pos,
                               int32_t *d_status, cudaStream_t stream) {
  using namespace lbx::paged;
  if (!cfg_ok(c)) return LBX_EINVAL;
  for (const void *p : {ctx_len, new_len, held, n_free, (const int32_t *)block_table,
                        (const int32_t *)free_list, (const int32_t *)held_out,
                        (const int32_t *)n_free_out, (const int32_t *)start,
                        (const int32_t *)slot, (const int32_t *)pos})
    if (!aligned_to(p, 4)) return LBX_EINVAL;
  if (d_status && !aligned_to(d_status, 4)) return LBX_EINVAL;
  // CTAs read the inputs while others write the outputs
  const size_t per = (size_t)c->Bq * 4, rows = (size_t)c->M * 4;
  if (!all_apart({{held_out, per}, {n_free_out, 4}, {start, per + 4}, {slot, rows}, {pos, rows},
                  {block_table, per * c->max_pages}, {free_list, (size_t)c->n_pages * 4}},
                 {{ctx_len, per}, {new_len, per}, {held, per}, {n_free, 4}}))
    return LBX_EINVAL;
  int shift = 0;
  while (1 << shift < c->page) ++shift;
  const TableArgs A = {c->Bq, c->M, c->page, shift, c->n_pages, c->max_pages, ctx_len, new_len,
                       held, n_free, block_table, free_list, held_out, n_free_out, start, slot,
                       pos, d_status};
  const int by_rows = (int)(((long long)c->M + kRowsPerCta - 1) / kRowsPerCta);
  const int by_requests = (c->Bq + 63) / 64, nsm = lbx::cache::grid_limit();
  if (nsm < 1) return LBX_ECUDA;
  int grid = by_rows > by_requests ? by_rows : by_requests;
  if (grid > nsm) grid = nsm;
  page_tables_kernel<<<grid, kThreads, 0, stream>>>(A);
  return cudaGetLastError() == cudaSuccess ? LBX_OK : LBX_ECUDA;
}
