// Device check of find_begin: for random batches, where every CTA's range of the list begins
// is where walking the requests and tiles one by one comes to.  Prints "ok" or the first fault.
#include <cstdio>
#include <cstdlib>
#include <vector>

#include "page_attn.cuh"

using namespace lbx::paged;

struct Found {
  int bad, more, n, lh, b, t;
  i64 from, X;
};

__global__ void __launch_bounds__(kThreads) find(const PageArgs A, Found *out) {
  __shared__ i64 sums[2 * (kThreads / 32)];
  int units = 0;
  Window win;
  win.load(A, 0);
  const int bad = check_batch(A, sums, units);
  if (threadIdx.x / 32 != 9) return;
  Begin g = {};
  const bool more = !bad && find_begin(A, blockIdx.x, gridDim.x, sums, win, g);
  if (threadIdx.x % 32 == 0) out[blockIdx.x] = {bad, more, g.cut.n, g.lh, g.b, g.t, g.from, g.X};
}

#define CHECK(x)                                                                  \
  do {                                                                            \
    if (!(x)) {                                                                   \
      std::printf("case %d, range %d of %d: %s\n", it, me, c.n, #x);              \
      return 1;                                                                   \
    }                                                                             \
  } while (0)

int main() {
  std::srand(3);
  constexpr int kMost = LBX_PAGE_MAX_REQUESTS, kRowsMost = 1 << 17, kCtasMost = 160;
  int *start, *ctx, *parent;
  Found *out;
  if (cudaMallocManaged(&start, (kMost + 1) * 4) != cudaSuccess || cudaMallocManaged(&ctx, kMost * 4) != cudaSuccess ||
      cudaMallocManaged(&parent, kRowsMost * 4) != cudaSuccess ||
      cudaMallocManaged(&out, kCtasMost * sizeof(Found)) != cudaSuccess)
    return std::printf("no memory\n"), 1;
  for (int it = 0; it < 400; ++it) {
    const bool tree = std::rand() % 3 == 0;
    PageArgs A = {};
    A.G = 1 + std::rand() % (std::rand() % 3 ? 8 : 128);
    A.shape = shape_of(A.G, it % 2 ? 2 : 4, tree);
    const int most = it % 5 == 0 ? kMost : it % 5 == 1 ? 1 : 400;
    const int B = it % 5 == 0 ? kMost - std::rand() % 300 : 1 + std::rand() % most, ctas = 1 + std::rand() % kCtasMost;
    const int longest = tree ? 64 : B > 400 ? 60 : B > 40 ? 300 : 3000;
    std::vector<i64> per(B);
    i64 all = 0;
    start[0] = 0;
    for (int b = 0; b < B; ++b) {
      const int n = std::rand() % 4 == 0 ? 0 : 1 + std::rand() % (std::rand() % 2 ? longest : 3);
      ctx[b] = std::rand() % (std::rand() % 2 ? 20000 : 20);
      start[b + 1] = start[b] + n;
      for (int i = 0; i < n; ++i) parent[start[b] + i] = i - 1;
      for (int t = 0; t < tiles_of(A.shape, n); ++t) per[b] += kLead + blocks_of(A.shape, ctx[b], n, t);
      all += per[b];
    }
    A.c.L = 1 + std::rand() % 3, A.c.Hkv = 1 + std::rand() % 4, A.c.Bq = B;
    A.c.M = start[B] > 0 ? start[B] : 1, A.c.max_pages = 1 << 22, A.c.page = 16;
    A.start = start, A.ctx_len = ctx, A.parent = tree ? parent : nullptr;
    find<<<ctas, kThreads>>>(A, out);
    if (cudaDeviceSynchronize() != cudaSuccess) return std::printf("launch\n"), 1;
    const Cut c = cut_of(all * A.c.L * A.c.Hkv, ctas);
    for (int me = 0; me < ctas; ++me) {
      const Found &f = out[me];
      CHECK(!f.bad);
      CHECK(f.more == (all > 0 && me < c.n));
      if (!f.more) continue;
      const i64 x = c.at(me);
      CHECK(f.n == c.n && f.from == x);
      const int lh = (int)(x / all);
      i64 at = lh * all;
      int b = 0, t = 0;
      while (at + per[b] <= x) at += per[b++];
      const int n = start[b + 1] - start[b];
      for (; at + kLead + blocks_of(A.shape, ctx[b], n, t) <= x; ++t) at += kLead + blocks_of(A.shape, ctx[b], n, t);
      CHECK(f.lh == lh && f.b == b && f.t == t && f.X == at);
    }
  }
  std::printf("ok\n");
  return 0;
}
