// Host check of page_walk.cuh: for random batches, the ranges of all CTAs together cover
// every block of every tile once, pieces agree on their number, order and owner, and
// entries_upto is the sum it stands for.  Prints "ok" or the first fault.
#include <array>
#include <cstdio>
#include <cstdlib>
#include <map>
#include <tuple>
#include <vector>

#include "page_walk.cuh"

using namespace lbx::paged;

#define CHECK(x)                                                 \
  do {                                                           \
    if (!(x)) {                                                  \
      std::printf("case %d: %s\n", it, #x);                      \
      return 1;                                                  \
    }                                                            \
  } while (0)

int main() {
  std::srand(1);
  for (int it = 0; it < 6000; ++it) {
    const int G = 1 + std::rand() % (std::rand() % 3 ? 8 : 128);
    const bool tree = std::rand() % 3 == 0;
    const Shape s = shape_of(G, it % 2 ? 2 : 4, tree);
    const int B = 1 + std::rand() % 6, LH = 1 + std::rand() % 5, ctas = 1 + std::rand() % 160;
    std::vector<int> ctx(B), n(B);
    std::vector<i64> per(B);
    i64 all = 0;
    for (int b = 0; b < B; ++b) {
      ctx[b] = std::rand() % (std::rand() % 2 ? 3000 : 20);
      n[b] = std::rand() % 4 == 0 ? 0 : 1 + std::rand() % (tree ? 64 : std::rand() % 2 ? 2000 : 3);
      i64 e = 0;
      for (int t = 0; t < tiles_of(s, n[b]); ++t) {
        CHECK(entries_upto(s, ctx[b], n[b], t) == e);
        e += kLead + blocks_of(s, ctx[b], n[b], t);
      }
      CHECK(entries_of(s, ctx[b], n[b]) == e);
      per[b] = e, all += e;
    }
    if (all == 0) continue;
    const Cut c = cut_of(all * LH, ctas);
    CHECK(c.n >= 1 && c.n <= ctas);
    std::map<std::tuple<int, int, int>, std::vector<std::array<int, 5>>> got;
    for (int me = 0; me < c.n; ++me) {
      const i64 x = c.at(me);
      int lh = (int)(x / all), b = 0, t = 0;
      i64 y = x % all;
      while (y >= per[b]) y -= per[b++];
      for (int u = 1; u < tiles_of(s, n[b]); ++u)
        if (entries_upto(s, ctx[b], n[b], u) <= y) t = u;
      const i64 off = y - entries_upto(s, ctx[b], n[b], t);
      i64 X = x - off;
      auto step = [&]() {
        X += kLead + blocks_of(s, ctx[b], n[b], t++);
        while (lh < LH && t >= tiles_of(s, n[b])) {
          t = 0;
          if (++b == B) b = 0, ++lh;
        }
      };
      if (off >= kLead + kLeast && off > kLead + blocks_of(s, ctx[b], n[b], t) - kLeast) step();
      while (lh < LH) {
        Piece p;
        if (!piece_of(c, me, c.at(me), c.at(me + 1), X, blocks_of(s, ctx[b], n[b], t), p)) break;
        got[{lh, b, t}].push_back({p.blk0, p.blk1, p.pieces, p.mine, p.owner});
        if (p.last) break;
        step();
      }
    }
    for (int lh = 0; lh < LH; ++lh)
      for (int b = 0; b < B; ++b)
        for (int t = 0; t < tiles_of(s, n[b]); ++t) {
          const auto &v = got[{lh, b, t}];
          int at = 0, k = 0;
          for (const auto &p : v) {
            CHECK(p[0] == at && p[1] > p[0] && p[2] == (int)v.size() && p[3] == k && p[4] == v[0][4]);
            CHECK(v.size() == 1 || p[1] - p[0] >= kLeast);
            at = p[1], ++k;
          }
          CHECK(at == blocks_of(s, ctx[b], n[b], t));
        }
  }
  std::printf("ok\n");
  return 0;
}
