// The cut's arithmetic against walks over everything (compiled and run by test_attention_cut.py).
#include <algorithm>
#include <cstdio>
#include <cstdlib>
#include <random>
#include <vector>

#include "mk_attn_cut.h"

using namespace mk_cut;

static std::mt19937 rng(1);
static int draw(int lo, int hi) { return lo + (int)(rng() % (unsigned)(hi - lo + 1)); }
static int spread(int hi) { return draw(0, 1 << draw(0, 30)) % (hi + 1); }
#define CHECK(c, ...)                                     \
  do {                                                    \
    if (!(c)) {                                           \
      std::printf("line %d: %s", __LINE__, #c);           \
      std::printf(" " __VA_ARGS__);                       \
      std::printf("\n");                                  \
      std::exit(1);                                       \
    }                                                     \
  } while (0)

// pairs_before against the sum over the blocks
static void blocks() {
  const int G[] = {1, 2, 3, 5, 6, 7, 8, 16, 24, 33, 64};
  for (int k = 0; k < 20000; ++k) {
    const int TB = kTile / G[draw(0, 10)], T = spread(k % 50 ? 3000 : 1 << 20);
    const int len = k % 3 ? T + spread(1 << 18) : spread(2 * T + 1);
    const int start = spread(len) / 16 * 16, nb = pair_blocks(T, TB);
    long long cost = 0;
    for (int j = 0; j <= nb; ++j) {
      if (nb < 200 || j == nb || draw(0, 50) == 0)
        CHECK(pairs_before(start, len, T, TB, j) == (int)cost, "start %d len %d T %d TB %d j %d", start,
              len, T, TB, j);
      if (j < nb) cost += item_cost(0, key_tiles(start, block_end(len, T, TB, j)));
      if (cost > (1 << 30)) break; // refused by the host
    }
  }
}

struct Item {
  int begin, nt;
};

// Every tile has one owner; the workers from the first tile's to the last one's follow one
// another without a gap, and those are where worker_of says; only an owner of a first tile may
// own nothing of an item's beginning.
static void line(const std::vector<int> &pairs, const std::vector<int> &singles, int n_cta) {
  std::vector<Item> items[2];
  int length[2] = {0, 0};
  for (int l = 0; l < 2; ++l)
    for (int nt : l ? singles : pairs) {
      if (nt) items[l].push_back({length[l], nt});
      length[l] += item_cost(l, nt);
    }
  const int total = length[0] + length[1], n = active_ctas(total, n_cta);
  if (!total) return;
  int reach[2] = {0, 0};
  std::vector<std::vector<int>> owner[2];
  for (int l = 0; l < 2; ++l)
    for (auto &i : items[l]) owner[l].push_back(std::vector<int>(i.nt, -1));
  for (int c = 0; c < n; ++c)
    for (int l = 0; l < 2; ++l)
      for (int s = 0; s < 2; ++s) {
        const Share h = share_of(c, s, total, length[0], n);
        int x = l ? h.x1 : h.x, end = l ? h.end1 : h.end;
        if (l == 0 && s == 1) continue; // the same pairs as stream 0
        CHECK(x == reach[l], "shares leave a gap");
        reach[l] = end;
        size_t i = 0;
        while (x < end) {
          while (i + 1 < items[l].size() && items[l][i + 1].begin <= x) ++i;
          const Range r = piece_range(l, items[l][i].begin, items[l][i].nt, x, end);
          CHECK(r.next > x && r.next <= end, "x %d next %d end %d", x, r.next, end);
          CHECK(r.t0 >= 0 && r.t0 + r.n <= items[l][i].nt, "tiles");
          for (int t = r.t0; t < r.t0 + r.n; ++t) {
            CHECK(owner[l][i][t] == -1, "a tile with two owners");
            owner[l][i][t] = l ? 2 * c + s : c;
          }
          x = r.next;
        }
      }
  for (int l = 0; l < 2; ++l) {
    CHECK(reach[l] == length[l], "shares end early");
    for (size_t i = 0; i < items[l].size(); ++i) {
      const std::vector<int> &o = owner[l][i];
      const int at = items[l][i].begin + fixed_cost(l);
      CHECK(o[0] == worker_of(l, at, total, length[0], n), "first worker");
      CHECK(o.back() == worker_of(l, at + (items[l][i].nt - 1) * tile_cost(l), total, length[0], n),
            "last worker");
      for (size_t t = 0; t < o.size(); ++t)
        CHECK(o[t] >= 0 && (t == 0 || o[t] == o[t - 1] || o[t] == o[t - 1] + 1), "worker %d behind %d",
              o[t], o[t ? t - 1 : 0]);
    }
  }
}

int main() {
  blocks();
  for (int k = 0; k < 60000; ++k) {
    const int many[] = {0, 0, 1, 2, 5, 30}, longest[] = {1, 2, 5, 60, 2000};
    std::vector<int> p(many[draw(0, 5)]), s(many[draw(0, 5)]);
    const int hi = longest[draw(0, 4)], hs = longest[draw(0, 4)];
    for (int &x : p) x = draw(0, hi);
    for (int &x : s) x = draw(0, hs);
    const int ctas[] = {1, 2, 3, 16, 152};
    line(p, s, ctas[draw(0, 4)]);
  }
  // lines of every small length, and the longest that a call can have
  for (int a = 0; a < 60; ++a)
    for (int b = 0; b < 60; ++b)
      for (int c : {1, 5, 152}) line({a}, {b, b / 2}, c);
  line({(1 << 29) / kPairTile}, {(1 << 28) / kSingleTile, 100}, 152);
  std::printf("ok\n");
}
