// Host check of csrc/attn_index.h against brute force: every sequence, page and key-tile decision of the attention
// kernels, over random and hostile inputs.  Prints "ok" or the first difference.
#include <stdio.h>
#include <stdlib.h>

#include <set>
#include <vector>

#include "attn_index.h"

using namespace moe;

static int rnd(int lo, int hi) { return lo + (int)((unsigned)rand() % (unsigned)(hi - lo + 1)); }

#define CHECK(cond, ...)                  \
  do {                                    \
    if (!(cond)) {                        \
      printf("line %d: ", __LINE__);      \
      printf(__VA_ARGS__);                \
      return 1;                           \
    }                                     \
  } while (0)

int main() {
  srand(7);
  // sequences: whatever the arrays hold, rows stay inside [0, T] and lengths inside [0, cap]
  const int hostile[] = {INT32_MIN, -5, -1, 0, 1, 7, 64, 65, 1 << 30, INT32_MAX};
  for (int s : hostile)
    for (int e : hostile)
      for (int n : hostile) {
        const int32_t qs[2] = {s, e}, kv[1] = {n};
        const int T = 64, cap = 128;
        const SeqView v = seq_view(qs, kv, 0, 0, T, cap);
        CHECK(v.q0 >= 0 && v.m >= 0 && v.q0 + v.m <= T && v.n >= 0 && v.n <= cap, "seq %d %d %d\n", s, e, n);
        const bool good = s >= 0 && e >= s && e <= T && n >= 0 && n <= cap;
        CHECK(v.bad == !good, "bad flag %d %d %d\n", s, e, n);
        if (good) CHECK(v.q0 == s && v.m == e - s && v.n == n, "values %d %d %d\n", s, e, n);
      }
  // pages: a row inside the cache or -1, also far beyond 32 bits of elements
  for (int i = 0; i < 200000; ++i) {
    const int log_ps = rnd(4, 7), ps = 1 << log_ps, heads = rnd(1, 9), n_pages = rnd(1, 40), p = rnd(0, 4 * ps - 1);
    int32_t table[4];
    for (int32_t &t : table) t = rnd(0, 3) ? rnd(0, n_pages - 1) : hostile[rnd(0, 9)];
    const int64_t r = cache_row(table, p, log_ps, n_pages, heads);
    const int32_t page = table[p / ps];
    if (page < 0 || page >= n_pages) {
      CHECK(r == -1, "bad page %d taken\n", page);
    } else {
      CHECK(r == (int64_t)page * heads * ps + p % ps, "row of page %d\n", page);
      CHECK(r + (int64_t)(heads - 1) * ps < (int64_t)n_pages * heads * ps, "row outside\n");
    }
  }
  // key tiles
  for (int i = 0; i < 300000; ++i) {
    const int log_bk = rnd(0, 1) ? 6 : 3, bk = 1 << log_bk;
    const int n = rnd(0, rnd(0, 1) ? 40 : 700);
    const int p0 = rnd(-20, n), p1 = p0 + rnd(0, 30);
    const int window = rnd(0, 2) ? rnd(1, 300) : 0, sinks = rnd(0, 1) ? rnd(0, 90) : 0;
    const int q1 = p1 < n ? p1 : n - 1;  // a query stands at one of the n tokens
    if (q1 < p0) continue;
    const TileRange r = tile_range(p0, q1, n, window, sinks, log_bk);
    std::set<int> got;
    for (int t = 0; t < r.count; ++t) {
      const int x = tile_of(r, t);
      CHECK(x >= 0 && x * bk < n && got.insert(x).second, "tile %d twice or outside\n", x);
    }
    for (int t = 0; t * bk < n; ++t) {
      bool any = false, all = true;
      for (int p = p0; p <= q1; ++p)
        for (int j = t * bk; j < (t + 1) * bk; ++j) {
          const bool seen = p >= 0 && j <= p && j < n && (window == 0 || p - j < window || j < sinks);
          CHECK(key_seen(p, j, n, window, sinks) == (seen), "seen %d %d\n", p, j);
          any |= seen;
          all &= seen;
        }
      CHECK(!any || got.count(t), "tile %d missed: p %d..%d n %d w %d s %d\n", t, p0, q1, n, window, sinks);
      CHECK(tile_full(p0, q1, t * bk, bk, n, window, sinks) <= all, "tile %d called full\n", t);
      // a key that neither the first nor the last query could see is seen by none between
      for (int j = t * bk; j < (t + 1) * bk; ++j) {
        const bool ok = j <= q1 && j < n && (window <= 0 || p0 - j < window || j < sinks);
        for (int p = p0; p <= q1; ++p) CHECK(ok || !key_seen(p, j, n, window, sinks), "cleared key %d\n", j);
      }
    }
  }
  // the largest positions: nothing overflows
  const int big = 1 << 30;
  for (int w : {0, 1, 4096, INT32_MAX})
    for (int s : {0, 4, INT32_MAX}) {
      const TileRange r = tile_range(big - 8, big - 1, big, w, s, 6);
      CHECK(r.count >= 1 && tile_of(r, r.count - 1) == (big - 1) >> 6, "large %d %d\n", w, s);
    }
  printf("ok\n");
  return 0;
}
