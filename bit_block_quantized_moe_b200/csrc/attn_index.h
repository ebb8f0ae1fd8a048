// Index arithmetic of the attention kernels: sequences, pages, and the key tiles that a tile of queries sees.
// Plain C++ (host and device), so that a host program can run the same code over every bad input.
#pragma once

#include <stddef.h>
#include <stdint.h>

#ifdef __CUDACC__
#define MOE_HD __host__ __device__ __forceinline__
#else
#define MOE_HD inline
#endif

namespace moe {

// One sequence of a call: rows q0 .. q0 + m - 1 are its new tokens, n its tokens in all; new token i stands at
// position n - m + i.
struct SeqView {
  int q0, m, n;
  bool bad;  // a start, end or length out of range: made empty or of length 0
};

// q_start null: `per` rows each.  cap = max_pages * page_size (below 2^31).
MOE_HD SeqView seq_view(const int32_t *q_start, const int32_t *kv_len, int b, int per, int T, int cap) {
  SeqView v;
  v.bad = false;
  if (q_start) {
    const int s = q_start[b], e = q_start[b + 1];
    v.q0 = s;
    v.m = e - s;
    if (s < 0 || e < s || e > T) {
      v.q0 = v.m = 0;
      v.bad = true;
    }
  } else {
    v.q0 = b * per;
    v.m = per;
  }
  v.n = kv_len[b];
  if (v.n < 0 || v.n > cap) {
    v.n = 0;
    v.bad = true;
  }
  return v;
}

// The cache row (units of head_dim elements, head 0) of position p >= 0 in the sequence's table row, or -1 when its
// page is outside the cache.  Rows of head h are h * page_size further.  log_ps: log2(page_size).
MOE_HD int64_t cache_row(const int32_t *table_row, int p, int log_ps, int n_pages, int n_kv_heads) {
  const int32_t page = table_row[p >> log_ps];
  if (page < 0 || page >= n_pages) return -1;
  return (((int64_t)page * n_kv_heads) << log_ps) + (p & ((1 << log_ps) - 1));
}

// The key tiles (of 2^log_bk keys) that queries at positions p0 .. p1 see among n keys: first the tiles of the
// sinks, then a run of tiles from `first`.  Virtual tile t is tile t for t < sink_tiles, else first + t - sink_tiles.
struct TileRange {
  int sink_tiles, first, count;  // count = sink tiles + tiles of the run
};

MOE_HD TileRange tile_range(int p0, int p1, int n, int window, int n_sinks, int log_bk) {
  TileRange r;
  const int bk = 1 << log_bk;
  const int hi = p1 + 1 < n ? p1 + 1 : n;  // keys [0, hi) at most
  r.sink_tiles = r.first = r.count = 0;
  if (hi <= 0) return r;
  int lo = 0;
  if (window > 0 && p0 >= window) lo = p0 - window + 1;
  r.first = lo >> log_bk;
  const int end = (hi + bk - 1) >> log_bk;
  if (window > 0 && n_sinks > 0) {
    const int s = n_sinks < hi ? n_sinks : hi;
    const int st = (s + bk - 1) >> log_bk;
    r.sink_tiles = st < r.first ? st : r.first;
  }
  r.count = r.sink_tiles + (end > r.first ? end - r.first : 0);
  return r;
}

MOE_HD int tile_of(const TileRange &r, int t) { return t < r.sink_tiles ? t : r.first + (t - r.sink_tiles); }

// Whether the query at position i sees key j (of n).
MOE_HD bool key_seen(int i, int j, int n, int window, int n_sinks) {
  return j <= i && j < n && (window <= 0 || i - j < window || j < n_sinks);
}

// Whether every query at positions p0 .. p1 (p0 >= 0) sees all keys j0 .. j0 + bk - 1.
MOE_HD bool tile_full(int p0, int p1, int j0, int bk, int n, int window, int n_sinks) {
  if (p0 < 0 || j0 + bk - 1 > p0 || j0 + bk > n) return false;
  return window <= 0 || p1 - j0 < window || j0 + bk <= n_sinks;
}

}  // namespace moe
