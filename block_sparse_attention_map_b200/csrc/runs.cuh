// The list of 128-key tiles that the attention and the weighing of a paged cache
// walk, cut into equal runs, one a CTA; read from the device's lengths, so that a
// captured launch follows them.
#pragma once

#include "serving.cuh"

namespace bsa {

// Sequence b has H_kv * groups(b) items of tiles(b) key tiles each, a row group
// being ROWS of its n * G rows (kAllRows: one group, even of no row); the list is
// all of them in order (b, kv head, row group, tile).
constexpr int kAllRows = 0;

template <int ROWS>
struct Seq {
  int len, n, tiles, groups;
  __device__ __forceinline__ int64_t work(int H_kv) const { return static_cast<int64_t>(H_kv) * groups * tiles; }
};

template <int ROWS>
__device__ __forceinline__ Seq<ROWS> sequence(const CacheView &c, const TokenView &t, int b, bool report) {
  Seq<ROWS> s;
  s.len = clamped_length(c, b, report);
  s.n = clamped_new(c, t, b, s.len, report);
  s.tiles = (s.len + s.n + kTile - 1) / kTile;
  s.groups = ROWS == kAllRows ? min(s.tiles, 1) : (s.n * t.G + max(ROWS, 1) - 1) / max(ROWS, 1);
  return s;
}

__device__ __forceinline__ int64_t run_start(int64_t total, int cta, int ctas) { return total * cta / ctas; }

struct RunStart {
  int b, item, tile, count;  // count: key tiles of the run
};

// Sum of work over the sequences, and the sequence that holds position `at`, by
// one warp.
template <int ROWS>
__device__ __forceinline__ int64_t total_work(const CacheView &c, const TokenView &t, int lane, bool report) {
  int64_t sum = 0;
  for (int b0 = 0; b0 < c.B; b0 += 32)
    if (b0 + lane < c.B) sum += sequence<ROWS>(c, t, b0 + lane, report).work(c.H_kv);
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
  return sum;
}

template <int ROWS>
__device__ __forceinline__ RunStart find_start(const CacheView &c, const TokenView &t, int64_t at, int count, int lane) {
  RunStart r{0, 0, 0, count};
  int64_t base = 0;
  for (int b0 = 0; b0 < c.B; b0 += 32) {
    Seq<ROWS> s{0, 0, 0, 0};
    if (b0 + lane < c.B) s = sequence<ROWS>(c, t, b0 + lane, false);
    const int64_t w = s.work(c.H_kv);
    int64_t incl = w;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int64_t o = __shfl_up_sync(0xffffffffu, incl, d);
      if (lane >= d) incl += o;
    }
    const bool here = w > 0 && at >= base + incl - w && at < base + incl;
    const uint32_t who = __ballot_sync(0xffffffffu, here);
    if (who != 0u) {
      const int src = __ffs(who) - 1;
      const int64_t off = at - (base + incl - w);
      const int item = here ? static_cast<int>(off / s.tiles) : 0, tile = here ? static_cast<int>(off % s.tiles) : 0;
      r.b = b0 + src;
      r.item = __shfl_sync(0xffffffffu, item, src);
      r.tile = __shfl_sync(0xffffffffu, tile, src);
      return r;
    }
    base += __shfl_sync(0xffffffffu, incl, 31);
  }
  r.count = 0;
  return r;
}

// One CTA's run, piece by piece (a piece: consecutive key tiles of one item).
template <int ROWS>
struct Walk {
  int b, item, tile, left, index;
  Seq<ROWS> s;
  int hk, rg, t0, t1;  // the piece: kv head, row group, key tiles [t0, t1)
  bool whole;
  __device__ __forceinline__ Walk(const CacheView &c, const TokenView &t, const RunStart &r)
      : b(r.b), item(r.item), tile(r.tile), left(r.count), index(-1) {
    if (left > 0) s = sequence<ROWS>(c, t, b, false);
  }
  __device__ __forceinline__ bool next(const CacheView &c, const TokenView &t) {
    if (left <= 0) return false;
    while (item >= c.H_kv * s.groups) {
      item = 0;
      if (++b >= c.B) return false;  // never, with lengths that stay as they are
      s = sequence<ROWS>(c, t, b, false);
    }
    hk = item / s.groups;
    rg = item % s.groups;
    t0 = tile;
    t1 = min(s.tiles, tile + left);
    whole = t0 == 0 && t1 == s.tiles;
    left -= t1 - t0;
    tile = 0;
    ++item;
    ++index;
    return true;
  }
};

constexpr uint64_t kWaitLimitNs = 2000000000ull;

// Bounded wait that ignores the abort flag: used only to drain copies already
// in flight before the CTA exits.
__device__ __forceinline__ void drain_wait(uint64_t *bar, uint32_t parity) {
  const uint32_t a = smem_u32(bar);
  const uint64_t t0 = globaltimer_ns();
  while (!mbar_try_wait(a, parity)) {
    if (globaltimer_ns() - t0 > 200000000ull) return;
  }
}

// The page of the box of key tile `t` that starts `first` slots into it: n_pages (a
// page past the end, which reads as zeros) where no slot of the box is in use.
template <int ROWS>
__device__ __forceinline__ int box_page(const CacheView &c, const Walk<ROWS> &w, int t, int first) {
  const int s = t * kTile + first;
  if (first >= kTile || s >= w.s.len + w.s.n) return c.n_pages;
  const int pg = page_of(c, w.b, s);
  if (pg < 0) record_status(c.status, BSA_ERR_BAD_CACHE);
  return pg < 0 ? c.n_pages : pg;
}

}  // namespace bsa
