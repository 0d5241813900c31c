// The list of 128-key tiles that the attention and the weighing of a paged cache
// walk, cut into equal runs, one a CTA; read from the device's lengths, so that a
// captured launch follows them.
#pragma once

#include "serving.cuh"

namespace bsa {

// Sequence b has H_kv * groups(b) items of tiles(b) key tiles each, a row group
// being ROWS of its n * G rows (kAllRows: one group, even of no row); the list is
// all of them in order (b, kv head, row group, tile).
// With WHOLE, the list is of items instead, every row of the T * G in one, and a
// run takes each item from its first tile to its last.
constexpr int kAllRows = 0;

template <int ROWS, bool WHOLE = false>
struct Seq {
  int len, n, tiles, groups;
  __device__ __forceinline__ uint32_t units() const { return WHOLE ? 1u : tiles; }  // of an item
  __device__ __forceinline__ uint32_t work(int H_kv) const { return static_cast<uint32_t>(H_kv) * groups * units(); }
};

template <int ROWS, bool WHOLE = false>
__device__ __forceinline__ Seq<ROWS, WHOLE> sequence(const CacheView &c, const TokenView &t, int b, bool report) {
  Seq<ROWS, WHOLE> s;
  s.len = clamped_length(c, b, report);
  s.n = clamped_new(c, t, b, s.len, report);
  s.tiles = WHOLE && s.n == 0 ? 0 : (s.len + s.n + kTile - 1) / kTile;
  s.groups = ROWS == kAllRows ? min(s.tiles, 1) : ((WHOLE ? t.T : s.n) * t.G + max(ROWS, 1) - 1) / max(ROWS, 1);
  return s;
}

// The list (fewer than 2^31 tiles) in `ctas` runs of one length, the first ones a
// tile longer: run c is [start(c), start(c + 1)).
struct Runs {
  uint32_t total, base, rem;
  __device__ __forceinline__ Runs(uint32_t total_, int ctas)
      : total(total_), base(total_ / ctas), rem(total_ - base * ctas) {}
  __device__ __forceinline__ uint32_t start(uint32_t c) const { return c * base + min(c, rem); }
  // the run that holds list position x < total
  __device__ __forceinline__ uint32_t of(uint32_t x) const {
    const uint32_t longer = rem * (base + 1);
    return x < longer ? x / (base + 1) : rem + (x - longer) / base;
  }
};

struct RunStart {
  int b, item, tile, count;  // count: key tiles of the run
};

// Length of the list, and of its part before sequence `upto`, by one warp.
template <int ROWS, bool WHOLE = false>
__device__ __forceinline__ uint32_t total_work(const CacheView &c, const TokenView &t, int lane, bool report, int upto,
                                               uint32_t *before) {
  uint32_t sum = 0, head = 0;
  for (int b0 = 0; b0 < c.B; b0 += 32) {
    const int b = b0 + lane;
    const uint32_t w = b < c.B ? sequence<ROWS, WHOLE>(c, t, b, report).work(c.H_kv) : 0u;
    sum += w;
    head += b < upto ? w : 0u;
  }
  *before = __reduce_add_sync(0xffffffffu, head);
  return __reduce_add_sync(0xffffffffu, sum);
}

// Where list position `at` lies, by one warp.
template <int ROWS, bool WHOLE = false>
__device__ __forceinline__ RunStart find_start(const CacheView &c, const TokenView &t, uint32_t at, int count, int lane) {
  RunStart r{0, 0, 0, count};
  uint32_t base = 0;
  for (int b0 = 0; b0 < c.B; b0 += 32) {
    Seq<ROWS, WHOLE> s{0, 0, 0, 0};
    if (b0 + lane < c.B) s = sequence<ROWS, WHOLE>(c, t, b0 + lane, false);
    const uint32_t w = s.work(c.H_kv);
    uint32_t incl = w;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const uint32_t o = __shfl_up_sync(0xffffffffu, incl, d);
      if (lane >= d) incl += o;
    }
    const uint32_t off = at - (base + incl - w);  // past w where `at` lies before this sequence too
    const bool here = off < w;
    const uint32_t who = __ballot_sync(0xffffffffu, here);
    if (who != 0u) {
      const int src = __ffs(who) - 1;
      const int item = here ? static_cast<int>(off / s.units()) : 0, tile = here ? static_cast<int>(off % s.units()) : 0;
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

// This CTA's run, by one warp.
template <int ROWS, bool WHOLE = false>
__device__ __forceinline__ RunStart find_run(const CacheView &c, const TokenView &t, int lane) {
  uint32_t unused;
  const Runs runs(total_work<ROWS, WHOLE>(c, t, lane, blockIdx.x == 0, 0, &unused), gridDim.x);
  const uint32_t a = runs.start(blockIdx.x), z = runs.start(blockIdx.x + 1);
  return z > a ? find_start<ROWS, WHOLE>(c, t, a, static_cast<int>(z - a), lane) : RunStart{0, 0, 0, 0};
}

// One CTA's run, piece by piece (a piece: consecutive key tiles of one item).
template <int ROWS, bool WHOLE = false>
struct Walk {
  int b, item, tile, left, index;
  Seq<ROWS, WHOLE> s;
  int hk, rg, t0, t1;  // the piece: kv head, row group, key tiles [t0, t1)
  bool whole;
  __device__ __forceinline__ Walk(const CacheView &c, const TokenView &t, const RunStart &r)
      : b(r.b), item(r.item), tile(r.tile), left(r.count), index(-1) {
    if (left > 0) s = sequence<ROWS, WHOLE>(c, t, b, false);
  }
  __device__ __forceinline__ bool next(const CacheView &c, const TokenView &t) {
    if (left <= 0) return false;
    while (item >= c.H_kv * s.groups) {
      item = 0;
      if (++b >= c.B) return false;  // never, with lengths that stay as they are
      s = sequence<ROWS, WHOLE>(c, t, b, false);
    }
    hk = item / s.groups;
    rg = item % s.groups;
    t0 = tile;
    t1 = WHOLE ? s.tiles : min(s.tiles, tile + left);
    whole = t0 == 0 && t1 == s.tiles;
    left -= WHOLE ? 1 : t1 - t0;
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
template <int ROWS, bool WHOLE>
__device__ __forceinline__ int box_page(const CacheView &c, const Walk<ROWS, WHOLE> &w, int t, int first) {
  const int s = t * kTile + first;
  if (first >= kTile || s >= w.s.len + w.s.n) return c.n_pages;
  const int pg = page_of(c, w.b, s);
  if (pg < 0) record_status(c.status, BSA_ERR_BAD_CACHE);
  return pg < 0 ? c.n_pages : pg;
}

}  // namespace bsa
