// The list of 128-key tiles that the attention and the weighing of a paged cache
// walk, cut into equal runs, one a CTA; read from the device's lengths, so that a
// captured launch follows them.
#pragma once

#include "serving.cuh"

namespace bsa {

// Sequence b has H_kv * groups(b) items of tiles(b) key tiles each, a row group
// being ROWS of its n * G rows (kAllRows: one group, even of no row); the list is
// all of them in order (b, kv head, row group, tile).  It is measured in units: a
// key tile of a group with two row tiles is 3, of one with a single one 2 (4240
// against about 2700 clocks measured; with equal shares of tiles 2 sequences x 64
// tokens x 5 heads a group, rows 256 + 64, over 75600 keys took 341 us, now 285),
// where every group is alike 1; and each item begins with kSwitch units of no tile,
// for what changing to it costs the run's CTA (the sums and O of the item before, the
// pipeline's refill: the CTAs with an item's start among their tiles were last by 6
// of 34 us at 8 sequences x 1 token over 8192 keys, 36.4 us in all without, 33.6
// with; 2048 keys 20.9 and 18.0).  With WHOLE, the list is of items instead, every
// row of the T * G in one, and a run takes each from its first tile to its last.
constexpr int kAllRows = 0;

template <int ROWS, bool WHOLE = false>
struct Seq {
  int len, n, tiles, groups;
  int last;  // the cost of a tile of the last group
  static constexpr int kCost = ROWS > kTile && !WHOLE ? 3 : 1;  // of the others
  static constexpr int kSwitch = WHOLE ? 0 : ROWS > kTile ? 8 : 5;
  __device__ __forceinline__ int cost(int rg) const { return kCost == 1 ? 1 : rg == groups - 1 ? last : kCost; }
  // units of an item, and of a kv head
  __device__ __forceinline__ uint32_t units(int rg) const {
    return WHOLE ? 1u : static_cast<uint32_t>(tiles) * cost(rg) + kSwitch;
  }
  __device__ __forceinline__ uint32_t head_units() const {
    if (WHOLE) return groups;
    return groups == 0 ? 0u : static_cast<uint32_t>(tiles) * ((groups - 1) * kCost + cost(groups - 1)) + groups * kSwitch;
  }
  __device__ __forceinline__ uint32_t work(int H_kv) const { return H_kv * head_units(); }
  // the first unit of group rg within its kv head
  __device__ __forceinline__ uint32_t group_start(int rg) const {
    return WHOLE ? rg : (static_cast<uint32_t>(tiles) * kCost + kSwitch) * rg;
  }
};

template <int ROWS, bool WHOLE = false>
__device__ __forceinline__ Seq<ROWS, WHOLE> sequence(const CacheView &c, const TokenView &t, int b, bool report) {
  Seq<ROWS, WHOLE> s;
  s.len = clamped_length(c, b, report);
  s.n = clamped_new(c, t, b, s.len, report);
  s.tiles = WHOLE && s.n == 0 ? 0 : (s.len + s.n + kTile - 1) / kTile;
  s.groups = ROWS == kAllRows ? min(s.tiles, 1) : ((WHOLE ? t.T : s.n) * t.G + max(ROWS, 1) - 1) / max(ROWS, 1);
  s.last = s.kCost == 1 ? 1 : s.n * t.G - (s.groups - 1) * ROWS > kTile ? 3 : 2;
  return s;
}

// The list (fewer than 2^31 units) in `ctas` runs of one length, the first ones a
// unit longer: run c is [start(c), start(c + 1)).
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
  int b, item, at, count;  // at: units into the item; count: units of the run
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
    Seq<ROWS, WHOLE> s{0, 0, 0, 0, 1};
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
      int item = 0, into = 0;
      if (here) {
        const uint32_t hk = off / s.head_units(), rest = off - hk * s.head_units();
        const uint32_t other = WHOLE ? 1u : static_cast<uint32_t>(s.tiles) * s.kCost + s.kSwitch;
        const int rg = min(static_cast<int>(rest / other), s.groups - 1);
        item = static_cast<int>(hk) * s.groups + rg;
        into = static_cast<int>(rest - s.group_start(rg));
      }
      r.b = b0 + src;
      r.item = __shfl_sync(0xffffffffu, item, src);
      r.at = __shfl_sync(0xffffffffu, into, src);
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

// The units [p0, p1) of an item hold the key tiles [first_tile(p0), first_tile(p1)).
template <typename S>
__device__ __forceinline__ int first_tile(const S &s, uint32_t p, int rg) {
  const uint32_t x = p > S::kSwitch ? p - S::kSwitch : 0u;
  return static_cast<int>(S::kCost == 1 ? x : (x + s.cost(rg) - 1) / s.cost(rg));
}

// One CTA's run, piece by piece (a piece: consecutive key tiles of one item).
template <int ROWS, bool WHOLE = false>
struct Walk {
  int b, item, at, left, index, slot;
  Seq<ROWS, WHOLE> s;
  int hk, rg, t0, t1;  // the piece: kv head, row group, key tiles [t0, t1)
  bool whole;
  __device__ __forceinline__ Walk(const CacheView &c, const TokenView &t, const RunStart &r)
      : b(r.b), item(r.item), at(r.at), left(r.count), index(-1), slot(-1) {
    if (left > 0) s = sequence<ROWS, WHOLE>(c, t, b, false);
  }
  // index counts the pieces; slot is 0 in the run's first item, else 1
  __device__ __forceinline__ bool next(const CacheView &c, const TokenView &t) {
    while (left > 0) {
      while (item >= c.H_kv * s.groups) {
        item = 0;
        if (++b >= c.B) return false;  // never, with lengths that stay as they are
        s = sequence<ROWS, WHOLE>(c, t, b, false);
      }
      hk = item / s.groups;
      rg = item % s.groups;
      const int units = static_cast<int>(s.units(rg)), end = min(units, at + left);
      t0 = WHOLE ? 0 : first_tile(s, at, rg);
      t1 = WHOLE ? s.tiles : first_tile(s, end, rg);
      whole = t0 == 0 && t1 == s.tiles;
      left -= end - at;
      at = 0;
      ++item;
      slot = min(slot + 1, 1);
      if (WHOLE || t0 < t1) {
        ++index;
        return true;
      }
    }
    return false;
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
