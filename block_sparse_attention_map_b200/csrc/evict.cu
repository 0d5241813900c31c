// Eviction from a paged cache: each (sequence, key head) keeps `budget` of its
// slots, by a radix selection on
//   key(slot) = 2^32 - 1 for protected positions (sinks, recent), else the
//               score's bits in an order-preserving form (NaN lowest, -0 as 0),
// highest first, equal keys lowest slot first.
//
// Kept slots at or past the budget move into the dropped ones below it, the
// i-th into the i-th.  Sources lie at or past the budget and destinations below
// it, so the moves need no order among themselves and touch only what changes.
//
// k_evict_select: a cluster of up to 16 CTAs per head, each with an equal share of
// the head's slots in slot order and their keys in shared memory.  Four 8-bit
// histogram passes (the CTAs' histograms summed over distributed shared memory)
// find the key at the budget; two ordered counts over warps and CTAs then number
// ties, holes and movers.  Bound: the latency of the passes, about 1 us each (3.4 in a cluster); one
// CTA a head took 337 us for 65536 slots and 49 us for 4097.
// k_evict_move: a group of D/8 lanes moves one slot's K and V, 16 bytes a lane,
// over all SMs.  Bound: HBM.
#include <cooperative_groups.h>

#include "serving.cuh"

namespace bsa {
namespace {

namespace cg = cooperative_groups;

constexpr int kMaxSelCtas = 16;     // the largest cluster (above 8 a kernel has to ask for it)
constexpr int kMaxKeys = 48 * 1024;  // of a CTA's slots in shared memory (more are read again for each pass)

__device__ __forceinline__ uint32_t score_key(float s) {
  if (s != s) return 0u;
  const uint32_t u = __float_as_uint(s == 0.f ? 0.f : s);
  return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}

struct HeadKeys {
  const float *score;
  const int32_t *pos;
  int sinks, recent_from;
  __device__ __forceinline__ uint32_t of(int p, float sc) const {
    return p < sinks || p >= recent_from ? 0xffffffffu : score_key(sc);
  }
  __device__ __forceinline__ uint32_t operator()(int i) const { return of(pos[i], score[i]); }
};

// Exclusive prefix over the CTA's warps of two counts a warp, by every thread of
// the CTA; the CTA's totals are left in warp_n[kSelWarps].
template <int kSelWarps>
__device__ __forceinline__ int2 count_warps(int2 (&warp_n)[kSelWarps + 1], int2 n) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (lane == 0) warp_n[warp] = n;
  __syncthreads();
  if (warp == 0) {
    const int2 v = lane < kSelWarps ? warp_n[lane] : make_int2(0, 0);
    int2 incl = v;
#pragma unroll
    for (int d = 1; d < kSelWarps; d <<= 1) {
      const int ox = __shfl_up_sync(0xffffffffu, incl.x, d), oy = __shfl_up_sync(0xffffffffu, incl.y, d);
      if (lane >= d) {
        incl.x += ox;
        incl.y += oy;
      }
    }
    if (lane < kSelWarps) warp_n[lane] = make_int2(incl.x - v.x, incl.y - v.y);
    if (lane == kSelWarps - 1) warp_n[kSelWarps] = incl;
  }
  __syncthreads();
  return warp_n[warp];
}

// The moves [0, m) of a head, by the part-th of `parts` blocks: a group of D/8
// lanes moves one slot's K and V, the block's moves of a step next to each other
// (rows of one DRAM page: 74 us against 50 for 16 heads of 65536 slots with the
// groups' moves apart).  AHEAD: the next step's slots and pages are looked up while
// this one's rows are in flight (the same 16 heads: 93 -> 84 us for the whole call).
template <bool AHEAD>
__device__ __forceinline__ void move_rows(const EvictArgs &a, int head, int m, int part, int parts) {
  constexpr int U = 2;  // moves of a group in flight
  const int b = head / a.cache.H_kv, hk = head % a.cache.H_kv;
  const int lanes = a.cache.D >> 3, moves = blockDim.x / lanes;
  const int sub = threadIdx.x % lanes, grp = threadIdx.x / lanes;
  const int64_t lb = static_cast<int64_t>(head) * a.list_cap, base = static_cast<int64_t>(head) * a.cache.capacity;
  int to[U], from[U], pt[U], pf[U];
  // slots and pages of the moves i0, i0 + moves, ...
  auto look = [&](int i0) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = i0 + u * moves;
      to[u] = i < m ? a.to[lb + i] : -1;
      from[u] = i < m ? a.from[lb + i] : -1;
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      pt[u] = to[u] >= 0 ? page_of(a.cache, b, to[u]) : -1;
      pf[u] = to[u] >= 0 ? page_of(a.cache, b, from[u]) : -1;
    }
  };
  const int first = part * U * moves + grp, step = parts * U * moves;
  if (AHEAD && first < m) look(first);
  for (int i0 = first; i0 < m; i0 += step) {
    if (!AHEAD) look(i0);
    int4 kv[U], vv[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (pt[u] < 0 || pf[u] < 0) continue;
      kv[u] = *reinterpret_cast<const int4 *>(a.cache.k + slot_offset(a.cache.ks, a.cache, pf[u], from[u], hk) + sub * 8);
      vv[u] = *reinterpret_cast<const int4 *>(a.cache.v + slot_offset(a.cache.vs, a.cache, pf[u], from[u], hk) + sub * 8);
    }
    int now[U];
    bool good[U];
    float sc[U];
    int ps[U];
    uint16_t *kd[U], *vd[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      now[u] = to[u];
      good[u] = pt[u] >= 0 && pf[u] >= 0;
      if (good[u]) {
        kd[u] = a.cache.k + slot_offset(a.cache.ks, a.cache, pt[u], to[u], hk) + sub * 8;
        vd[u] = a.cache.v + slot_offset(a.cache.vs, a.cache, pt[u], to[u], hk) + sub * 8;
      }
      if (sub == 0 && to[u] >= 0) {
        sc[u] = a.mscore[lb + i0 + u * moves];
        ps[u] = a.mpos[lb + i0 + u * moves];
      }
    }
    if (AHEAD && i0 + step < m) look(i0 + step);  // under the rows' loads
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (now[u] < 0) continue;
      if (good[u]) {
        *reinterpret_cast<int4 *>(kd[u]) = kv[u];
        *reinterpret_cast<int4 *>(vd[u]) = vv[u];
      } else if (sub == 0) {
        record_status(a.cache.status, BSA_ERR_BAD_CACHE);
      }
      if (sub == 0) {
        a.score_out[base + now[u]] = sc[u];
        a.pos_out[base + now[u]] = ps[u];
      }
    }
  }
}

// CLUSTER: a head has several CTAs.  K > 0: a thread's keys in K registers; K = 0: in shared memory where key_cap
// holds them, else read again by each pass.  MOVES: the CTAs move their head's rows
// too (and where the lengths do not change in place, write them).
template <int kSelThreads, int K, bool CLUSTER, bool MOVES>
__global__ void __launch_bounds__(kSelThreads, 1024 / kSelThreads) k_evict_select(const EvictArgs a, int key_cap) {
  constexpr int kSelWarps = kSelThreads / 32;
  extern __shared__ uint32_t keys[];  // [key_cap]: this CTA's, where they fit
  __shared__ __align__(16) uint32_t hist[2][256];   // one a pass by turns, so that a pass needs one cluster barrier
  __shared__ uint32_t sel[3];         // chosen digit, what is still wanted within it, the keys of it in lower CTAs
  __shared__ int2 counts[2][kSelWarps + 1];
  cg::cluster_group cluster = cg::this_cluster();
  const unsigned ctas = CLUSTER ? cluster.num_blocks() : 1u, rank = CLUSTER ? cluster.block_rank() : 0u;
  const int head = blockIdx.x / ctas, b = head / a.cache.H_kv;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t base = static_cast<int64_t>(head) * a.cache.capacity;
  pdl_wait();
  const int n = clamped_length(a.cache, b, tid == 0 && rank == 0);
  const float *score = a.score_in + base;
  const int32_t *pos = a.pos_in + base;
  float *score_out = a.score_out + base;
  int32_t *pos_out = a.pos_out + base;
  // only this call's second kernel may start under it: another's may not expect it
  if (!MOVES || a.length_out == a.cache.length) pdl_trigger();
  if (MOVES && a.length_out != a.cache.length && head % a.cache.H_kv == 0 && rank == 0 && tid == 0)
    a.length_out[b] = min(n, a.budget);
  if (n <= a.budget) {  // the whole cluster
    if (!MOVES && tid == 0 && rank == 0) a.count[head] = 0;
    if (score_out != score)
      for (int i = rank * kSelThreads + tid; i < n; i += ctas * kSelThreads) score_out[i] = score[i];
    if (pos_out != pos)
      for (int i = rank * kSelThreads + tid; i < n; i += ctas * kSelThreads) pos_out[i] = pos[i];
    return;
  }
  // next_pos - recent below the int32 range: everything is recent
  const int64_t rf = static_cast<int64_t>(a.next_pos[b]) - a.recent;
  const HeadKeys key_of{score, pos, a.sinks, static_cast<int>(rf < INT_MIN ? INT_MIN : rf)};

  // this warp's slots [w0, w1), in slot order over the warps of the cluster's CTAs
  const int chunks = (n + 31) / 32, per_warp = (chunks + ctas * kSelWarps - 1) / (ctas * kSelWarps) * 32;
  const int s0 = static_cast<int>(rank) * kSelWarps * per_warp;  // the CTA's first
  const int w0 = min(s0 + warp * per_warp, n), w1 = min(w0 + per_warp, n);
  const bool kept_here = kSelWarps * per_warp <= key_cap;
  uint32_t regs[K > 0 ? K : 1];
  // f(k, slot) for the warp's slots in order, 32 at a time, by all lanes (the last slots may lie at or past w1)
  auto each = [&](auto f) {
    if constexpr (K > 0) {
#pragma unroll
      for (int k = 0; k < K; ++k)
        if (w0 + 32 * k < w1) f(k, w0 + 32 * k + lane);
    } else {
#pragma unroll 4
      for (int i0 = w0; i0 < w1; i0 += 32) f(0, i0 + lane);
    }
  };
  static_assert(K == 0 || K == 8, "a cluster's last pass takes a lane's slots eight at a time");
  auto key = [&](int k, int i) {
    if constexpr (K > 0) return regs[k];
    else return i >= w1 ? 0u : kept_here ? keys[i - s0] : key_of(i);
  };
  for (int i = tid; i < 256; i += kSelThreads) hist[0][i] = 0;
  if constexpr (K > 0) {
    int ps[K];
    float sc[K];
#pragma unroll
    for (int k = 0; k < K; ++k) {  // all loads in flight
      const int i = min(w0 + 32 * k + lane, n - 1);
      ps[k] = pos[i];
      sc[k] = score[i];
    }
#pragma unroll
    for (int k = 0; k < K; ++k) regs[k] = w0 + 32 * k + lane < w1 ? key_of.of(ps[k], sc[k]) : 0u;
  } else if (kept_here) {
    constexpr int U = 8;  // loads of U slots in flight
    for (int i0 = w0 + lane; i0 < w1; i0 += 32 * U) {
      int ps[U];
      float sc[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int i = min(i0 + 32 * u, n - 1);
        ps[u] = pos[i];
        sc[u] = score[i];
      }
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (i0 + 32 * u < w1) keys[i0 + 32 * u - s0] = key_of.of(ps[u], sc[u]);
    }
  }
  __syncthreads();

  // the key at the budget, digit by digit from the top
  uint32_t prefix = 0, want = static_cast<uint32_t>(a.budget);
#pragma unroll 1
  for (int pass = 0; pass < 4; ++pass) {
    const int shift = 24 - 8 * pass;
    uint32_t *mine = hist[pass & 1];
    const uint32_t mask = pass == 0 ? 0u : ~0u << (shift + 8);
    each([&](int k, int i) {
      const uint32_t x = key(k, i);
      if (i < w1 && (x & mask) == prefix) atomicAdd(&mine[(x >> shift) & 255u], 1u);
    });
    if (CLUSTER) cluster.sync();
    else __syncthreads();
    if (warp == 0) {
      // lane l: the digits 255 - 8 l down to 248 - 8 l
      uint32_t v[8], sum = 0;
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] = 0;
      uint32_t low[8];  // of the CTAs before this one
#pragma unroll
      for (int k = 0; k < 8; ++k) low[k] = 0;
      if (!CLUSTER) {
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] = mine[255 - 8 * lane - k];
      } else {
#pragma unroll 1
        for (unsigned c0 = 0; c0 < ctas; c0 += 4) {
          uint4 x[4], y[4];  // four CTAs' loads in flight (a cluster is 1, 4, 8 or 16)
#pragma unroll
          for (unsigned c = 0; c < 4; ++c) {
            const uint4 *theirs = reinterpret_cast<const uint4 *>(cluster.map_shared_rank(mine, c0 + c) + 248 - 8 * lane);
            x[c] = theirs[0];
            y[c] = theirs[1];
          }
#pragma unroll
          for (unsigned c = 0; c < 4; ++c) {
            const uint32_t t8[8] = {y[c].w, y[c].z, y[c].y, y[c].x, x[c].w, x[c].z, x[c].y, x[c].x};
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              v[k] += t8[k];
              low[k] += c0 + c < rank ? t8[k] : 0u;
            }
          }
        }
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) sum += v[k];
      uint32_t incl = sum;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const uint32_t o = __shfl_up_sync(0xffffffffu, incl, d);
        if (lane >= d) incl += o;
      }
      const uint32_t excl = incl - sum;
      if (excl < want && want <= incl) {  // one lane
        uint32_t left = want - excl;
        bool found = false;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          if (!found && v[k] >= left) {
            found = true;
            sel[0] = static_cast<uint32_t>(255 - 8 * lane - k);
            sel[1] = left;
            sel[2] = low[k];
          }
          if (!found) left -= v[k];
        }
      }
    } else {
      // the next pass's histogram: its last readers passed the barrier above
      for (int i = tid - 32; i < 256; i += kSelThreads - 32) hist[(pass + 1) & 1][i] = 0;
    }
    __syncthreads();
    prefix |= sel[0] << shift;
    want = sel[1];
    __syncthreads();
  }

  // In slot order: keep keys above `prefix` and the first `want` equal to it.  The
  // warp's equal keys, those of them below the budget, and of the other keys the
  // holes and movers; which equal keys stay follows from how many came before.
  const uint32_t below = (1u << lane) - 1u;
  int ties = 0, low_ties = 0, holes = 0, movers = 0;
  each([&](int k, int i) {
    const bool in = i < w1;
    const uint32_t x = key(k, i);
    const uint32_t tb = __ballot_sync(0xffffffffu, in && x == prefix), lb = __ballot_sync(0xffffffffu, i < a.budget);
    ties += __popc(tb);
    low_ties += __popc(tb & lb);
    holes += __popc(__ballot_sync(0xffffffffu, in && x < prefix) & lb);
    movers += __popc(__ballot_sync(0xffffffffu, in && x > prefix) & ~lb);
  });
  // equal keys of lower CTAs (from the last pass's histograms) and lower warps
  const int ties_before = static_cast<int>(sel[2]) + count_warps<kSelWarps>(counts[0], make_int2(ties, 0)).x;
  const int tie_keep = min(max(static_cast<int>(want) - ties_before, 0), ties), low_keep = min(tie_keep, low_ties);
  holes += low_ties - low_keep;
  movers += tie_keep - low_keep;
  const int2 in_cta = count_warps<kSelWarps>(counts[1], make_int2(holes, movers));
  int hole_at = in_cta.x, mover_at = in_cta.y, moved = counts[1][kSelWarps].y;
  if (CLUSTER) {
    cluster.sync();
    // every lane one CTA's totals, added up over the warp
    const int2 t = lane < static_cast<int>(ctas) ? cluster.map_shared_rank(&counts[1][kSelWarps], lane)[0] : make_int2(0, 0);
    const bool lower = lane < static_cast<int>(rank);
    hole_at += __reduce_add_sync(0xffffffffu, lower ? t.x : 0);
    mover_at += __reduce_add_sync(0xffffffffu, lower ? t.y : 0);
    moved = __reduce_add_sync(0xffffffffu, t.y);
  }
  int32_t *to = a.to + static_cast<int64_t>(head) * a.list_cap;
  int32_t *from = a.from + static_cast<int64_t>(head) * a.list_cap;
  int32_t *mpos = a.mpos + static_cast<int64_t>(head) * a.list_cap;
  float *mscore = a.mscore + static_cast<int64_t>(head) * a.list_cap;
  // Kept slots below the budget stay where they are: nothing to do for them where
  // the outputs are the inputs.
  const bool copies = score_out != score || pos_out != pos;
  int seen = ties_before;
  auto place = [&](uint32_t x, int i, auto get) {
    const bool in = i < w1;
    const uint32_t tb = __ballot_sync(0xffffffffu, in && x == prefix);
    const bool k = in && (x > prefix || (x == prefix && seen + __popc(tb & below) < static_cast<int>(want)));
    seen += __popc(tb);
    const bool hole = in && !k && i < a.budget, mover = k && i >= a.budget;
    const uint32_t hb = __ballot_sync(0xffffffffu, hole), mb = __ballot_sync(0xffffffffu, mover);
    // (never past the lists, whatever another stream does to the inputs meanwhile)
    const int ha = hole_at + __popc(hb & below), ma = mover_at + __popc(mb & below);
    if (hole && ha < a.list_cap) to[ha] = i;
    const bool copy = k && copies && i < a.budget;  // (holes are filled by the move)
    if (mover || copy) {
      float sc;
      int ps;
      get(sc, ps);
      if (copy) {
        score_out[i] = sc;
        pos_out[i] = ps;
      } else if (ma < a.list_cap) {
        from[ma] = i;
        mpos[ma] = ps;
        mscore[ma] = sc;
      }
    }
    if (in && i >= a.budget) {
      score_out[i] = 0.f;
      pos_out[i] = -1;
    }
    hole_at += __popc(hb);
    mover_at += __popc(mb);
  };
  if constexpr (CLUSTER) {
    // all of what may move or be copied, eight slots of a lane in flight (65536 slots to half: 38 -> 34 us; a CTA alone
    // has too many threads for the registers, 11.6 -> 12.5 us for 4097 slots)
    constexpr int U = 8;
    for (int i0 = w0; i0 < w1; i0 += 32 * U) {
      float sc[U];
      int ps[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int i = i0 + 32 * u + lane;
        sc[u] = 0.f;
        ps[u] = 0;
        if (i < w1 && (copies || i >= a.budget)) {
          sc[u] = score[i];
          ps[u] = pos[i];
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int i = i0 + 32 * u + lane;
        if (i0 + 32 * u < w1)
          place(key(u, i), i, [&](float &x, int &y) {
            x = sc[u];
            y = ps[u];
          });
      }
    }
  } else {
    each([&](int k, int i) {
      place(key(k, i), i, [&](float &x, int &y) {
        x = score[i];
        y = pos[i];
      });
    });
  }
  if (!MOVES && tid == 0 && rank == 0) a.count[head] = min(moved, a.list_cap);
  // no CTA leaves while another may read its shared memory; and the lists are whole
  if (CLUSTER) cluster.sync();
  else __syncthreads();
  if (MOVES) move_rows<false>(a, head, min(moved, a.list_cap), rank, ctas);
}

// The moves by every SM, and the new lengths (the selection is done with the old ones).
__global__ void __launch_bounds__(256) k_evict_move(const EvictArgs a, int per_head) {
  const int head = blockIdx.x / per_head, part = blockIdx.x % per_head;
  pdl_wait();
  move_rows<true>(a, head, a.count[head], part, per_head);
  if (part == 0 && head % a.cache.H_kv == 0 && threadIdx.x == 0) {
    const int b = head / a.cache.H_kv;
    a.length_out[b] = min(min(max(a.cache.length[b], 0), a.cache.capacity), a.budget);
  }
}

// The new lengths alone.
__global__ void __launch_bounds__(256) k_evict_length(const EvictArgs a) {
  const int b = blockIdx.x * 256 + threadIdx.x;
  pdl_wait();
  if (b < a.cache.B) a.length_out[b] = min(min(max(a.cache.length[b], 0), a.cache.capacity), a.budget);
}

template <int THREADS, int K, bool CLUSTER, bool MOVES>
cudaError_t select(const EvictArgs &a, int heads, int ctas, cudaStream_t s) {
  constexpr int kWarps = THREADS / 32;
  const auto kernel = k_evict_select<THREADS, K, CLUSTER, MOVES>;
  // a CTA's slots, at most
  const int share = ((a.cache.capacity + 31) / 32 + ctas * kWarps - 1) / (ctas * kWarps) * THREADS;
  const int key_cap = K == 0 && share <= kMaxKeys ? share : 0;
  static std::atomic<uint64_t> smem_done{0}, size_done{0};
  cudaError_t e = cudaSuccess;
  if (K == 0 && (e = allow(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxKeys * 4, smem_done)) != cudaSuccess)
    return e;
  if (ctas > 8 && (e = allow(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1, size_done)) != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(heads) * ctas);
  cfg.blockDim = dim3(THREADS);
  cfg.dynamicSmemBytes = static_cast<size_t>(key_cap) * 4;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = ctas;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  count_launch();
  return cudaLaunchKernelEx(&cfg, kernel, a, key_cap);
}

template <int THREADS, int K, bool CLUSTER>
cudaError_t evict(const EvictArgs &a, int ctas, cudaStream_t s) {
  const int heads = a.cache.B * a.cache.H_kv;
  // The CTAs that select move the rows too where no more than a few can move (one
  // launch less: 4097 slots to 4096 13.3 -> 11.5 us); else a second kernel on all SMs
  // (32 heads of 32768 slots to half by the selecting CTAs: 104 us against 75).
  if (a.list_cap <= 512) {
    const cudaError_t e = select<THREADS, K, CLUSTER, true>(a, heads, ctas, s);
    if (e != cudaSuccess || a.length_out != a.cache.length) return e;
    count_launch();
    return launch_pdl(k_evict_length, dim3((a.cache.B + 255) / 256), dim3(256), 0, s, a);
  }
  const cudaError_t e = select<THREADS, K, CLUSTER, false>(a, heads, ctas, s);
  if (e != cudaSuccess) return e;
  const int per_head = std::max(1, std::min((148 * 8 + heads - 1) / heads, (a.list_cap + 15) / 16));
  count_launch();
  return launch_pdl(k_evict_move, dim3(heads * per_head), dim3(256), 0, s, a, per_head);
}

}  // namespace

cudaError_t launch_evict(const EvictArgs &a, cudaStream_t s) {
  // A head's slots are 8 a thread of one CTA up to 8192 (few slots in a large CTA
  // are slots for no one: 512 heads of 1025 slots 39 us with 1024 threads), else of
  // a cluster of CTAs of 512 threads, so that an SM holds two (16 clusters of 8 x
  // 1024 did not fit the GPU at once: over twice the time for the selection of 65536).
  const int cap = a.cache.capacity;
  if (cap <= 2048) return evict<256, 8, false>(a, 1, s);
  if (cap <= 4096) return evict<512, 8, false>(a, 1, s);
  if (cap <= 8192) return evict<1024, 8, false>(a, 1, s);
  if (cap <= 16384) return evict<512, 8, true>(a, 4, s);
  if (cap <= 32768) return evict<512, 8, true>(a, 8, s);
  // 16 CTAs where the heads are few (1 head of 10^6 slots 806 -> 442 us; 16 heads of
  // 65536 found too few places for such clusters: 83 -> 101 us), and where the keys
  // of a head do not fit the shared memory of 8 (16 heads of 500000 444 -> 227 us)
  if (cap <= 65536 && a.cache.B * a.cache.H_kv <= 4) return evict<512, 8, true>(a, 16, s);
  if (cap > 8 * kMaxKeys || a.cache.B * a.cache.H_kv <= 4) return evict<512, 0, true>(a, 16, s);
  return evict<512, 0, true>(a, 8, s);
}

}  // namespace bsa
