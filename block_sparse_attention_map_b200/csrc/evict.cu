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
// k_evict_select: one CTA per head; four 8-bit histogram passes find the key at
// the budget, then one ordered pass numbers ties, holes and movers.
// k_evict_move: a group of D/8 lanes moves one slot's K and V, 16 bytes a lane.
#include "serving.cuh"

namespace bsa {
namespace {

constexpr int kSelThreads = 1024;

__device__ __forceinline__ uint32_t score_key(float s) {
  if (s != s) return 0u;
  const uint32_t u = __float_as_uint(s == 0.f ? 0.f : s);
  return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}

struct HeadKeys {
  const float *score;
  const int32_t *pos;
  int sinks, recent_from;
  __device__ __forceinline__ uint32_t operator()(int i) const {
    const int p = pos[i];
    return p < sinks || p >= recent_from ? 0xffffffffu : score_key(score[i]);
  }
};

__global__ void __launch_bounds__(kSelThreads) k_evict_select(const EvictArgs a) {
  __shared__ uint32_t hist[256];
  __shared__ uint32_t sel[2];       // chosen digit, what is still wanted within it
  __shared__ int warp_tot[3][32];
  const int head = blockIdx.x, b = head / a.cache.H_kv;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t base = static_cast<int64_t>(head) * a.cache.capacity;
  const int n = clamped_length(a.cache, b, tid == 0);
  const float *score = a.score_in + base;
  const int32_t *pos = a.pos_in + base;
  float *score_out = a.score_out + base;
  int32_t *pos_out = a.pos_out + base;
  if (n <= a.budget) {
    if (tid == 0) a.count[head] = 0;
    if (score_out != score)
      for (int i = tid; i < n; i += kSelThreads) score_out[i] = score[i];
    if (pos_out != pos)
      for (int i = tid; i < n; i += kSelThreads) pos_out[i] = pos[i];
    return;
  }
  // next_pos - recent below the int32 range: everything is recent
  const int64_t rf = static_cast<int64_t>(a.next_pos[b]) - a.recent;
  const HeadKeys key{score, pos, a.sinks, static_cast<int>(rf < INT_MIN ? INT_MIN : rf)};

  // the key at the budget, digit by digit from the top
  uint32_t prefix = 0, want = static_cast<uint32_t>(a.budget);
#pragma unroll 1
  for (int shift = 24; shift >= 0; shift -= 8) {
    if (tid < 256) hist[tid] = 0;
    __syncthreads();
    const uint32_t mask = shift == 24 ? 0u : ~0u << (shift + 8);
    for (int i = tid; i < n; i += kSelThreads) {
      const uint32_t x = key(i);
      if ((x & mask) == prefix) atomicAdd(&hist[(x >> shift) & 255u], 1u);
    }
    __syncthreads();
    if (tid == 0) {
      uint32_t left = want;
      int d = 255;
      for (; d > 0 && hist[d] < left; --d) left -= hist[d];
      sel[0] = static_cast<uint32_t>(d);
      sel[1] = left;
    }
    __syncthreads();
    prefix |= sel[0] << shift;
    want = sel[1];
    __syncthreads();
  }

  // in slot order: keep keys above `prefix` and the first `want` equal to it
  int ties = 0, holes = 0, movers = 0;  // so far, over the chunks done
  int32_t *to = a.to + static_cast<int64_t>(head) * a.list_cap;
  int32_t *from = a.from + static_cast<int64_t>(head) * a.list_cap;
  int32_t *mpos = a.mpos + static_cast<int64_t>(head) * a.list_cap;
  float *mscore = a.mscore + static_cast<int64_t>(head) * a.list_cap;
  const uint32_t below = (1u << lane) - 1u;
  for (int i0 = 0; i0 < n; i0 += kSelThreads) {
    const int i = i0 + tid;
    const bool in = i < n;
    const uint32_t x = in ? key(i) : 0u;
    const bool tie = in && x == prefix;
    const uint32_t tb = __ballot_sync(0xffffffffu, tie);
    if (lane == 0) warp_tot[0][warp] = __popc(tb);
    __syncthreads();
    int before = ties + __popc(tb & below), all = 0;
    for (int w = 0; w < 32; ++w) {
      if (w < warp) before += warp_tot[0][w];
      all += warp_tot[0][w];
    }
    ties += all;
    const bool keep = in && (x > prefix || (tie && before < static_cast<int>(want)));
    const bool hole = in && !keep && i < a.budget, mover = keep && i >= a.budget;
    const uint32_t hb = __ballot_sync(0xffffffffu, hole), mb = __ballot_sync(0xffffffffu, mover);
    if (lane == 0) {
      warp_tot[1][warp] = __popc(hb);
      warp_tot[2][warp] = __popc(mb);
    }
    __syncthreads();
    int hi = holes + __popc(hb & below), mi = movers + __popc(mb & below), ha = 0, ma = 0;
    for (int w = 0; w < 32; ++w) {
      if (w < warp) {
        hi += warp_tot[1][w];
        mi += warp_tot[2][w];
      }
      ha += warp_tot[1][w];
      ma += warp_tot[2][w];
    }
    holes += ha;
    movers += ma;
    if (hole) to[hi] = i;
    if (mover) {
      from[mi] = i;
      mpos[mi] = pos[i];
      mscore[mi] = score[i];
    }
    if (in) {
      // movers were read above by this thread; holes are filled by the move
      if (i >= a.budget) {
        score_out[i] = 0.f;
        pos_out[i] = -1;
      } else if (keep) {
        score_out[i] = score[i];
        pos_out[i] = pos[i];
      }
    }
  }
  if (tid == 0) a.count[head] = movers;
}

template <int D>
__global__ void __launch_bounds__(256) k_evict_move(const EvictArgs a, int per_head) {
  constexpr int L = D / 8;  // lanes a row
  const int head = blockIdx.x / per_head, part = blockIdx.x % per_head;
  const int b = head / a.cache.H_kv, hk = head % a.cache.H_kv;
  const int sub = threadIdx.x % L, grp = threadIdx.x / L;
  constexpr int kGroups = 256 / L;
  pdl_wait();
  const int m = a.count[head];
  const int64_t lb = static_cast<int64_t>(head) * a.list_cap, base = static_cast<int64_t>(head) * a.cache.capacity;
  for (int i = part * kGroups + grp; i < m; i += per_head * kGroups) {
    const int to = a.to[lb + i], from = a.from[lb + i];
    const int pt = page_of(a.cache, b, to), pf = page_of(a.cache, b, from);
    if (pt >= 0 && pf >= 0) {
      const int4 kv = *reinterpret_cast<const int4 *>(a.cache.k + slot_offset(a.cache.ks, a.cache, pf, from, hk) + sub * 8);
      const int4 vv = *reinterpret_cast<const int4 *>(a.cache.v + slot_offset(a.cache.vs, a.cache, pf, from, hk) + sub * 8);
      *reinterpret_cast<int4 *>(a.cache.k + slot_offset(a.cache.ks, a.cache, pt, to, hk) + sub * 8) = kv;
      *reinterpret_cast<int4 *>(a.cache.v + slot_offset(a.cache.vs, a.cache, pt, to, hk) + sub * 8) = vv;
    } else if (sub == 0) {
      record_status(a.cache.status, BSA_ERR_BAD_CACHE);
    }
    if (sub == 0) {
      a.score_out[base + to] = a.mscore[lb + i];
      a.pos_out[base + to] = a.mpos[lb + i];
    }
  }
  if (part == 0 && hk == 0 && threadIdx.x == 0) {
    // k_evict_select is done with the lengths
    const int n = min(max(a.cache.length[b], 0), a.cache.capacity);
    a.length_out[b] = min(n, a.budget);
  }
}

}  // namespace

cudaError_t launch_evict(const EvictArgs &a, cudaStream_t s) {
  const int heads = a.cache.B * a.cache.H_kv;
  count_launch(2);
  k_evict_select<<<heads, kSelThreads, 0, s>>>(a);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const int per_head = std::max(1, std::min((148 * 8 + heads - 1) / heads, (a.list_cap + 15) / 16));
  return a.cache.D == 64
             ? launch_pdl(k_evict_move<64>, dim3(heads * per_head), dim3(256), 0, s, a, per_head)
             : launch_pdl(k_evict_move<128>, dim3(heads * per_head), dim3(256), 0, s, a, per_head);
}

}  // namespace bsa
