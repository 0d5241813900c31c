// Attention of a few new tokens (a tree of drafted tokens, or one) over a paged
// cache: O = softmax(scale q K^T) V and the LSE, row (token t, head h) seeing
// the slots below length and the new tokens of its tree word.
//
// The T * G rows of a kv head's group (row = t * G + g) share its keys, so K and
// V are read once for up to 256 of them: one or two 128-row tiles (NX) against
// 128-key tiles.  Up to about 200 rows the floor is HBM (4 D bytes a key).
//
// k_attend: one CTA per SM.  The (sequence, kv head, row group, key tile) list is
// cut into equal runs, one a CTA, whatever the lengths are (they are read on the
// device, so a captured launch follows them).  A run that covers all key tiles
// of its rows writes their result; the pieces of the others go to the workspace
// as unnormalised O with the running maximum and sums, and k_attend_join adds
// them in tile order, so the same inputs give the same bits.
//   warp 0      TMA producer: a 128-key tile is 128 / page_size boxes of one page
//               each (lane i looks up and loads box i); a box of no slot in use,
//               and a page index out of range, reads a page past the end: zeros.
//   warp 1      tcgen05 issuer, one lane: S = Q K^T (SS), O += P V (TS, P over
//               the S columns).  NX = 1: the S of tile j+1 is computed under the
//               softmax of tile j (two S buffers); NX = 2: the two row tiles
//               alternate.
//   warps 4-7, 8-11   softmax of row tile x, one row a thread: Q into shared
//               memory, the tile's maximum, lazy rescale of O, P as 16-bit, the
//               epilogue.  Tiles with new tokens are masked by the tree word.
// V of what no row may see: slots past the new tokens are zeroed in shared memory
// (0 * NaN is NaN in the product), and a new token's infinities and NaN are taken
// out of the tile and added back in the epilogue of the rows that see the token.
// TMEM columns: S_0 [0,128) S_1 [128,256) O_0 [256,256+D) O_1 [256+D,256+2D).
#include "runs.cuh"

namespace bsa {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kRescaleThreshold = 8.0f;  // log2 units: tolerate p up to 2^8

struct AttendParams {
  CacheView cache;
  TokenView tok;
  const uint16_t *q;
  uint16_t *out;
  int64_t qs[3], os[3];
  float *lse;
  float scale_log2;
  int box_rows, box_log;  // keys of one TMA box: min(page_size, 128)
  float *part_o;          // [2 * CTAs, 128 * NX, D] unnormalised O of the pieces
  float4 *part_ml;        // [2 * CTAs, 128 * NX] maximum (log2), sum, sum of rounded weights
};

template <int D, int NX>
struct AttendSmem {
  static constexpr int kTB = kTile * D * 2;
  static constexpr int NK = D == 128 ? 3 : 5, NV = D == 128 ? (NX == 1 ? 3 : 2) : 5;
  static constexpr int kQ = 0, kK = NX * kTB, kV = kK + NK * kTB, kBar = kV + NV * kTB;
  static constexpr int bKFull = 0, bKEmpty = NK, bVFull = 2 * NK, bVEmpty = bVFull + NV, bQFull = bVEmpty + NV,
                       bSFull = bQFull + NX, bPFull = bSFull + 2, bPVDone = bPFull + 2, bFinal = bPVDone + NX,
                       kNumBars = bFinal + 1;
  static constexpr int kBad = kBar + kNumBars * 8;     // uint32 [4][2]: new tokens whose V is not finite
  static constexpr int kRun = kBad + 32;               // RunStart
  static constexpr int kMisc = kRun + 16;              // tmem slot, abort flag
  static constexpr int kAlloc = kMisc + 16;
};

// Mask of the 16-bit halves of `w` that are infinite or NaN.
template <bool FP16>
__device__ __forceinline__ uint32_t not_finite(uint32_t w) {
  constexpr uint32_t e = FP16 ? 0x7c00u : 0x7f80u;
  return ((w & e) == e ? 0xffffu : 0u) | ((w & (e << 16)) == (e << 16) ? 0xffff0000u : 0u);
}

template <bool FP16, int D, int NX>
__global__ void __launch_bounds__(NX == 1 ? 256 : 384, 1)
k_attend(const __grid_constant__ CUtensorMap tk, const __grid_constant__ CUtensorMap tv, const AttendParams p) {
  using L = AttendSmem<D, NX>;
  extern __shared__ __align__(1024) uint8_t sm[];
  uint64_t *bars = reinterpret_cast<uint64_t *>(sm + L::kBar);
  uint32_t *bad = reinterpret_cast<uint32_t *>(sm + L::kBad);
  RunStart *run_sm = reinterpret_cast<RunStart *>(sm + L::kRun);
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(sm + L::kMisc);
  int *abort_flag = reinterpret_cast<int *>(sm + L::kMisc + 4);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  constexpr int kTB = L::kTB, NK = L::NK, NV = L::NV;

  if (threadIdx.x == 32) {
    for (int i = 0; i < L::kNumBars; ++i)
      mbar_init(&bars[i], (i >= L::bQFull && i < L::bQFull + NX) || (i >= L::bPFull && i < L::bPFull + 2) ? 128 : 1);
    *abort_flag = 0;
    for (int i = 0; i < 8; ++i) bad[i] = 0;
    fence_mbar_init();
    fence_proxy_async_smem();
  }
  if (warp == 0) {
    if (lane == 0) {
      tma_prefetch_desc(&tk);
      tma_prefetch_desc(&tv);
    }
    const int64_t total = total_work<kTile * NX>(p.cache, p.tok, lane, blockIdx.x == 0);
    const int64_t a = run_start(total, blockIdx.x, gridDim.x), z = run_start(total, blockIdx.x + 1, gridDim.x);
    const RunStart r = z > a ? find_start<kTile * NX>(p.cache, p.tok, a, static_cast<int>(z - a), lane) : RunStart{0, 0, 0, 0};
    if (lane == 0) *run_sm = r;
  }
  if (warp == 1) {
    __syncwarp();
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  pdl_trigger();
  const uint32_t tmem = *tmem_slot;
  Watchdog wd{abort_flag, p.cache.status, kWaitLimitNs};
  const RunStart run = *run_sm;
  if (threadIdx.x == 0 && (smem_u32(sm) & 1023u) != 0u) wd.trip(BSA_ERR_UNSUPPORTED);
  __syncthreads();

  constexpr uint32_t kIdescS = FP16 ? idesc_f16_f32(128, 128, 0, 0) : idesc_bf16_f32(128, 128, 0, 0);
  constexpr uint32_t kIdescPV = FP16 ? idesc_f16_f32(128, D, 0, 1) : idesc_bf16_f32(128, D, 0, 1);

  if (wd.aborted()) {
  } else if (warp == 0) {
    // ------------------------------------------------------------ producer
    Walk<kTile * NX> w(p.cache, p.tok, run);
    uint32_t kv = 0;
    bool stop = false;
    const int boxes = kTile >> p.box_log;
    auto page_for = [&](int t) { return box_page(p.cache, w, t, lane << p.box_log); };
    while (!stop && w.next(p.cache, p.tok)) {
      int page_next = page_for(w.t0);
      for (int t = w.t0; t < w.t1; ++t, ++kv) {
        const int page = page_next;
        const int row = (t * kTile + (lane << p.box_log)) & ((1 << p.cache.page_log) - 1);
        if (t + 1 < w.t1) page_next = page_for(t + 1);
        const uint32_t ks = kv % NK, vs = kv % NV;
        bool ok = kv < NK || wd.wait(&bars[L::bKEmpty + ks], ((kv / NK) - 1) & 1);
        if (!__all_sync(0xffffffffu, ok)) { stop = true; break; }
        if (lane == 0) mbar_arrive_expect_tx(&bars[L::bKFull + ks], kTB);
        __syncwarp();
        if (lane < boxes) {
#pragma unroll
          for (int c = 0; c < D / 64; ++c)
            tma_load_4d(sm + L::kK + ks * kTB + c * 16384 + (lane << p.box_log) * 128, &tk, &bars[L::bKFull + ks],
                        c * 64, row, w.hk, page);
        }
        ok = kv < NV || wd.wait(&bars[L::bVEmpty + vs], ((kv / NV) - 1) & 1);
        if (!__all_sync(0xffffffffu, ok)) {
          // the K tile in flight lands before this CTA's shared memory goes away
          drain_wait(&bars[L::bKFull + ks], (kv / NK) & 1);
          stop = true;
          break;
        }
        if (lane == 0) mbar_arrive_expect_tx(&bars[L::bVFull + vs], kTB);
        __syncwarp();
        if (lane < boxes) {
#pragma unroll
          for (int c = 0; c < D / 64; ++c)
            tma_load_4d(sm + L::kV + vs * kTB + c * 16384 + (lane << p.box_log) * 128, &tv, &bars[L::bVFull + vs],
                        c * 64, row, w.hk, page);
        }
      }
    }
    if (wd.aborted()) {
      for (uint32_t t = (kv > NK ? kv - NK : 0); t < kv; ++t) drain_wait(&bars[L::bKFull + t % NK], (t / NK) & 1);
      for (uint32_t t = (kv > NV ? kv - NV : 0); t < kv; ++t) drain_wait(&bars[L::bVFull + t % NV], (t / NV) & 1);
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    if (lane == 0) {
      Walk<kTile * NX> w(p.cache, p.tok, run);
      uint32_t kv = 0;  // key tiles done
      bool stop = false;
      // S = Q_x K^T of key tile number i into S buffer `buf`
      auto issue_s = [&](int x, int buf, uint32_t i) -> bool {
        if (!wd.wait(&bars[L::bKFull + i % NK], (i / NK) & 1)) return false;
        tc_fence_after();
        const uint32_t q_addr = smem_u32(sm + L::kQ + x * kTB), k_addr = smem_u32(sm + L::kK + (i % NK) * kTB);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t off = (kk >> 2) * 16384 + (kk & 3) * 32;
          mma_ss(tmem + buf * 128, sw128_desc(q_addr + off, 16, 1024), sw128_desc(k_addr + off, 16, 1024), kIdescS,
                 kk > 0);
        }
        mma_commit(&bars[L::bSFull + buf]);
        return true;
      };
      // O_x += P V of key tile number i, P in S buffer `buf`
      auto issue_pv = [&](int x, int buf, uint32_t i, bool first) -> bool {
        if (!wd.wait(&bars[L::bPFull + buf], (NX == 1 ? i >> 1 : i) & 1)) return false;
        tc_fence_after();
        const uint32_t v_addr = smem_u32(sm + L::kV + (i % NV) * kTB);
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)
          mma_ts(tmem + 256 + x * D, tmem + buf * 128 + kk * 8, sw128_desc(v_addr + kk * 2048, 16384, 1024), kIdescPV,
                 (!first || kk > 0) ? 1u : 0u);
        mma_commit(&bars[L::bPVDone + x]);
        return true;
      };
      while (!stop && w.next(p.cache, p.tok)) {
        const int nt = w.t1 - w.t0;
        for (int x = 0; x < NX && !stop; ++x) {
          if (!wd.wait(&bars[L::bQFull + x], w.index & 1)) stop = true;
          tc_fence_after();
          if (!stop && !issue_s(x, NX == 1 ? kv & 1 : x, kv)) stop = true;
        }
        if (stop) break;
        mma_commit(&bars[L::bKEmpty + kv % NK]);
        for (int j = 0; j < nt; ++j, ++kv) {
          const bool more = j + 1 < nt;
          if constexpr (NX == 1) {
            // the other S buffer: its P (tile kv - 1) is read by MMAs issued before
            if (more) {
              if (!issue_s(0, (kv + 1) & 1, kv + 1)) { stop = true; break; }
              mma_commit(&bars[L::bKEmpty + (kv + 1) % NK]);
            }
            if (!wd.wait(&bars[L::bVFull + kv % NV], (kv / NV) & 1)) { stop = true; break; }
            if (!issue_pv(0, kv & 1, kv, j == 0)) { stop = true; break; }
          } else {
            if (!wd.wait(&bars[L::bVFull + kv % NV], (kv / NV) & 1)) { stop = true; break; }
            for (int x = 0; x < NX; ++x) {
              if (!issue_pv(x, x, kv, j == 0)) { stop = true; break; }
              if (more && !issue_s(x, x, kv + 1)) { stop = true; break; }
            }
            if (stop) break;
            if (more) mma_commit(&bars[L::bKEmpty + (kv + 1) % NK]);
          }
          mma_commit(&bars[L::bVEmpty + kv % NV]);
        }
      }
      mma_commit(&bars[L::bFinal]);
      drain_wait(&bars[L::bFinal], 0);
    }
  } else if (warp >= 4) {
    // ------------------------------------------------------------ softmax of row tile x
    const int x = (warp - 4) >> 2;
    const int quarter = warp & 3, r = quarter * 32 + lane;
    const uint32_t lane_off = static_cast<uint32_t>(quarter * 32) << 16;
    const uint32_t t_o = tmem + lane_off + 256 + x * D;
    const int G = p.tok.G;
    auto wwait = [&](uint64_t *bar, uint32_t parity) {
      return __all_sync(0xffffffffu, wd.wait(bar, parity)) != 0;
    };
    Walk<kTile * NX> w(p.cache, p.tok, run);
    uint32_t kv = 0;
    bool stop = false;
    while (!stop && w.next(p.cache, p.tok)) {
      const int row0 = (w.rg * NX + x) * kTile, rows = min(w.s.n * G - row0, kTile);
      const int row = row0 + r, tok = row / G, h = w.hk * G + row % G;
      const bool row_ok = r < rows, warp_on = quarter * 32 < rows;
      uint32_t *bad_w = bad + (w.index & 3) * 2;
      if (x == 0 && r == 0) {  // the next piece's words: their last readers are three pieces back
        bad[((w.index + 1) & 3) * 2] = 0;
        bad[((w.index + 1) & 3) * 2 + 1] = 0;
      }
      // Q rows -> shared memory (the last S of the piece before has read them), 16 bytes a lane
      constexpr int kPieces = D / 8;
#pragma unroll 4
      for (int i = r; i < kTile * kPieces; i += kTile) {
        const int rr = i / kPieces, c = i % kPieces, grow = row0 + rr;
        if (rr < rows) {
          const int4 v = *reinterpret_cast<const int4 *>(p.q + w.b * p.qs[0] + (grow / G) * p.qs[1] +
                                                         (w.hk * G + grow % G) * p.qs[2] + c * 8);
          *reinterpret_cast<int4 *>(sm + L::kQ + x * kTB + (c >> 3) * 16384 + rr * 128 + (((c & 7) ^ (rr & 7)) << 4)) = v;
        }
      }
      fence_proxy_async_smem();
      mbar_arrive(&bars[L::bQFull + x]);
      const uint64_t word = row_ok ? tree_word(p.tok, w.b, tok, w.s.n) : 0ull;
      float m_ref = -INFINITY, l = 0.f, l_r = 0.f;

      for (int t = w.t0; t < w.t1; ++t, ++kv) {
        const int buf = NX == 1 ? kv & 1 : x;
        const uint32_t t_s = tmem + lane_off + buf * 128;
        const int j0 = t * kTile;
        const bool edge = j0 + kTile > w.s.len;
        uint32_t allow[4] = {~0u, ~0u, ~0u, ~0u};
        if (edge) {
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const int d0 = j0 + 32 * q - w.s.len;  // the new token of the word's bit 0
            if (d0 >= 64) allow[q] = 0u;
            else if (d0 >= 0) allow[q] = static_cast<uint32_t>(word >> d0);
            else if (d0 > -32) allow[q] = static_cast<uint32_t>(word << -d0) | ((1u << -d0) - 1u);
          }
          if (x == 0) {
            // this thread's key: V past the new tokens becomes zero, what is not
            // finite in a new token's V is taken out
            if (!wwait(&bars[L::bVFull + kv % NV], (kv / NV) & 1)) { stop = true; break; }
            uint8_t *vrow = sm + L::kV + (kv % NV) * kTB + r * 128;
            const int d = j0 + r - w.s.len;
            if (d >= 0) {
              bool found = false;
#pragma unroll 1
              for (int c = 0; c < kPieces; ++c) {
                int4 *q4 = reinterpret_cast<int4 *>(vrow + (c >> 3) * 16384 + (((c & 7) ^ (r & 7)) << 4));
                int4 v = make_int4(0, 0, 0, 0);
                if (d < w.s.n) {
                  v = *q4;
                  const uint32_t n0 = not_finite<FP16>(v.x), n1 = not_finite<FP16>(v.y), n2 = not_finite<FP16>(v.z),
                                 n3 = not_finite<FP16>(v.w);
                  if ((n0 | n1 | n2 | n3) == 0u) continue;
                  found = true;
                  v = make_int4(v.x & ~n0, v.y & ~n1, v.z & ~n2, v.w & ~n3);
                }
                *q4 = v;
              }
              if (found) atomicOr(bad_w + (d >> 5), 1u << (d & 31));
              fence_proxy_async_smem();
            }
          }
        }
        if (!wwait(&bars[L::bSFull + buf], (NX == 1 ? kv >> 1 : kv) & 1)) { stop = true; break; }
        tc_fence_after();
        if (warp_on) {
          float mx = -INFINITY;
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            uint32_t sv[32];
            tmem_ld32(t_s + 32 * c, sv);
            tmem_wait_ld();
            if (edge) {
#pragma unroll
              for (int q = 0; q < 32; ++q)
                mx = fmaxf(mx, ((allow[c] >> q) & 1u) ? __uint_as_float(sv[q]) : -INFINITY);
            } else {
#pragma unroll
              for (int q = 0; q < 32; ++q) mx = fmaxf(mx, __uint_as_float(sv[q]));
            }
          }
          const float mt = mx * p.scale_log2;
          const bool need = mt > m_ref + kRescaleThreshold;
          const bool resc = need && l > 0.f;
          float alpha = 1.f;
          if (need) {
            alpha = fast_exp2(m_ref - mt);
            l *= alpha;
            l_r *= alpha;
            m_ref = mt;
          }
          if (__any_sync(0xffffffffu, resc)) {
            // every PV so far is in O (resc: this piece has had one)
            if (!wwait(&bars[L::bPVDone + x], (kv - 1) & 1)) { stop = true; break; }
            tc_fence_after();
            const float a = resc ? alpha : 1.f;
#pragma unroll
            for (int c = 0; c < D / 32; ++c) {
              uint32_t o[32];
              tmem_ld32(t_o + c * 32, o);
              tmem_wait_ld();
#pragma unroll
              for (int q = 0; q < 32; ++q) o[q] = __float_as_uint(__uint_as_float(o[q]) * a);
              tmem_st32(t_o + c * 32, o);
            }
            tmem_wait_st();
          }
          // P = exp2(s * scale * log2e - m) as 16-bit over the first 64 S columns.  l sums the exact weights
          // (for the LSE), l_r the rounded ones that the product uses (they normalise O, so that numerator and
          // denominator carry the same rounding)
          const float mu = m_ref == -INFINITY ? 0.f : m_ref;
          const float2 sc2 = make_float2(p.scale_log2, p.scale_log2), nmu = make_float2(-mu, -mu);
          float2 rs2 = make_float2(0.f, 0.f), rr2 = make_float2(0.f, 0.f);
          uint32_t svb[2][16];
          tmem_ld16(t_s, svb[0]);
          tmem_wait_ld();
#pragma unroll
          for (int sc = 0; sc < 8; ++sc) {
            if (sc + 1 < 8) tmem_ld16(t_s + 16 * (sc + 1), svb[(sc + 1) & 1]);
            const uint32_t *sv = svb[sc & 1];
            const uint32_t bits = allow[sc >> 1] >> (16 * (sc & 1));
            uint32_t pk[8];
#pragma unroll
            for (int q = 0; q < 8; ++q) {
              const float2 e = __ffma2_rn(make_float2(__uint_as_float(sv[2 * q]), __uint_as_float(sv[2 * q + 1])), sc2, nmu);
              float p0 = fast_exp2(e.x), p1 = fast_exp2(e.y);
              if (edge) {
                p0 = ((bits >> (2 * q)) & 1u) ? p0 : 0.f;
                p1 = ((bits >> (2 * q + 1)) & 1u) ? p1 : 0.f;
              }
              pk[q] = pack16<FP16>(p0, p1);
              rs2 = __fadd2_rn(rs2, make_float2(p0, p1));
              rr2 = __fadd2_rn(rr2, unpack16<FP16>(pk[q]));
            }
            tmem_st8(t_s + 8 * sc, pk);
            if (sc + 1 < 8) tmem_wait_ld();
          }
          l += rs2.x + rs2.y;
          l_r += rr2.x + rr2.y;
          tmem_wait_st();
        }
        tc_fence_before();
        mbar_arrive(&bars[L::bPFull + buf]);
      }
      if (stop) break;
      // ---------------------------------------------------------- epilogue
      // NX = 1 issues S of the last tile before the PV of the one before it, so that PV may still run: its phase
      // first (a wait two phases ahead would pass at once)
      if (NX == 1 && w.t1 - w.t0 > 1 && !wwait(&bars[L::bPVDone + x], kv & 1)) break;
      if (!wwait(&bars[L::bPVDone + x], (kv - 1) & 1)) break;
      tc_fence_after();
      if (warp_on) {
        const uint32_t bad_lo = bad_w[0] & static_cast<uint32_t>(word), bad_hi = bad_w[1] & static_cast<uint32_t>(word >> 32);
        const bool any_bad = __any_sync(0xffffffffu, (bad_lo | bad_hi) != 0u);
        const float inv = w.whole ? (l_r > 0.f ? 1.f / l_r : 0.f) : 1.f;
        uint16_t *orow = p.out + w.b * p.os[0] + tok * p.os[1] + h * p.os[2];
        // a piece that starts this CTA's run goes to slot 0, one that ends it to slot 1
        const int64_t part = (static_cast<int64_t>(blockIdx.x) * 2 + (w.index > 0 ? 1 : 0)) * (kTile * NX) + x * kTile + r;
        float *prow = p.part_o + part * D;
        uint32_t ob[2][16];
        tmem_ld16(t_o, ob[0]);
        tmem_wait_ld();
#pragma unroll
        for (int c = 0; c < D / 16; ++c) {
          if (c + 1 < D / 16) tmem_ld16(t_o + (c + 1) * 16, ob[(c + 1) & 1]);
          uint32_t *o = ob[c & 1];
          if (any_bad) {
            // the seen tokens' infinities and NaN, in this row's 16 columns
            for (uint64_t todo = bad_lo | static_cast<uint64_t>(bad_hi) << 32; todo != 0ull; todo &= todo - 1) {
              const int s = w.s.len + __ffsll(static_cast<long long>(todo)) - 1, page = page_of(p.cache, w.b, s);
              if (page < 0) continue;
              const uint32_t *src = reinterpret_cast<const uint32_t *>(
                  p.cache.v + slot_offset(p.cache.vs, p.cache, page, s, w.hk) + c * 16);
#pragma unroll
              for (int q = 0; q < 8; ++q) {
                const uint32_t v = src[q], nf = not_finite<FP16>(v);
                const float2 f = unpack16<FP16>(v);
                if (nf & 0xffffu) o[2 * q] = __float_as_uint(__uint_as_float(o[2 * q]) + f.x);
                if (nf >> 16) o[2 * q + 1] = __float_as_uint(__uint_as_float(o[2 * q + 1]) + f.y);
              }
            }
            __syncwarp();
          }
          if (row_ok) {
            if (w.whole) {
              uint32_t wv[8];
#pragma unroll
              for (int q = 0; q < 8; ++q)
                wv[q] = pack16<FP16>(__uint_as_float(o[2 * q]) * inv, __uint_as_float(o[2 * q + 1]) * inv);
              int4 *dst = reinterpret_cast<int4 *>(orow + c * 16);
              dst[0] = make_int4(wv[0], wv[1], wv[2], wv[3]);
              dst[1] = make_int4(wv[4], wv[5], wv[6], wv[7]);
            } else {
              const uint32_t(&lo)[8] = *reinterpret_cast<const uint32_t(*)[8]>(o);
              const uint32_t(&hi)[8] = *reinterpret_cast<const uint32_t(*)[8]>(o + 8);
              st_global_v8(prow + c * 16, lo);
              st_global_v8(prow + c * 16 + 8, hi);
            }
          }
          if (c + 1 < D / 16) tmem_wait_ld();
        }
        tc_fence_before();
        if (row_ok) {
          if (w.whole) p.lse[(static_cast<int64_t>(w.b) * p.tok.H + h) * p.tok.T + tok] =
              l == 0.f ? -INFINITY : (m_ref + __log2f(l)) * kLn2;
          else p.part_ml[part] = make_float4(m_ref, l, l_r, 0.f);
        }
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Joins the pieces of the rows whose key tiles several runs share, one warp a
// row, the pieces in tile order:
//   M = max m_i, O = sum 2^(m_i - M) O_i / sum 2^(m_i - M) lr_i,
//   LSE = (M + log2 sum 2^(m_i - M) l_i) ln 2.
// Rows at or past n_new are written as 0 / -inf here.
template <bool FP16, int D, int NX>
__global__ void __launch_bounds__(256) k_attend_join(const AttendParams p, int ctas) {
  constexpr int E = D / 32;
  const int lane = threadIdx.x & 31;
  const int64_t rows = static_cast<int64_t>(p.cache.B) * p.tok.T * p.tok.H;
  const int64_t total = total_work<kTile * NX>(p.cache, p.tok, lane, false);
  bool waited = false;
  for (int64_t i = (static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x) >> 5; i < rows;
       i += static_cast<int64_t>(gridDim.x) * (blockDim.x >> 5)) {
    const int h = static_cast<int>(i % p.tok.H), t = static_cast<int>(i / p.tok.H % p.tok.T);
    const int b = static_cast<int>(i / p.tok.H / p.tok.T);
    const Seq<kTile * NX> s = sequence<kTile * NX>(p.cache, p.tok, b, false);
    uint16_t *orow = p.out + b * p.os[0] + t * p.os[1] + h * p.os[2] + lane * E;
    float *lse = p.lse + (static_cast<int64_t>(b) * p.tok.H + h) * p.tok.T + t;
    if (t >= s.n) {
#pragma unroll
      for (int e = 0; e < E; e += 2) *reinterpret_cast<uint32_t *>(orow + e) = 0u;
      if (lane == 0) *lse = -INFINITY;
      continue;
    }
    // this row's item in the list: [a, a + tiles)
    int64_t a = 0;
    for (int b0 = 0; b0 < b; b0 += 32)
      if (b0 + lane < b) a += sequence<kTile * NX>(p.cache, p.tok, b0 + lane, false).work(p.cache.H_kv);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) a += __shfl_xor_sync(0xffffffffu, a, d);
    const int hk = h / p.tok.G, row = t * p.tok.G + h % p.tok.G, rg = row / (kTile * NX);
    a += (static_cast<int64_t>(hk) * s.groups + rg) * s.tiles;
    // the run that holds list position x: the largest c with total c / ctas <= x
    auto run_of = [&](int64_t x) {
      int c = static_cast<int>(((x + 1) * ctas - 1) / total);
      return min(c, ctas - 1);
    };
    const int c0 = run_of(a), c1 = run_of(a + s.tiles - 1);
    if (c0 == c1) continue;  // one run did it all
    if (!waited) {
      pdl_wait();
      waited = true;
    }
    const int in = row - rg * kTile * NX;
    auto part_of = [&](int c) {
      const int slot = run_start(total, c, ctas) >= a ? 0 : 1;
      return (static_cast<int64_t>(c) * 2 + slot) * (kTile * NX) + in;
    };
    float M = -INFINITY;
    for (int c = c0 + lane; c <= c1; c += 32)
      if (run_start(total, c, ctas) < run_start(total, c + 1, ctas)) M = fmaxf(M, p.part_ml[part_of(c)].x);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, d));
    const float Mu = M == -INFINITY ? 0.f : M;
    float o[E], l = 0.f, l_r = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = 0.f;
#pragma unroll 4
    for (int c = c0; c <= c1; ++c) {
      if (run_start(total, c, ctas) >= run_start(total, c + 1, ctas)) continue;  // an empty run
      const int64_t part = part_of(c);
      const float4 ml = p.part_ml[part];
      const float f = exp2f(ml.x - Mu);
      l = fmaf(f, ml.y, l);
      l_r = fmaf(f, ml.z, l_r);
      const float *src = p.part_o + part * D + lane * E;
#pragma unroll
      for (int e = 0; e < E; e += 2) {
        const float2 v = *reinterpret_cast<const float2 *>(src + e);
        o[e] = fmaf(f, v.x, o[e]);
        o[e + 1] = fmaf(f, v.y, o[e + 1]);
      }
    }
    const float inv = l_r > 0.f ? 1.f / l_r : 0.f;
#pragma unroll
    for (int e = 0; e < E; e += 2) *reinterpret_cast<uint32_t *>(orow + e) = pack16<FP16>(o[e] * inv, o[e + 1] * inv);
    if (lane == 0) *lse = l == 0.f ? -INFINITY : (M + __log2f(l)) * kLn2;
  }
  // a grid that ends before the one it depends on would let the next kernel of the stream start early
  if (!waited) pdl_wait();
}

template <bool FP16, int D, int NX>
cudaError_t launch(const AttendParams &p, const CUtensorMap &tk, const CUtensorMap &tv, int ctas, cudaStream_t s) {
  using L = AttendSmem<D, NX>;
  static_assert(L::kAlloc <= 232448, "shared memory of one CTA");
  cudaError_t e = cudaFuncSetAttribute(k_attend<FP16, D, NX>, cudaFuncAttributeMaxDynamicSharedMemorySize, L::kAlloc);
  if (e != cudaSuccess) return e;
  count_launch(2);
  k_attend<FP16, D, NX><<<ctas, NX == 1 ? 256 : 384, L::kAlloc, s>>>(tk, tv, p);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  const int64_t rows = static_cast<int64_t>(p.cache.B) * p.tok.T * p.tok.H;
  const int64_t blocks = std::min<int64_t>((rows + 7) / 8, 4 * ctas);
  return launch_pdl(k_attend_join<FP16, D, NX>, dim3(static_cast<unsigned>(blocks)), dim3(256), 0, s, p, ctas);
}

}  // namespace

size_t attend_scratch_bytes(int D) {
  return static_cast<size_t>(2 * kMaxCtas) * (2 * kTile) * (static_cast<size_t>(D) * 4 + 16);
}

cudaError_t launch_attend(const AttendArgs &a, const CUtensorMap &tk, const CUtensorMap &tv, bool fp16, int sms,
                          cudaStream_t s) {
  AttendParams p{};
  p.cache = a.cache;
  p.tok = a.tok;
  p.q = a.q;
  p.out = a.out;
  for (int i = 0; i < 3; ++i) {
    p.qs[i] = a.qs[i];
    p.os[i] = a.os[i];
  }
  p.lse = a.lse;
  p.scale_log2 = a.scale * kLog2e;
  p.box_log = std::min(a.cache.page_log, 7);
  p.box_rows = 1 << p.box_log;
  p.part_ml = reinterpret_cast<float4 *>(a.scratch);
  p.part_o = reinterpret_cast<float *>(a.scratch + static_cast<size_t>(2 * kMaxCtas) * (2 * kTile) * 16);
  const int ctas = std::min(sms, kMaxCtas);
  // one row tile where it holds the rows; two share each key tile's load otherwise
  const bool two = a.tok.T * a.tok.G > kTile;
  if (a.cache.D == 64) {
    if (fp16) return two ? launch<true, 64, 2>(p, tk, tv, ctas, s) : launch<true, 64, 1>(p, tk, tv, ctas, s);
    return two ? launch<false, 64, 2>(p, tk, tv, ctas, s) : launch<false, 64, 1>(p, tk, tv, ctas, s);
  }
  if (fp16) return two ? launch<true, 128, 2>(p, tk, tv, ctas, s) : launch<true, 128, 1>(p, tk, tv, ctas, s);
  return two ? launch<false, 128, 2>(p, tk, tv, ctas, s) : launch<false, 128, 1>(p, tk, tv, ctas, s);
}

}  // namespace bsa
