// Attention of a few new tokens (a tree of drafted tokens, or one) over a paged
// cache: O = softmax(scale q K^T) V and the LSE, row (token t, head h) seeing
// the slots below length and the new tokens of its tree word.
//
// The T * G rows of a kv head's group (row = t * G + g) share its keys, so K and
// V are read once for up to 256 of them: one or two 128-row tiles (NX) against
// 128-key tiles.  Up to about 200 rows the floor is HBM (4 D bytes a key): 6.4 TB/s
// at 4 sequences x 1 token, 40 heads on 8, over 65536 keys (166 us), 5.5 at 16 x 32
// tokens, 16 on 4, over up to 33002 (152 us; called among others with inputs that
// change 178); at 256 rows 880 TFLOP/s (4 x 64 tokens, 32 on 8, 65536 keys, 310 us).
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
//               the S columns).
//   warps 4-7, 8-11   two softmax groups, one row a thread with its 128 scores in
//               registers (224 a thread, from the other warps' share): the tile's
//               maximum (P and the sums are relative to it, less kLift), lazy
//               rescale of O, P as 16-bit.  Where the piece has two row tiles,
//               each group has one; where it has one, the groups take
//               the key tiles in turn, each with its own running maximum, sums and
//               O, and add the two up in the epilogue, each for half the columns
//               (one group alone left the tensor and load pipes waiting for its
//               chain of latencies and took 1.26 times as long, 16 sequences x 32
//               tokens x 4 heads a group over 33002 keys; key tiles taken as two
//               halves, to overlap more, spent more on the barriers: 1.23 times
//               at 24000 keys).
// V of what no row may see (0 * NaN is NaN in the product): infinities and NaN past
// the new tokens are taken out of the tile in shared memory, and so are those of a
// new token, which the epilogue of the rows that see the token adds back.
// TMEM columns: S_0 [0,128) S_1 [128,256) O_0 [256,256+D) O_1 [256+D,256+2D).
#include "runs.cuh"

namespace bsa {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
// Up to this capacity a CTA takes its rows' whole sequence, padding rows too, and
// nothing is joined: four key tiles one after the other take less than a second
// launch (8 sequences x 1 token over 400 keys: 12.4 us with it, 11.4 without).
constexpr int kWholeSlots = 512;
constexpr float kRescaleThreshold = 8.0f;  // log2 units: tolerate p up to 2^8 times what it is lifted to
// log2 of the P that a running maximum's own key gets: in fp16 the largest P is 2^15, of 2^16 that it holds, so
// that what rounds to zero are weights below 2^-32 of the heaviest (2^-25 where P starts at 1: a few percent of V
// over 2^21 keys that lie 18 under one heavy key, which their LSE counts)
template <bool FP16>
constexpr float kLift = FP16 ? 7.0f : 0.0f;

struct AttendParams {
  CacheView cache;
  TokenView tok;
  const uint16_t *q;
  uint16_t *out;
  int64_t qs[3], os[3];
  float *lse;
  float scale_log2;
  int box_log;            // log2 of the keys of one TMA box: min(page_size, 128)
  float *part_o;          // [2 * CTAs, 128 * NX, D] unnormalised O of the pieces
  float4 *part_ml;        // [2 * CTAs, 128 * NX] reference (log2: the maximum less kLift), sum, sum of rounded weights
};

template <int D, int NX>
struct AttendSmem {
  static constexpr int kTB = kTile * D * 2;
  static constexpr int NK = D == 128 ? 3 : 5, NV = D == 128 ? (NX == 1 ? 3 : 2) : 5;
  static constexpr int kQ = 0, kK = NX * kTB, kV = kK + NK * kTB, kBar = kV + NV * kTB;
  static constexpr int bKFull = 0, bKEmpty = NK, bVFull = 2 * NK, bVEmpty = bVFull + NV, bQFull = bVEmpty + NV,
                       bSFull = bQFull + 1, bPFull = bSFull + 2, bPVDone = bPFull + 2, bQEmpty = bPVDone + 2,
                       bFinal = bQEmpty + 1,
                       kNumBars = bFinal + 1;
  static constexpr int kBad = kBar + kNumBars * 8;     // uint32 [4][2]: new tokens whose V is not finite
  static constexpr int kRun = kBad + 32;               // RunStart
  static constexpr int kMisc = kRun + 16;              // tmem slot, abort flag
  // for the other group, where the groups take the key tiles in turn: maximum and rounded sum of group 0's rows; maximum, sum and rounded sum of group 1's
  static constexpr int kSums = kMisc + 16;
  static constexpr int kAlloc = kSums + 5 * kTile * 4;
};

// Mask of the 16-bit halves of `w` that are infinite or NaN.
template <bool FP16>
__device__ __forceinline__ uint32_t not_finite(uint32_t w) {
  constexpr uint32_t e = FP16 ? 0x7c00u : 0x7f80u;
  return ((w & e) == e ? 0xffffu : 0u) | ((w & (e << 16)) == (e << 16) ? 0xffff0000u : 0u);
}

template <bool FP16, int D, int NX, bool WHOLE>
__global__ void __launch_bounds__(384, 1)
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
      mbar_init(&bars[i], i == L::bQFull ? 256 : i >= L::bPFull && i < L::bPFull + 2 ? 128 : 1);
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
    pdl_wait();  // everything before this may run under the stream's preceding kernel
    const RunStart r = find_run<kTile * NX, WHOLE>(p.cache, p.tok, lane);
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
  pdl_wait();
  // only the join may start under this kernel: another's kernel may not expect it
  if (!WHOLE) pdl_trigger();
  const uint32_t tmem = *tmem_slot;
  Watchdog wd{abort_flag, p.cache.status, kWaitLimitNs};
  const RunStart run = *run_sm;
  if (threadIdx.x == 0 && (smem_u32(sm) & 1023u) != 0u) wd.trip(BSA_ERR_UNSUPPORTED);
  __syncthreads();

  // row tiles of a piece with rows in them
  auto row_tiles = [&](const Walk<kTile * NX, WHOLE> &w) {
    return NX == 1 || w.s.n * p.tok.G - w.rg * kTile * NX <= kTile ? 1 : 2;
  };
  constexpr uint32_t kIdescS = FP16 ? idesc_f16_f32(128, 128, 0, 0) : idesc_bf16_f32(128, 128, 0, 0);
  constexpr uint32_t kIdescPV = FP16 ? idesc_f16_f32(128, D, 0, 1) : idesc_bf16_f32(128, D, 0, 1);

  // the launch's 384 x 168 registers: 128 x 56 + 256 x 224
  if (warp < 4) {
  regs_dec<56>();
  if (wd.aborted()) {
  } else if (warp == 0) {
    // ------------------------------------------------------------ producer
    Walk<kTile * NX, WHOLE> w(p.cache, p.tok, run);
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
      Walk<kTile * NX, WHOLE> w(p.cache, p.tok, run);
      uint32_t kv = 0, used0 = 0, used1 = 0;  // key tiles done; tiles each group has had
      bool stop = false;
      // S_x = Q_q K^T of key tile number i
      auto issue_s = [&](int x, int q, uint32_t i) -> bool {
        if (!wd.wait(&bars[L::bKFull + i % NK], (i / NK) & 1)) return false;
        tc_fence_after();
        const uint32_t q_addr = smem_u32(sm + L::kQ + q * kTB), k_addr = smem_u32(sm + L::kK + (i % NK) * kTB);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t off = (kk >> 2) * 16384 + (kk & 3) * 32;
          mma_ss(tmem + x * 128, sw128_desc(q_addr + off, 16, 1024), sw128_desc(k_addr + off, 16, 1024), kIdescS,
                 kk > 0);
        }
        mma_commit(&bars[L::bSFull + x]);
        return true;
      };
      // O_x += P_x V of key tile number i
      auto issue_pv = [&](int x, uint32_t i, bool first) -> bool {
        if (!wd.wait(&bars[L::bPFull + x], (x == 0 ? used0 : used1) & 1)) return false;
        (x == 0 ? used0 : used1) += 1;
        tc_fence_after();
        const uint32_t v_addr = smem_u32(sm + L::kV + (i % NV) * kTB);
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)
          mma_ts(tmem + 256 + x * D, tmem + x * 128 + kk * 8, sw128_desc(v_addr + kk * 2048, 16384, 1024), kIdescPV,
                 (!first || kk > 0) ? 1u : 0u);
        mma_commit(&bars[L::bPVDone + x]);
        return true;
      };
      while (!stop && w.next(p.cache, p.tok)) {
        const int nt = w.t1 - w.t0;
        if (!wd.wait(&bars[L::bQFull], w.index & 1)) break;
        tc_fence_after();
        // an S follows the P V that reads P from its columns in issue order, so needs no wait for it
        if (row_tiles(w) == 1) {
          for (int j = 0; j < min(nt, 2) && !stop; ++j) {
            stop = !issue_s((kv + j) & 1, 0, kv + j);
            if (!stop) mma_commit(&bars[L::bKEmpty + (kv + j) % NK]);
          }
          if (nt <= 2) mma_commit(&bars[L::bQEmpty]);
          for (int j = 0; j < nt && !stop; ++j, ++kv) {
            if (!wd.wait(&bars[L::bVFull + kv % NV], (kv / NV) & 1)) { stop = true; break; }
            if (!issue_pv(kv & 1, kv, j < 2)) { stop = true; break; }
            mma_commit(&bars[L::bVEmpty + kv % NV]);
            if (j + 2 < nt) {
              if (!issue_s(kv & 1, 0, kv + 2)) { stop = true; break; }
              mma_commit(&bars[L::bKEmpty + (kv + 2) % NK]);
            }
            // the piece's last S is issued: Q's shared memory is free once it is done
            if (nt > 2 && j + 3 == nt) mma_commit(&bars[L::bQEmpty]);
          }
        } else {
          for (int x = 0; x < 2 && !stop && nt > 0; ++x) stop = !issue_s(x, x, kv);
          if (stop) break;
          if (nt > 0) mma_commit(&bars[L::bKEmpty + kv % NK]);
          if (nt <= 1) mma_commit(&bars[L::bQEmpty]);
          for (int j = 0; j < nt && !stop; ++j, ++kv) {
            if (!wd.wait(&bars[L::bVFull + kv % NV], (kv / NV) & 1)) { stop = true; break; }
            for (int x = 0; x < 2 && !stop; ++x) {
              stop = !issue_pv(x, kv, j == 0);
              if (!stop && j + 1 < nt) stop = !issue_s(x, x, kv + 1);
            }
            if (stop) break;
            mma_commit(&bars[L::bVEmpty + kv % NV]);
            if (j + 1 < nt) mma_commit(&bars[L::bKEmpty + (kv + 1) % NK]);
            if (j + 2 == nt) mma_commit(&bars[L::bQEmpty]);
          }
        }
      }
      mma_commit(&bars[L::bFinal]);
      drain_wait(&bars[L::bFinal], 0);
    }
  }
  } else {
    // ------------------------------------------------------------ softmax group x
    regs_inc<224>();
    const int x = (warp - 4) >> 2;
    const int quarter = warp & 3, r = quarter * 32 + lane;
    const uint32_t lane_off = static_cast<uint32_t>(quarter * 32) << 16;
    const uint32_t t_s = tmem + lane_off + x * 128, t_o = tmem + lane_off + 256 + x * D;
    const int G = p.tok.G;
    constexpr int kPieces = D / 8;
    auto wwait = [&](uint64_t *bar, uint32_t parity) {
      return __all_sync(0xffffffffu, wd.wait(bar, parity)) != 0;
    };
    Walk<kTile * NX, WHOLE> w(p.cache, p.tok, run);
    uint32_t kv = 0, used = 0;  // key tiles of the run so far, and this group's among them
    bool stop = wd.aborted();
    // a piece's Q rows -> shared memory, by both groups, 16 bytes a lane
    auto load_q = [&](const Walk<kTile * NX, WHOLE> &n) {
      const int row0 = n.rg * NX * kTile, rows = min(n.s.n * G - row0, kTile * NX);
#pragma unroll 4
      for (int i = threadIdx.x - 128; i < rows * kPieces; i += 256) {
        const int rr = i / kPieces, c = i % kPieces, grow = row0 + rr;
        const int4 v = *reinterpret_cast<const int4 *>(p.q + n.b * p.qs[0] + (grow / G) * p.qs[1] +
                                                       (n.hk * G + grow % G) * p.qs[2] + c * 8);
        *reinterpret_cast<int4 *>(sm + L::kQ + (rr >> 7) * kTB + (c >> 3) * 16384 + (rr & 127) * 128 +
                                  (((c & 7) ^ (rr & 7)) << 4)) = v;
      }
      fence_proxy_async_smem();
      mbar_arrive(&bars[L::bQFull]);
    };
    bool more = w.next(p.cache, p.tok);
    if (more && !stop) load_q(w);
    while (more) {
      const bool turns = row_tiles(w) == 1;  // the groups take the key tiles in turn; else each has a row tile
      const int row0 = w.rg * NX * kTile + (turns ? 0 : x * kTile), rows = min(w.s.n * G - row0, kTile);
      const int row = row0 + r, tok = row / G, h = w.hk * G + row % G;
      const bool row_ok = r < rows, warp_on = quarter * 32 < rows;
      uint32_t *bad_w = bad + (w.index & 3) * 2;
      if (x == 0 && r == 0) {  // the next piece's words: their last readers are three pieces back
        bad[((w.index + 1) & 3) * 2] = 0;
        bad[((w.index + 1) & 3) * 2 + 1] = 0;
      }
      const uint64_t word = row_ok ? tree_word(p.tok, w.b, tok, w.s.n) : 0ull;
      float m_ref = -INFINITY, l = 0.f, l_r = 0.f;

      for (int t = w.t0; t < w.t1 && !stop; ++t, ++kv) {
        if (turns && (kv & 1) != static_cast<uint32_t>(x)) continue;
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
        }
        if (!wwait(&bars[L::bSFull + x], used & 1)) { stop = true; break; }
        tc_fence_after();
        // After S: the products of the tiles that had this V stage before are done (they were issued before S), so
        // the stage's phase is this tile's.  (Waited for before S, it could still be at the tile before in the stage,
        // whose V this would have changed.)
        if (edge && (turns || x == 0)) {
          // this thread's key: what is not finite in V of a new token, or past them, is taken out
          if (!wwait(&bars[L::bVFull + kv % NV], (kv / NV) & 1)) { stop = true; break; }
          uint8_t *vrow = sm + L::kV + (kv % NV) * kTB + r * 128;
          const int d = j0 + r - w.s.len;
          if (d >= 0) {
            bool found = false;
#pragma unroll 8
            for (int c = 0; c < kPieces; ++c) {
              int4 *q4 = reinterpret_cast<int4 *>(vrow + (c >> 3) * 16384 + (((c & 7) ^ (r & 7)) << 4));
              const int4 v = *q4;
              const uint32_t n0 = not_finite<FP16>(v.x), n1 = not_finite<FP16>(v.y), n2 = not_finite<FP16>(v.z),
                             n3 = not_finite<FP16>(v.w);
              if ((n0 | n1 | n2 | n3) == 0u) continue;
              found = true;
              *q4 = make_int4(v.x & ~n0, v.y & ~n1, v.z & ~n2, v.w & ~n3);
            }
            if (found) {
              if (d < w.s.n) atomicOr(bad_w + (d >> 5), 1u << (d & 31));
              fence_proxy_async_smem();
            }
          }
          __syncwarp();
        }
        if (warp_on) {
          uint32_t sv[4][32];
#pragma unroll
          for (int c = 0; c < 4; ++c) tmem_ld32(t_s + 32 * c, sv[c]);
          tmem_wait_ld();
          if (edge) {
            // what this row does not see, whatever it holds
#pragma unroll
            for (int c = 0; c < 4; ++c)
#pragma unroll
              for (int q = 0; q < 32; ++q) sv[c][q] = ((allow[c] >> q) & 1u) ? sv[c][q] : 0xff800000u;
          }
          float mx4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int q = 0; q < 32; ++q)
#pragma unroll
            for (int c = 0; c < 4; ++c) mx4[c] = fmaxf(mx4[c], __uint_as_float(sv[c][q]));
          // (exponents as the weights below have them, one rounding: large scores' products lose whole powers of two)
          const float top = fmaxf(fmaxf(mx4[0], mx4[1]), fmaxf(mx4[2], mx4[3]));
          const float mt = fmaf(top, p.scale_log2, -kLift<FP16>);
          const bool need = fmaf(top, p.scale_log2, -m_ref) > kLift<FP16> + kRescaleThreshold;
          const bool resc = need && l > 0.f;
          float alpha = 1.f;
          if (need) {
            alpha = fast_exp2(m_ref - mt);
            l *= alpha;
            l_r *= alpha;
            m_ref = mt;
          }
          if (__any_sync(0xffffffffu, resc)) {
            // every PV of this group so far is in O (resc: this piece has had one)
            if (!wwait(&bars[L::bPVDone + x], (used - 1) & 1)) { stop = true; break; }
            tc_fence_after();
            const float a = resc ? alpha : 1.f;
#pragma unroll
            for (int c = 0; c < D / 16; ++c) {
              uint32_t o[16];
              tmem_ld16(t_o + c * 16, o);
              tmem_wait_ld();
#pragma unroll
              for (int q = 0; q < 16; ++q) o[q] = __float_as_uint(__uint_as_float(o[q]) * a);
              tmem_st16(t_o + c * 16, o);
            }
            tmem_wait_st();
          }
          // P = exp2(s * scale * log2e - m) as 16-bit over the first 64 S columns.  l sums the exact weights
          // (for the LSE), l_r the rounded ones that the product uses (they normalise O, so that numerator and
          // denominator carry the same rounding)
          const float mu = m_ref == -INFINITY ? 0.f : m_ref;
          const float2 sc2 = make_float2(p.scale_log2, p.scale_log2), nmu = make_float2(-mu, -mu);
          float2 rs2[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)}, rr2[2] = {rs2[0], rs2[0]};
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            uint32_t pk[16];
#pragma unroll
            for (int q = 0; q < 16; ++q) {
              const float2 e =
                  __ffma2_rn(make_float2(__uint_as_float(sv[c][2 * q]), __uint_as_float(sv[c][2 * q + 1])), sc2, nmu);
              const float2 pp = make_float2(fast_exp2(e.x), fast_exp2(e.y));
              pk[q] = pack16<FP16>(pp.x, pp.y);
              rs2[q & 1] = __fadd2_rn(rs2[q & 1], pp);
              rr2[q & 1] = __fadd2_rn(rr2[q & 1], unpack16<FP16>(pk[q]));
            }
            tmem_st16(t_s + 16 * c, pk);
          }
          l += (rs2[0].x + rs2[1].x) + (rs2[0].y + rs2[1].y);
          l_r += (rr2[0].x + rr2[1].x) + (rr2[0].y + rr2[1].y);
          tmem_wait_st();
        }
        tc_fence_before();
        mbar_arrive(&bars[L::bPFull + x]);
        ++used;
      }
      // the next piece's Q, so that its first S runs under this piece's epilogue
      Walk<kTile * NX, WHOLE> next = w;
      more = next.next(p.cache, p.tok);
      if (more && !stop) {
        if (wwait(&bars[L::bQEmpty], w.index & 1)) load_q(next);
        else stop = true;
      }
      // ---------------------------------------------------------- epilogue
      // (a group that has had no tile in the piece has nothing to wait for)
      const int nt = w.t1 - w.t0;
      const bool had = turns ? nt > 1 || (nt == 1 && ((kv - 1) & 1) == static_cast<uint32_t>(x)) : nt > 0;
      if (!stop && had && !wwait(&bars[L::bPVDone + x], (used - 1) & 1)) stop = true;
      tc_fence_after();
      float f_mine = 1.f, f_other = 0.f;
      const bool both = turns && nt > 1;
      {
        // the other group's maximum and sums, through shared memory
        float *sums = reinterpret_cast<float *>(sm + L::kSums);
        float *mine = sums + x * 2 * kTile, *other = sums + (x ^ 1) * 2 * kTile;
        mine[r] = m_ref;
        mine[kTile + r] = l_r;
        if (x == 1) mine[2 * kTile + r] = l;
        tc_fence_before();
        named_bar_sync(1, 256);  // in every path, so that the two groups' barriers pair up
        tc_fence_after();
        if (both) {
          const float mo = other[r], M = fmaxf(m_ref, mo), Mu = M == -INFINITY ? 0.f : M;
          f_mine = exp2f(m_ref - Mu);
          f_other = exp2f(mo - Mu);
          if (x == 0) l = f_mine * l + f_other * other[2 * kTile + r];
          l_r = f_mine * l_r + f_other * other[kTile + r];
          m_ref = M;
        }
      }
      if (!stop && warp_on && had) {
        const uint32_t bad_lo = bad_w[0] & static_cast<uint32_t>(word), bad_hi = bad_w[1] & static_cast<uint32_t>(word >> 32);
        const bool any_bad = __any_sync(0xffffffffu, (bad_lo | bad_hi) != 0u);
        const float inv = w.whole ? (l_r > 0.f ? 1.f / l_r : 0.f) : 1.f;
        f_mine *= inv;
        f_other *= inv;
        uint16_t *orow = p.out + w.b * p.os[0] + tok * p.os[1] + h * p.os[2];
        // a piece of the run's first item goes to slot 0, one of its last to slot 1
        const int64_t part = (static_cast<int64_t>(blockIdx.x) * 2 + w.slot) * (kTile * NX) +
                             (turns ? 0 : x * kTile) + r;
        float *prow = p.part_o + part * D;
        // the columns [c0, c1) * 32: half of them where both groups hold a part of the row
        const int c0 = both ? x * (D / 64) : 0, c1 = both ? c0 + D / 64 : D / 32;
#pragma unroll 1
        for (int c = c0; c < c1; ++c) {
          uint32_t o[32];
          tmem_ld32(t_o + c * 32, o);
          if (both) {
            uint32_t o2[32];
            tmem_ld32(tmem + lane_off + 256 + (x ^ 1) * D + c * 32, o2);
            tmem_wait_ld();
#pragma unroll
            for (int q = 0; q < 32; ++q)
              o[q] = __float_as_uint(__uint_as_float(o[q]) * f_mine + __uint_as_float(o2[q]) * f_other);
          } else {
            tmem_wait_ld();
#pragma unroll
            for (int q = 0; q < 32; ++q) o[q] = __float_as_uint(__uint_as_float(o[q]) * f_mine);
          }
          if (any_bad) {
            // the seen tokens' infinities and NaN, in this row's 32 columns
            for (uint64_t todo = bad_lo | static_cast<uint64_t>(bad_hi) << 32; todo != 0ull; todo &= todo - 1) {
              const int s = w.s.len + __ffsll(static_cast<long long>(todo)) - 1, page = page_of(p.cache, w.b, s);
              if (page < 0) continue;
              const uint32_t *src = reinterpret_cast<const uint32_t *>(
                  p.cache.v + slot_offset(p.cache.vs, p.cache, page, s, w.hk) + c * 32);
#pragma unroll
              for (int q = 0; q < 16; ++q) {
                const uint32_t v = src[q], nf = not_finite<FP16>(v);
                const float2 f = unpack16<FP16>(v);
                if (nf & 0xffffu) o[2 * q] = __float_as_uint(__uint_as_float(o[2 * q]) + f.x);
                if (nf >> 16) o[2 * q + 1] = __float_as_uint(__uint_as_float(o[2 * q + 1]) + f.y);
              }
            }
            __syncwarp();
          }
          if (row_ok) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              if (w.whole) {
                uint32_t wv[4];
#pragma unroll
                for (int q = 0; q < 4; ++q)
                  wv[q] = pack16<FP16>(__uint_as_float(o[8 * k + 2 * q]), __uint_as_float(o[8 * k + 2 * q + 1]));
                reinterpret_cast<int4 *>(orow + c * 32)[k] = make_int4(wv[0], wv[1], wv[2], wv[3]);
              } else {
                st_global_v8(prow + c * 32 + 8 * k, *reinterpret_cast<const uint32_t(*)[8]>(&o[8 * k]));
              }
            }
          }
          __syncwarp();
        }
        if (row_ok && !(both && x == 1)) {
          if (w.whole) p.lse[(static_cast<int64_t>(w.b) * p.tok.H + h) * p.tok.T + tok] =
              l == 0.f ? -INFINITY : (m_ref + __log2f(l)) * kLn2;
          else p.part_ml[part] = make_float4(m_ref, l, l_r, 0.f);
        }
      }
      // padding rows: those of this group's row tile, and of the other one where no row of it is real
      const int last = turns && NX == 2 && x == 1 ? kTile : 0;
      if (WHOLE && (turns ? x == 0 || NX == 2 : true) && row + last >= w.s.n * G && row + last < p.tok.T * G) {
        const int tok = (row + last) / G, h = w.hk * G + (row + last) % G;
        uint16_t *orow = p.out + w.b * p.os[0] + tok * p.os[1] + h * p.os[2];
#pragma unroll 1
        for (int c = 0; c < D / 8; ++c) reinterpret_cast<int4 *>(orow)[c] = make_int4(0, 0, 0, 0);
        p.lse[(static_cast<int64_t>(w.b) * p.tok.H + h) * p.tok.T + tok] = -INFINITY;
      }
      tc_fence_before();
      __syncwarp();
      // both groups have read both O's (and the sums) before either's next product writes them
      named_bar_sync(2, 256);
      w = next;
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Joins the pieces of the rows whose key tiles several runs share, the pieces in
// tile order:
//   M = max m_i, O = sum 2^(m_i - M) O_i / sum 2^(m_i - M) lr_i,
//   LSE = (M + log2 sum 2^(m_i - M) l_i) ln 2.
// A row is WARPS warps of a block, which share out its pieces (a long sequence
// alone on the GPU is in up to 148) and add their parts up in order, so the same
// lengths give the same bits.  Rows at or past n_new are written as 0 / -inf here.
template <bool FP16, int D, int NX, int WARPS>
__global__ void __launch_bounds__(256) k_attend_join(const AttendParams p, int ctas) {
  constexpr int E = D / 32, kRowsPerBlock = 8 / WARPS;
  __shared__ float part_sm[WARPS > 1 ? 8 : 1][D + 4];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, sub = warp % WARPS;
  const int64_t rows = static_cast<int64_t>(p.cache.B) * p.tok.T * p.tok.H;
  const int64_t i = static_cast<int64_t>(blockIdx.x) * kRowsPerBlock + warp / WARPS;
  const bool in = i < rows;
  const int h = in ? static_cast<int>(i % p.tok.H) : 0, t = in ? static_cast<int>(i / p.tok.H % p.tok.T) : 0;
  const int b = in ? static_cast<int>(i / p.tok.H / p.tok.T) : 0;
  uint32_t a;
  // (lengths and counts, before the wait: k_attend lets this kernel start only past its own wait, when what wrote
  // them is done)
  const Runs runs(total_work<kTile * NX>(p.cache, p.tok, lane, false, b, &a), ctas);
  const Seq<kTile * NX> s = sequence<kTile * NX>(p.cache, p.tok, b, false);
  uint16_t *orow = p.out + b * p.os[0] + t * p.os[1] + h * p.os[2] + lane * E;
  float *lse = p.lse + (static_cast<int64_t>(b) * p.tok.H + h) * p.tok.T + t;
  const bool padding = t >= s.n;
  uint32_t c0 = 0, c1 = 0, units = 0;
  int rg = 0;
  int64_t row_part = 0;
  // whether run c has key tiles of this row's item
  auto has = [&](uint32_t c) {
    const uint32_t z = min(runs.start(c + 1) - a, units), y = runs.start(c) > a ? runs.start(c) - a : 0u;
    return first_tile(s, y, rg) < first_tile(s, z, rg);
  };
  if (in && !padding) {
    // this row's item in the list: [a, a + units)
    const int hk = h / p.tok.G, row = t * p.tok.G + h % p.tok.G;
    rg = row / (kTile * NX);
    a += static_cast<uint32_t>(hk) * s.head_units() + s.group_start(rg);
    units = s.units(rg);
    c0 = runs.of(a);
    c1 = runs.of(a + units - 1);
    while (c0 < c1 && !has(c0)) ++c0;
    while (c1 > c0 && !has(c1)) --c1;
    row_part = row - rg * kTile * NX;
  }
  const bool joined = c0 != c1;  // else one run has written the row
  // a grid that ends before the one it depends on would let the next kernel of the
  // stream start early, so every warp waits
  pdl_wait();
  // the running maximum and sums, U pieces at a time with all their loads in flight (one
  // after the other they took 3 us here, most of it latency)
  constexpr int U = 4;
  float M = -INFINITY, l = 0.f, l_r = 0.f, o[E];
#pragma unroll
  for (int e = 0; e < E; ++e) o[e] = 0.f;
  auto scale = [&](float f) {
    l *= f;
    l_r *= f;
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] *= f;
  };
  if (joined) {
    const uint32_t n = c1 - c0 + 1, z = c0 + n * (sub + 1) / WARPS;
#pragma unroll 1
    for (uint32_t c = c0 + n * sub / WARPS; c < z; c += U) {
      float4 ml[U];
      float v[U][E];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const uint32_t cu = min(c + u, z - 1);
        // c0's piece is its run's last, unless the run starts there
        const int slot = runs.start(cu) >= a ? 0 : 1;
        const int64_t part = (static_cast<int64_t>(cu) * 2 + slot) * (kTile * NX) + row_part;
        ml[u] = p.part_ml[part];
        const float *src = p.part_o + part * D + lane * E;
#pragma unroll
        for (int e = 0; e < E; e += 2) *reinterpret_cast<float2 *>(&v[u][e]) = *reinterpret_cast<const float2 *>(src + e);
      }
      const float before = M;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (c + u >= z || !has(c + u)) {  // what is there is no piece of this call
          ml[u] = make_float4(-INFINITY, 0.f, 0.f, 0.f);
#pragma unroll
          for (int e = 0; e < E; ++e) v[u][e] = 0.f;
        }
        M = fmaxf(M, ml[u].x);
      }
      const float Mu = M == -INFINITY ? 0.f : M;
      scale(exp2f(before - Mu));
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const float f = exp2f(ml[u].x - Mu);
        l = fmaf(f, ml[u].y, l);
        l_r = fmaf(f, ml[u].z, l_r);
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] = fmaf(f, v[u][e], o[e]);
      }
    }
  }
  if constexpr (WARPS > 1) {
#pragma unroll
    for (int e = 0; e < E; ++e) part_sm[warp][lane * E + e] = o[e];
    if (lane == 0) {
      part_sm[warp][D] = l;
      part_sm[warp][D + 1] = l_r;
      part_sm[warp][D + 2] = M;
    }
    __syncthreads();
    if (sub != 0) return;
    const float mine = M;
#pragma unroll
    for (int x = 1; x < WARPS; ++x) M = fmaxf(M, part_sm[warp + x][D + 2]);
    const float Mu = M == -INFINITY ? 0.f : M;
    scale(exp2f(mine - Mu));
#pragma unroll
    for (int x = 1; x < WARPS; ++x) {
      const float f = exp2f(part_sm[warp + x][D + 2] - Mu);
#pragma unroll
      for (int e = 0; e < E; ++e) o[e] = fmaf(f, part_sm[warp + x][lane * E + e], o[e]);
      l = fmaf(f, part_sm[warp + x][D], l);
      l_r = fmaf(f, part_sm[warp + x][D + 1], l_r);
    }
  }
  if (!in || !(joined || padding)) return;
  const float inv = l_r > 0.f ? 1.f / l_r : (l_r == 0.f ? 0.f : l_r);
#pragma unroll
  for (int e = 0; e < E; e += 2)
    *reinterpret_cast<uint32_t *>(orow + e) = padding ? 0u : pack16<FP16>(o[e] * inv, o[e + 1] * inv);
  if (lane == 0) *lse = l == 0.f ? -INFINITY : (M + __log2f(l)) * kLn2;
}

template <bool FP16, int D, int NX, int WARPS>
cudaError_t join(const AttendParams &p, int ctas, cudaStream_t s) {
  constexpr int kRowsPerBlock = 8 / WARPS;
  const int64_t rows = static_cast<int64_t>(p.cache.B) * p.tok.T * p.tok.H;
  return launch_pdl(k_attend_join<FP16, D, NX, WARPS>, dim3(static_cast<unsigned>((rows + kRowsPerBlock - 1) / kRowsPerBlock)),
                    dim3(256), 0, s, p, ctas);
}

template <bool FP16, int D, int NX>
cudaError_t launch(const AttendParams &p, const CUtensorMap &tk, const CUtensorMap &tv, int ctas, cudaStream_t s) {
  using L = AttendSmem<D, NX>;
  static_assert(L::kAlloc <= 232448, "shared memory of one CTA");
  const int64_t items = static_cast<int64_t>(p.cache.B) * p.cache.H_kv * ((p.tok.T * p.tok.G + kTile * NX - 1) / (kTile * NX));
  if (p.cache.capacity <= kWholeSlots) {
    static std::atomic<uint64_t> done{0};
    const cudaError_t e = allow_smem(k_attend<FP16, D, NX, true>, L::kAlloc, done);
    if (e != cudaSuccess) return e;
    count_launch();
    return launch_pdl(k_attend<FP16, D, NX, true>, dim3(static_cast<unsigned>(std::min<int64_t>(items, ctas))), dim3(384),
                      L::kAlloc, s, tk, tv, p);
  }
  static std::atomic<uint64_t> done{0};
  cudaError_t e = allow_smem(k_attend<FP16, D, NX, false>, L::kAlloc, done);
  if (e != cudaSuccess) return e;
  count_launch(2);
  if ((e = launch_pdl(k_attend<FP16, D, NX, false>, dim3(ctas), dim3(384), L::kAlloc, s, tk, tv, p)) != cudaSuccess) return e;
  // an item's tiles lie in about ctas / items runs, a few more where lengths differ
  return ctas > 8 * items ? join<FP16, D, NX, 8>(p, ctas, s) : join<FP16, D, NX, 1>(p, ctas, s);
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
