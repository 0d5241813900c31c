// Accumulated attention weight of a paged cache's slots:
//   score[b, hk, j] += sum over rows r = (t, h) of the group that see j of
//                      exp(scale q_r . k_j - lse_r)
//
// The transposed product S^T = K Q^T puts a key in each TMEM lane and the group's
// rows in the columns, so a thread owns a key and adds its weights up in
// registers: no reduction across threads, no atomics, the same bits every time.
// Bound: HBM, one read of K (2 D bytes a key), up to about 170 rows a group; the
// exponentials past that (16 a clock and SM).
//
// One CTA per SM over an equal run of the (sequence, kv head, 128-key tile) list.
//   warp 0      TMA producer of K tiles, one box a page (as in the attention).
//   warp 1      tcgen05 issuer: S^T (128 keys x N rows, N <= 256) into one of two
//               256-column TMEM buffers, alternating.
//   warps 4-7, 8-11   the sums of the even and of the odd tiles; both load the
//               rows (up to 256 at a time: more rows walk the piece's tiles again,
//               adding to the same scores) and their -lse before a pass.
#include "runs.cuh"

namespace bsa {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr int kRows = 256;  // rows of one pass

struct WeighParams {
  CacheView cache;
  TokenView tok;
  const uint16_t *q;
  int64_t qs[3];
  const float *lse, *score_in;
  float *score_out;
  float scale_log2;
  int box_log;
};

template <int D>
struct WeighSmem {
  static constexpr int kTB = kTile * D * 2;
  static constexpr int NK = D == 128 ? 4 : 8;
  static constexpr int kQ = 0, kK = kRows * D * 2, kBar = kK + NK * kTB;
  static constexpr int bKFull = 0, bKEmpty = NK, bSFull = 2 * NK, bSEmpty = bSFull + 2, bQFull = bSEmpty + 2,
                       bFinal = bQFull + 1, kNumBars = bFinal + 1;
  static constexpr int kLse = kBar + ((kNumBars * 8 + 15) & ~15);  // float [kRows] -lse * log2e
  static constexpr int kWord = kLse + kRows * 4;                    // uint32 [2][kRows] tree words, low and high
  static constexpr int kRun = kWord + kRows * 8;
  static constexpr int kMisc = kRun + 16;
  static constexpr int kAlloc = kMisc + 16;
};

template <bool FP16, int D>
__global__ void __launch_bounds__(384, 1) k_weigh(const __grid_constant__ CUtensorMap tk, const WeighParams p) {
  using L = WeighSmem<D>;
  extern __shared__ __align__(1024) uint8_t sm[];
  uint64_t *bars = reinterpret_cast<uint64_t *>(sm + L::kBar);
  float *nlse = reinterpret_cast<float *>(sm + L::kLse);
  uint32_t *words = reinterpret_cast<uint32_t *>(sm + L::kWord);
  RunStart *run_sm = reinterpret_cast<RunStart *>(sm + L::kRun);
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(sm + L::kMisc);
  int *abort_flag = reinterpret_cast<int *>(sm + L::kMisc + 4);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  constexpr int kTB = L::kTB, NK = L::NK;

  if (threadIdx.x == 32) {
    for (int i = 0; i < L::kNumBars; ++i) mbar_init(&bars[i], i >= L::bSEmpty && i < L::bSEmpty + 2 ? 128 : 1);
    *abort_flag = 0;
    fence_mbar_init();
    fence_proxy_async_smem();
  }
  if (warp == 0) {
    if (lane == 0) tma_prefetch_desc(&tk);
    const int64_t total = total_work<kAllRows>(p.cache, p.tok, lane, blockIdx.x == 0);
    const int64_t a = run_start(total, blockIdx.x, gridDim.x), z = run_start(total, blockIdx.x + 1, gridDim.x);
    const RunStart r = z > a ? find_start<kAllRows>(p.cache, p.tok, a, static_cast<int>(z - a), lane) : RunStart{0, 0, 0, 0};
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
  const uint32_t tmem = *tmem_slot;
  Watchdog wd{abort_flag, p.cache.status, kWaitLimitNs};
  const RunStart run = *run_sm;
  if (threadIdx.x == 0 && (smem_u32(sm) & 1023u) != 0u) wd.trip(BSA_ERR_UNSUPPORTED);
  __syncthreads();
  const int G = p.tok.G;
  auto passes = [&](const Walk<kAllRows> &w) { return max(1, (w.s.n * G + kRows - 1) / kRows); };

  if (wd.aborted()) {
  } else if (warp == 0) {
    // ------------------------------------------------------------ producer
    Walk<kAllRows> w(p.cache, p.tok, run);
    uint32_t kv = 0;
    bool stop = false;
    const int first = lane << p.box_log;
    while (!stop && w.next(p.cache, p.tok)) {
      for (int pass = passes(w); pass > 0 && !stop; --pass) {
        int page_next = box_page(p.cache, w, w.t0, first);
        for (int t = w.t0; t < w.t1; ++t, ++kv) {
          const int page = page_next, row = (t * kTile + first) & ((1 << p.cache.page_log) - 1);
          if (t + 1 < w.t1) page_next = box_page(p.cache, w, t + 1, first);
          const uint32_t ks = kv % NK;
          const bool ok = kv < NK || wd.wait(&bars[L::bKEmpty + ks], ((kv / NK) - 1) & 1);
          if (!__all_sync(0xffffffffu, ok)) { stop = true; break; }
          if (lane == 0) mbar_arrive_expect_tx(&bars[L::bKFull + ks], kTB);
          __syncwarp();
          if (first < kTile) {
#pragma unroll
            for (int c = 0; c < D / 64; ++c)
              tma_load_4d(sm + L::kK + ks * kTB + c * 16384 + first * 128, &tk, &bars[L::bKFull + ks], c * 64, row, w.hk,
                          page);
          }
        }
      }
    }
    if (wd.aborted())
      for (uint32_t t = (kv > NK ? kv - NK : 0); t < kv; ++t) drain_wait(&bars[L::bKFull + t % NK], (t / NK) & 1);
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    if (lane == 0) {
      Walk<kAllRows> w(p.cache, p.tok, run);
      uint32_t kv = 0, loads = 0;
      bool stop = false;
      const uint32_t q_addr = smem_u32(sm + L::kQ);
      while (!stop && w.next(p.cache, p.tok)) {
        for (int pass = 0; pass < passes(w) && !stop; ++pass, ++loads) {
          const int rows = min(w.s.n * G - pass * kRows, kRows), N = max((rows + 15) & ~15, 16);
          const uint32_t idesc = FP16 ? idesc_f16_f32(128, N, 0, 0) : idesc_bf16_f32(128, N, 0, 0);
          if (!wd.wait(&bars[L::bQFull], loads & 1)) { stop = true; break; }
          tc_fence_after();
          for (int t = w.t0; t < w.t1; ++t, ++kv) {
            const uint32_t buf = kv & 1;
            if (!wd.wait(&bars[L::bKFull + kv % NK], (kv / NK) & 1)) { stop = true; break; }
            if (kv >= 2 && !wd.wait(&bars[L::bSEmpty + buf], ((kv >> 1) - 1) & 1)) { stop = true; break; }
            tc_fence_after();
            const uint32_t k_addr = smem_u32(sm + L::kK + (kv % NK) * kTB);
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk)
              mma_ss(tmem + buf * 256, sw128_desc(k_addr + (kk >> 2) * 16384 + (kk & 3) * 32, 16, 1024),
                     sw128_desc(q_addr + (kk >> 2) * (kRows * 128) + (kk & 3) * 32, 16, 1024), idesc, kk > 0);
            mma_commit(&bars[L::bSFull + buf]);
            mma_commit(&bars[L::bKEmpty + kv % NK]);
          }
        }
      }
      mma_commit(&bars[L::bFinal]);
      drain_wait(&bars[L::bFinal], 0);
    }
  } else if (warp >= 4) {
    // ------------------------------------------------------------ sums
    const uint32_t y = (warp - 4) >> 2;  // the tiles with kv mod 2 == y
    const int r = (warp & 3) * 32 + lane, th = threadIdx.x - 128;
    const uint32_t t_s = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + y * 256;
    auto wwait = [&](uint64_t *bar, uint32_t parity) {
      return __all_sync(0xffffffffu, wd.wait(bar, parity)) != 0;
    };
    Walk<kAllRows> w(p.cache, p.tok, run);
    uint32_t kv = 0;
    bool stop = false;
    while (w.next(p.cache, p.tok)) {
      const int64_t base = (static_cast<int64_t>(w.b) * p.cache.H_kv + w.hk) * p.cache.capacity;
      for (int pass = 0; pass < passes(w); ++pass) {
        const int row0 = pass * kRows, rows = min(w.s.n * G - row0, kRows);
        // the rows of this pass -> shared memory, once both halves are done with the last pass (after a timeout too:
        // the barriers pair up in every path)
        named_bar_sync(1, 256);
        constexpr int kPieces = D / 8;
        const int padded = max((rows + 15) & ~15, 16);
#pragma unroll 4
        for (int i = th; i < padded * kPieces; i += 256) {
          const int rr = i / kPieces, c = i % kPieces, grow = row0 + rr;
          int4 v = make_int4(0, 0, 0, 0);
          if (rr < rows)
            v = *reinterpret_cast<const int4 *>(p.q + w.b * p.qs[0] + (grow / G) * p.qs[1] +
                                                (w.hk * G + grow % G) * p.qs[2] + c * 8);
          *reinterpret_cast<int4 *>(sm + L::kQ + (c >> 3) * (kRows * 128) + rr * 128 + (((c & 7) ^ (rr & 7)) << 4)) = v;
        }
        {
          const int grow = row0 + th, tok = grow / G, h = w.hk * G + grow % G;
          float z = -INFINITY;
          uint64_t word = 0;
          if (th < rows) {
            const float x = p.lse[(static_cast<int64_t>(w.b) * p.tok.H + h) * p.tok.T + tok];
            z = x == -INFINITY ? -INFINITY : -x * kLog2e;
            word = tree_word(p.tok, w.b, tok, w.s.n);
          }
          nlse[th] = z;
          words[th] = static_cast<uint32_t>(word);
          words[kRows + th] = static_cast<uint32_t>(word >> 32);
        }
        fence_proxy_async_smem();
        named_bar_sync(2, 256);
        if (th == 0) mbar_arrive(&bars[L::bQFull]);
        for (int t = w.t0; t < w.t1; ++t, ++kv) {
          if ((kv & 1) != y || stop) continue;
          const int j = t * kTile + r, d = j - w.s.len;  // this thread's slot; a new token where d >= 0
          const bool live = d < w.s.n;
          float before = 0.f;
          if (live) before = pass == 0 ? p.score_in[base + j] : p.score_out[base + j];
          if (!wwait(&bars[L::bSFull + y], (kv >> 1) & 1)) { stop = true; continue; }
          tc_fence_after();
          const bool edge = t * kTile + kTile > w.s.len;
          const float2 sc2 = make_float2(p.scale_log2, p.scale_log2);
          float2 acc0 = make_float2(0.f, 0.f), acc1 = acc0;
          uint32_t sv[2][16];
          tmem_ld16(t_s, sv[0]);
          tmem_wait_ld();
          for (int c0 = 0; c0 < rows; c0 += 32) {
#pragma unroll
            for (int half = 0; half < 2; ++half) {
              const int c = c0 + 16 * half;
              if (c < rows) {
                if (c + 16 < rows) tmem_ld16(t_s + c + 16, sv[half ^ 1]);
                const uint32_t *s = sv[half];
                if (!edge && c + 16 <= rows) {
#pragma unroll
                  for (int q = 0; q < 4; ++q) {
                    const float4 z = *reinterpret_cast<const float4 *>(nlse + c + 4 * q);
                    const float2 e0 = __ffma2_rn(make_float2(__uint_as_float(s[4 * q]), __uint_as_float(s[4 * q + 1])), sc2,
                                                 make_float2(z.x, z.y));
                    const float2 e1 = __ffma2_rn(make_float2(__uint_as_float(s[4 * q + 2]), __uint_as_float(s[4 * q + 3])),
                                                 sc2, make_float2(z.z, z.w));
                    acc0 = __fadd2_rn(acc0, make_float2(fast_exp2(e0.x), fast_exp2(e0.y)));
                    acc1 = __fadd2_rn(acc1, make_float2(fast_exp2(e1.x), fast_exp2(e1.y)));
                  }
                } else {
                  // columns past the rows, and rows that do not see this new token, add nothing whatever they hold
#pragma unroll
                  for (int q = 0; q < 16; ++q) {
                    const uint32_t wd32 = words[(d >= 32 ? kRows : 0) + c + q];
                    const bool on = c + q < rows && nlse[c + q] != -INFINITY && (d < 0 || ((wd32 >> (d & 31)) & 1u));
                    const float e = fast_exp2(fmaf(__uint_as_float(s[q]), p.scale_log2, nlse[c + q]));
                    acc0.x += on ? e : 0.f;
                  }
                }
                if (c + 16 < rows) tmem_wait_ld();
              }
            }
          }
          tc_fence_before();
          mbar_arrive(&bars[L::bSEmpty + y]);
          if (live) p.score_out[base + j] = before + ((acc0.x + acc1.x) + (acc0.y + acc1.y));
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

template <bool FP16, int D>
cudaError_t launch(const WeighParams &p, const CUtensorMap &tk, int ctas, cudaStream_t s) {
  using L = WeighSmem<D>;
  static_assert(L::kAlloc <= 232448, "shared memory of one CTA");
  const cudaError_t e = cudaFuncSetAttribute(k_weigh<FP16, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, L::kAlloc);
  if (e != cudaSuccess) return e;
  count_launch();
  k_weigh<FP16, D><<<ctas, 384, L::kAlloc, s>>>(tk, p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_weigh(const WeighArgs &a, const CUtensorMap &tk, bool fp16, int sms, cudaStream_t s) {
  WeighParams p{};
  p.cache = a.cache;
  p.tok = a.tok;
  p.q = a.q;
  for (int i = 0; i < 3; ++i) p.qs[i] = a.qs[i];
  p.lse = a.lse;
  p.score_in = a.score_in;
  p.score_out = a.score_out;
  p.scale_log2 = a.scale * kLog2e;
  p.box_log = std::min(a.cache.page_log, 7);
  if (a.cache.D == 64) return fp16 ? launch<true, 64>(p, tk, sms, s) : launch<false, 64>(p, tk, sms, s);
  return fp16 ? launch<true, 128>(p, tk, sms, s) : launch<false, 128>(p, tk, sms, s);
}

}  // namespace bsa
