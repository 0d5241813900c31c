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
//   warp 1      tcgen05 issuer: S^T (128 keys x up to 128 rows) into the TMEM
//               buffer of the group whose tile it is.
//   warps 4-19  four groups, each with every fourth tile and a 128-column buffer
//               of its own (two groups on 256 columns, reading 16 columns at a
//               time, left the exponential unit idle two thirds of the time: 137
//               us against 100 at 4 x 16 tokens x 5 heads a group, 75600 keys).
// Up to 256 rows are in shared memory, as two halves that a batch of four tiles
// takes one after the other; more rows walk the piece's tiles again, adding to
// the same scores.
#include "runs.cuh"

namespace bsa {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr int kRows = 256;   // rows of one pass
constexpr int kGroups = 4;   // groups of 128 threads, a thread a key
constexpr int kSumThreads = kGroups * kTile;
constexpr int kMaxTok = 64;

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
  static constexpr int NK = D == 128 ? 5 : 8;
  static constexpr int kQ = 0, kK = kRows * D * 2, kBar = kK + NK * kTB;
  static constexpr int bKFull = 0, bKEmpty = NK, bSFull = 2 * NK, bSEmpty = bSFull + kGroups, bQFull = bSEmpty + kGroups,
                       bFinal = bQFull + 1, kNumBars = bFinal + 1;
  static constexpr int kLse = kBar + ((kNumBars * 8 + 15) & ~15);  // float [kRows] -lse * log2e
  static constexpr int kWord = kLse + kRows * 4;                    // uint64 [kMaxTok] tree words
  static constexpr int kAlive = kWord + kMaxTok * 8;                // uint32 [kRows / 32] rows that add anything (lse > -inf)
  static constexpr int kRun = kAlive + kRows / 8;
  static constexpr int kMisc = kRun + 16;
  static constexpr int kAlloc = kMisc + 16;
};

template <bool FP16, int D>
__global__ void __launch_bounds__(128 + kSumThreads, 1) k_weigh(const __grid_constant__ CUtensorMap tk, const WeighParams p) {
  using L = WeighSmem<D>;
  extern __shared__ __align__(1024) uint8_t sm[];
  uint64_t *bars = reinterpret_cast<uint64_t *>(sm + L::kBar);
  float *nlse = reinterpret_cast<float *>(sm + L::kLse);
  uint64_t *words = reinterpret_cast<uint64_t *>(sm + L::kWord);
  uint32_t *alive = reinterpret_cast<uint32_t *>(sm + L::kAlive);
  RunStart *run_sm = reinterpret_cast<RunStart *>(sm + L::kRun);
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(sm + L::kMisc);
  int *abort_flag = reinterpret_cast<int *>(sm + L::kMisc + 4);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  constexpr int kTB = L::kTB, NK = L::NK;

  if (threadIdx.x == 32) {
    for (int i = 0; i < L::kNumBars; ++i) mbar_init(&bars[i], i >= L::bSEmpty && i < L::bSEmpty + kGroups ? kTile : 1);
    *abort_flag = 0;
    fence_mbar_init();
    fence_proxy_async_smem();
  }
  if (warp == 0) {
    if (lane == 0) tma_prefetch_desc(&tk);
    pdl_wait();  // everything before this may run under the stream's preceding kernel
    const RunStart r = find_run<kAllRows>(p.cache, p.tok, lane);
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
      uint32_t kv = 0, loads = 0, ever = 0, odd = 0;  // bit y: buffer y has been used, an odd number of times
      bool stop = false;
      const uint32_t q_addr = smem_u32(sm + L::kQ);
      while (!stop && w.next(p.cache, p.tok)) {
        for (int pass = 0; pass < passes(w) && !stop; ++pass, ++loads) {
          const int rows = min(w.s.n * G - pass * kRows, kRows), halves = rows > 128 ? 2 : 1;
          if (!wd.wait(&bars[L::bQFull], loads & 1)) { stop = true; break; }
          tc_fence_after();
          const int nt = w.t1 - w.t0;
          for (int j = 0; j < nt && !stop; j += kGroups) {
            const int batch = min(nt - j, kGroups);
            for (int half = 0; half < halves && !stop; ++half) {
              const int cols = min(rows - half * 128, 128), N = max((cols + 15) & ~15, 16);
              const uint32_t idesc = FP16 ? idesc_f16_f32(128, N, 0, 0) : idesc_bf16_f32(128, N, 0, 0);
              for (int i = 0; i < batch; ++i) {
                const uint32_t x = kv + i, y = x % kGroups;
                if (half == 0 && !wd.wait(&bars[L::bKFull + x % NK], (x / NK) & 1)) { stop = true; break; }
                if (((ever >> y) & 1u) && !wd.wait(&bars[L::bSEmpty + y], ((odd >> y) & 1u) ^ 1u)) { stop = true; break; }
                ever |= 1u << y;
                odd ^= 1u << y;
                tc_fence_after();
                const uint32_t k_addr = smem_u32(sm + L::kK + (x % NK) * kTB);
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk)
                  mma_ss(tmem + y * 128, sw128_desc(k_addr + (kk >> 2) * 16384 + (kk & 3) * 32, 16, 1024),
                         sw128_desc(q_addr + half * 16384 + (kk >> 2) * (kRows * 128) + (kk & 3) * 32, 16, 1024), idesc,
                         kk > 0);
                mma_commit(&bars[L::bSFull + y]);
                if (half == halves - 1) mma_commit(&bars[L::bKEmpty + x % NK]);
              }
            }
            kv += batch;
          }
        }
      }
      mma_commit(&bars[L::bFinal]);
      drain_wait(&bars[L::bFinal], 0);
    }
  } else if (warp >= 4) {
    // ------------------------------------------------------------ sums
    const uint32_t y = (warp - 4) >> 2;  // the tiles with kv mod 4 == y
    const int r = (warp & 3) * 32 + lane, th = threadIdx.x - 128;
    const uint32_t t_s = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + y * 128;
    auto wwait = [&](uint64_t *bar, uint32_t parity) {
      return __all_sync(0xffffffffu, wd.wait(bar, parity)) != 0;
    };
    Walk<kAllRows> w(p.cache, p.tok, run);
    uint32_t kv = 0, used = 0;
    bool stop = false;
    while (w.next(p.cache, p.tok)) {
      const int64_t base = (static_cast<int64_t>(w.b) * p.cache.H_kv + w.hk) * p.cache.capacity;
      for (int pass = 0; pass < passes(w); ++pass) {
        const int row0 = pass * kRows, rows = min(w.s.n * G - row0, kRows);
        // the rows of this pass -> shared memory, once every group is done with the last pass (after a timeout too:
        // the barriers pair up in every path)
        named_bar_sync(1, kSumThreads);
        constexpr int kPieces = D / 8;
        const int padded = max((rows + 15) & ~15, 16);
#pragma unroll 4
        for (int i = th; i < padded * kPieces; i += kSumThreads) {
          const int rr = i / kPieces, c = i % kPieces, grow = row0 + rr;
          int4 v = make_int4(0, 0, 0, 0);
          if (rr < rows)
            v = *reinterpret_cast<const int4 *>(p.q + w.b * p.qs[0] + (grow / G) * p.qs[1] +
                                                (w.hk * G + grow % G) * p.qs[2] + c * 8);
          *reinterpret_cast<int4 *>(sm + L::kQ + (c >> 3) * (kRows * 128) + rr * 128 + (((c & 7) ^ (rr & 7)) << 4)) = v;
        }
        if (th < kRows) {
          const int grow = row0 + th, tok = grow / G, h = w.hk * G + grow % G;
          float z = -INFINITY;
          if (th < rows) {
            const float x = p.lse[(static_cast<int64_t>(w.b) * p.tok.H + h) * p.tok.T + tok];
            z = x == -INFINITY ? -INFINITY : -x * kLog2e;
          }
          nlse[th] = z;
          const uint32_t on = __ballot_sync(0xffffffffu, z != -INFINITY);
          if (lane == 0) alive[th >> 5] = on;
        } else if (th - kRows < kMaxTok) {
          const int tok = th - kRows;
          words[tok] = tok < w.s.n ? tree_word(p.tok, w.b, tok, w.s.n) : 0ull;
        }
        fence_proxy_async_smem();
        named_bar_sync(2, kSumThreads);
        if (th == 0) mbar_arrive(&bars[L::bQFull]);
        const int halves = rows > 128 ? 2 : 1;
        for (int t = w.t0; t < w.t1; ++t, ++kv) {
          if (kv % kGroups != y || stop) continue;
          const int j = t * kTile + r, d = j - w.s.len;  // this thread's slot; a new token where d >= 0
          const bool live = d < w.s.n, edge = t * kTile + kTile > w.s.len;
          float before = 0.f;
          if (live) before = pass == 0 ? p.score_in[base + j] : p.score_out[base + j];
          const float2 sc2 = make_float2(p.scale_log2, p.scale_log2);
          float2 acc[4] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
          for (int half = 0; half < halves; ++half) {
            const float *zs = nlse + half * 128;
            const int cols = min(rows - half * 128, 128);
            int fast = 0, c = 0;  // the columns [0, fast) all add something
            if (!edge)
              while (fast + 32 <= cols && alive[half * 4 + (fast >> 5)] == ~0u) fast += 32;
            if (!wwait(&bars[L::bSFull + y], used & 1)) { stop = true; break; }
            ++used;
            tc_fence_after();
            uint32_t s[32];
#pragma unroll 1
            for (; c < fast; c += 32) {
              tmem_ld32(t_s + c, s);
              tmem_wait_ld();
#pragma unroll
              for (int q = 0; q < 8; ++q) {
                const float4 z = *reinterpret_cast<const float4 *>(zs + c + 4 * q);
                const float2 e0 = __ffma2_rn(make_float2(__uint_as_float(s[4 * q]), __uint_as_float(s[4 * q + 1])), sc2,
                                             make_float2(z.x, z.y));
                const float2 e1 = __ffma2_rn(make_float2(__uint_as_float(s[4 * q + 2]), __uint_as_float(s[4 * q + 3])),
                                             sc2, make_float2(z.z, z.w));
                acc[2 * (q & 1)] = __fadd2_rn(acc[2 * (q & 1)], make_float2(fast_exp2(e0.x), fast_exp2(e0.y)));
                acc[2 * (q & 1) + 1] = __fadd2_rn(acc[2 * (q & 1) + 1], make_float2(fast_exp2(e1.x), fast_exp2(e1.y)));
              }
            }
            // the last columns, tiles with new tokens, and rows that add nothing: columns past the rows, rows whose lse
            // is -inf, and rows that do not see this thread's token, whatever they hold
#pragma unroll 1
            for (; c < cols; c += 32) {
              uint32_t on = alive[half * 4 + (c >> 5)];
              tmem_ld32(t_s + c, s);
              tmem_wait_ld();
              if (edge && d >= 0) {
                // the columns of the tokens that see new token d
                const int first = row0 + half * 128 + c;
                uint32_t sees = 0;
#pragma unroll 4
                for (int tok = first / G; tok * G < first + 32 && tok < w.s.n; ++tok)
                  if ((words[tok] >> (d & 63)) & 1ull) sees |= range_bits(tok * G - first, tok * G - first + G - 1, 0);
                on &= sees;
              }
#pragma unroll
              for (int q = 0; q < 32; ++q) {
                const float e = fast_exp2(fmaf(__uint_as_float(s[q]), p.scale_log2, zs[c + q]));
                acc[q & 3].x += ((on >> q) & 1u) ? e : 0.f;
              }
            }
            tc_fence_before();
            mbar_arrive(&bars[L::bSEmpty + y]);
          }
          if (live && !stop)
            p.score_out[base + j] =
                before + (((acc[0].x + acc[1].x) + (acc[2].x + acc[3].x)) + ((acc[0].y + acc[1].y) + (acc[2].y + acc[3].y)));
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
  static std::atomic<uint64_t> done{0};
  const cudaError_t e = allow_smem(k_weigh<FP16, D>, L::kAlloc, done);
  if (e != cudaSuccess) return e;
  count_launch();
  return launch_pdl(k_weigh<FP16, D>, dim3(ctas), dim3(128 + kSumThreads), L::kAlloc, s, tk, p);
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
