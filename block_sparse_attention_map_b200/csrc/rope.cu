// Rotary positions with several axes, forward and backward, and the serving
// form that puts the new tokens' K (rotated) and V into the paged cache.
//
//   angle = pos[axis[p], b, t] * inv_freq[p]
//   y0 = x0 cos - x1 sin,  y1 = x0 sin + x1 cos     (inverse: sin -> -sin)
//
// A block takes a few tokens: its threads compute the tokens' sines and cosines
// once, into shared memory (a thread for each pair and token), then each thread
// holds those of 8 pairs (a 16-byte chunk of each half, or two chunks of 4
// interleaved pairs D/2 elements apart) and walks a share of the token's heads with them.  Consecutive
// threads are consecutive chunks, then heads: a warp moves 512 contiguous bytes.
// Bound: HBM; the only reads besides the tensors are the positions and the two
// small tables.  (A thread that computed its own chunk's sines for each share of
// the heads spent more time on them than on the rows where heads are few: 8192
// tokens x 20 heads 30 us, now 17.)
//
// The angle is reduced before any rounding to 32 bits: the frequency in turns
// is a 64-bit fraction of a turn (from a two-word product with 1 / (2 pi): of one
// double the position would multiply its rounding, 3e-3 rad at 10^4 rad a position
// and position 2^31), so its product with the integer position wraps mod 2^64 to the
// fractional turn within |pos| * 2^-63 turns, of which the top 32 bits go to sincospi.
#include "serving.cuh"

namespace bsa {
namespace {

// A pair's frequency as a 64-bit fraction of a turn, and its axis (-1: the pair is
// copied).
struct Pair {
  uint64_t frac;
  int axis;
};

__device__ __forceinline__ Pair pair_of(const RopeArgs &a, int p) {
  if (p >= a.n_pairs) return Pair{0, -1};
  const int ax = a.axis[p];
  if (static_cast<unsigned>(ax) >= static_cast<unsigned>(a.n_axes)) return Pair{0, -1};
  // 1 / (2 pi) = kHi + kLo, so the frequency in turns = hi + lo; each word less its nearest integer as a multiple of 2^-64
  constexpr double kHi = 0x1.45f306dc9c883p-3, kLo = -0x1.6b01ec5417056p-57;
  const double f = a.inv_freq[p], hi = f * kHi, lo = fma(f, kHi, -hi) + f * kLo;
  if (!isfinite(f)) return Pair{0, ax};
  auto fraction = [](double x) { return static_cast<uint64_t>(__double2ll_rn((x - rint(x)) * 18446744073709551616.0)); };
  return Pair{fraction(hi) + fraction(lo), ax};
}

__device__ __forceinline__ void turn_of(const RopeArgs &a, const Pair &p, int b, int t, float &c, float &s) {
  c = 1.f;
  s = 0.f;
  if (p.axis < 0) return;
  const int64_t pos = a.pos[p.axis * a.pos_s[0] + b * a.pos_s[1] + t];
  const uint64_t turn = static_cast<uint64_t>(pos) * p.frac;
  const int32_t top = static_cast<int32_t>((turn + 0x80000000ull) >> 32);
  sincospif(static_cast<float>(top) * 4.656612873077393e-10f /* 2^-31 */, &s, &c);
  if (a.inverse) s = -s;
}

// Eight rotated elements as four pairs side by side.
template <bool FP16>
__device__ __forceinline__ int4 turn_interleaved(int4 v, const float *c, const float *s, uint32_t rot) {
  uint32_t w[4] = {static_cast<uint32_t>(v.x), static_cast<uint32_t>(v.y), static_cast<uint32_t>(v.z),
                   static_cast<uint32_t>(v.w)};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 x = unpack16<FP16>(w[i]);
    const uint32_t y = pack16<FP16>(x.x * c[i] - x.y * s[i], x.x * s[i] + x.y * c[i]);
    w[i] = (rot >> i) & 1u ? y : w[i];
  }
  return make_int4(w[0], w[1], w[2], w[3]);
}

template <bool FP16, bool APPEND>
__device__ __forceinline__ void turn_halves(int4 &v0, int4 &v1, const float (&c)[8], const float (&s)[8],
                                            uint32_t rot) {
  uint32_t x[4] = {static_cast<uint32_t>(v0.x), static_cast<uint32_t>(v0.y), static_cast<uint32_t>(v0.z),
                   static_cast<uint32_t>(v0.w)};
  uint32_t y[4] = {static_cast<uint32_t>(v1.x), static_cast<uint32_t>(v1.y), static_cast<uint32_t>(v1.z),
                   static_cast<uint32_t>(v1.w)};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 a = unpack16<FP16>(x[i]), b = unpack16<FP16>(y[i]);
    const uint32_t u = pack16<FP16>(a.x * c[2 * i] - b.x * s[2 * i], a.y * c[2 * i + 1] - b.y * s[2 * i + 1]);
    const uint32_t w = pack16<FP16>(a.x * s[2 * i] + b.x * c[2 * i], a.y * s[2 * i + 1] + b.y * c[2 * i + 1]);
    if (!APPEND && rot == 0xffu) {
      x[i] = u;
      y[i] = w;
      continue;
    }
    // a copied pair keeps its bits (0 * infinity would make it NaN)
    const uint32_t m = ((rot >> (2 * i)) & 1u ? 0xffffu : 0u) | ((rot >> (2 * i + 1)) & 1u ? 0xffff0000u : 0u);
    x[i] = (u & m) | (x[i] & ~m);
    y[i] = (w & m) | (y[i] & ~m);
  }
  v0 = make_int4(x[0], x[1], x[2], x[3]);
  v1 = make_int4(y[0], y[1], y[2], y[3]);
}

struct RopeGrid {
  int n_heads, n_chunks, tokens, lanes;  // a block's step: tokens x lanes (shares of the heads) x chunks
  int pairs;                             // whose sines are computed (0: k and v as they are)
};

// APPEND: k and v go into the cache's slots.  (One kernel for both had no registers
// left in the other case: 75600 tokens x 80 heads in halves 507 us, now 490, 8192 x
// 20 heads 17.4 and 16.4.)
template <bool FP16, bool HALVES, bool APPEND>
__global__ void __launch_bounds__(256, 4) k_rope(const RopeArgs a, const RopeGrid g) {
  constexpr int P = 8;  // pairs of a thread: one chunk of each half's, or two chunks of four
  constexpr int U = 2;  // heads in flight
  extern __shared__ float trig[];    // two of: cos [tokens][pairs], sin likewise; then which pairs turn
  const int pairs = g.pairs;
  uint8_t *turn_sm = reinterpret_cast<uint8_t *>(trig + 4 * g.tokens * pairs);
  const int rows = a.B * a.T, step = gridDim.x * g.tokens;  // rows < 2^31

  pdl_wait();
  // the sines' side: this thread's pair, and every n_sub-th token of a step
  const int n_sub = pairs > 0 ? 256 / pairs : 0, p_sub = pairs > 0 ? threadIdx.x / pairs : 0;
  const int p_id = pairs > 0 ? threadIdx.x % pairs : 0;
  Pair pair{0, -1};
  if (p_sub < n_sub) {
    pair = pair_of(a, p_id);
    if (p_sub == 0) turn_sm[p_id] = pair.axis >= 0;
  }
  // the rows' side: this thread's chunk (or one of each half), share and token
  const int c = threadIdx.x % g.n_chunks, u0 = threadIdx.x / g.n_chunks, h0 = u0 % g.lanes, tk = u0 / g.lanes;
  const int pair_chunks = HALVES ? a.n_pairs >> 3 : g.n_chunks;
  const bool both = c < pair_chunks;
  const int e0 = both ? c * 8 : (c + pair_chunks) * 8;
  const int gap = HALVES ? a.n_pairs : a.D >> 1;  // from the first chunk to the second
  const int s0 = HALVES ? c * 8 : c * 4, s1 = HALVES ? s0 + 4 : s0 + (a.D >> 2);  // its pairs: s0 .. s0+3, s1 .. s1+3
  const bool pair_chunk = a.rotate && both;
  const int nq = a.q != nullptr ? a.H : 0;

  int buf = 0;
  for (int row0 = blockIdx.x * g.tokens; row0 < rows; row0 += step, buf ^= 1) {
    const int row = row0 + tk;
    const bool on = tk < g.tokens && row < rows;
    const int b = on ? row / a.T : 0, t = on ? row - b * a.T : 0;
    // the token's rows: q heads, k heads, v heads (append), each with its head stride
    const uint16_t *q_src = a.q + b * a.qs[0] + t * a.qs[1] + e0;
    uint16_t *q_dst = a.qo + b * a.qos[0] + t * a.qos[1] + e0;
    const uint16_t *k_src = a.k + b * a.ks[0] + t * a.ks[1] + e0, *v_src = nullptr;
    uint16_t *k_dst = a.ko + b * a.kos[0] + t * a.kos[1] + e0, *v_dst = nullptr;
    int n_heads = on ? g.n_heads : 0;
    if (APPEND && on) {
      const bool report = c == 0 && h0 == 0;
      const int len = clamped_length(a.cache, b, report);
      const int n = clamped_new(a.cache, a.tok, b, len, report);
      const int slot = len + t, page = t < n ? page_of(a.cache, b, slot) : -1;
      if (page >= 0) {
        k_dst = a.cache.k + slot_offset(a.cache.ks, a.cache, page, slot, 0) + e0;
        v_dst = a.cache.v + slot_offset(a.cache.vs, a.cache, page, slot, 0) + e0;
        v_src = a.v + b * a.vs[0] + t * a.vs[1] + e0;
      } else {
        n_heads = nq;  // a padding token, or a bad page: its q alone
        if (report && t < n) record_status(a.cache.status, BSA_ERR_BAD_CACHE);
      }
    }
    const int64_t k_ds = APPEND ? a.cache.ks[2] : a.kos[2], v_ds = APPEND ? a.cache.vs[2] : 0;
    auto src_of = [&](int i) {
      return i < nq ? q_src + i * a.qs[2] : !APPEND || i < nq + a.H_kv ? k_src + (i - nq) * a.ks[2] : v_src + (i - nq - a.H_kv) * a.vs[2];
    };
    auto dst_of = [&](int i) {
      return i < nq ? q_dst + i * a.qos[2] : !APPEND || i < nq + a.H_kv ? k_dst + (i - nq) * k_ds : v_dst + (i - nq - a.H_kv) * v_ds;
    };
    int4 v0[U], v1[U];
    auto load = [&](int h) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int i = h + u * g.lanes;
        if (i < n_heads) {
          const uint16_t *src = src_of(i);
          v0[u] = *reinterpret_cast<const int4 *>(src);
          if (both) v1[u] = *reinterpret_cast<const int4 *>(src + gap);
        }
      }
    };
    load(h0);  // in flight under the sines

    float *cs_sm = trig + buf * 2 * g.tokens * pairs, *sn_sm = cs_sm + g.tokens * pairs;
    if (p_sub < n_sub) {
      for (int k = p_sub; k < g.tokens && row0 + k < rows; k += n_sub) {
        const int bb = (row0 + k) / a.T;
        float cv, sv;
        turn_of(a, pair, bb, row0 + k - bb * a.T, cv, sv);
        cs_sm[k * pairs + p_id] = cv;
        sn_sm[k * pairs + p_id] = sv;
      }
    }
    __syncthreads();  // one a step: the next one writes the other buffer
    float cs[P], sn[P];
    uint32_t rot = 0;
    if (pair_chunk && on) {
#pragma unroll
      for (int i = 0; i < P; i += 4) {
        const int at = i == 0 ? s0 : s1;
        const float4 x = *reinterpret_cast<const float4 *>(cs_sm + tk * pairs + at);
        const float4 y = *reinterpret_cast<const float4 *>(sn_sm + tk * pairs + at);
        cs[i] = x.x, cs[i + 1] = x.y, cs[i + 2] = x.z, cs[i + 3] = x.w;
        sn[i] = y.x, sn[i + 1] = y.y, sn[i + 2] = y.z, sn[i + 3] = y.w;
#pragma unroll
        for (int k = 0; k < 4; ++k) rot |= static_cast<uint32_t>(turn_sm[at + k]) << (i + k);
      }
    }
    for (int h = h0; h < n_heads; h += U * g.lanes) {
      if (h != h0) load(h);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int i = h + u * g.lanes;
        if (i >= n_heads) continue;
        if (rot != 0u && (!APPEND || i < nq + a.H_kv)) {
          if constexpr (HALVES) {
            turn_halves<FP16, APPEND>(v0[u], v1[u], cs, sn, rot);
          } else {
            v0[u] = turn_interleaved<FP16>(v0[u], cs, sn, rot);
            v1[u] = turn_interleaved<FP16>(v1[u], cs + 4, sn + 4, rot >> 4);
          }
        }
        uint16_t *dst = dst_of(i);
        *reinterpret_cast<int4 *>(dst) = v0[u];
        if (both) *reinterpret_cast<int4 *>(dst + gap) = v1[u];
      }
    }
  }
}

template <bool FP16, bool HALVES, bool APPEND>
cudaError_t launch(const RopeArgs &a, cudaStream_t s) {
  RopeGrid g;
  g.n_heads = (a.q != nullptr ? a.H : 0) + (APPEND ? 2 * a.H_kv : a.k != nullptr ? a.H_kv : 0);
  g.n_chunks = HALVES ? a.D / 8 - a.n_pairs / 8 : a.D / 16;
  g.pairs = !a.rotate ? 0 : HALVES ? a.n_pairs : a.D / 2;
  const int64_t rows = static_cast<int64_t>(a.B) * a.T;
  // a thread takes about 20 heads (few waits for the sines a byte: 75600 tokens x
  // 80 heads 499 us, with 8 heads 539) where there are tokens enough for four
  // blocks an SM, else fewer tokens a block and fewer heads a thread
  const int shares = 256 / g.n_chunks;
  const int64_t few = (rows + 4 * 148 - 1) / (4 * 148);
  g.tokens = static_cast<int>(std::min<int64_t>(few, shares / std::min(shares, (g.n_heads + 19) / 20)));
  g.lanes = std::max(1, std::min(shares / g.tokens, g.n_heads));
  const int64_t blocks = std::min<int64_t>((rows + g.tokens - 1) / g.tokens, 148 * 8);
  count_launch();
  return launch_pdl(k_rope<FP16, HALVES, APPEND>, dim3(static_cast<unsigned>(blocks)), dim3(256), (g.tokens * 16 + 1) * g.pairs, s, a, g);
}

}  // namespace

cudaError_t launch_rope(const RopeArgs &a, bool halves, bool fp16, bool append, cudaStream_t s) {
  if (append) {
    if (fp16) return halves ? launch<true, true, true>(a, s) : launch<true, false, true>(a, s);
    return halves ? launch<false, true, true>(a, s) : launch<false, false, true>(a, s);
  }
  if (fp16) return halves ? launch<true, true, false>(a, s) : launch<true, false, false>(a, s);
  return halves ? launch<false, true, false>(a, s) : launch<false, false, false>(a, s);
}

}  // namespace bsa
