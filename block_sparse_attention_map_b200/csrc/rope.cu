// Rotary positions with several axes, forward and backward, and the serving
// form that puts the new tokens' K (rotated) and V into the paged cache.
//
//   angle = pos[axis[p], b, t] * inv_freq[p]
//   y0 = x0 cos - x1 sin,  y1 = x0 sin + x1 cos     (inverse: sin -> -sin)
//
// A thread owns one 16-byte chunk of a token (4 interleaved pairs, or 8 pairs
// as one chunk of each half), takes the chunk's sines and cosines once, and
// walks the token's heads with them.  Consecutive threads are consecutive
// chunks, then heads: a warp moves 512 contiguous bytes.  Bound: HBM; the only
// reads besides the tensors are the positions and the two small tables.
//
// The angle is reduced before any rounding to 32 bits: the frequency in turns
// is a 64-bit fraction of a turn, so its product with the integer position
// wraps mod 2^64 to the exact fractional turn (within |pos| * 2^-54 turns, the
// double-precision frequency's own rounding), of which the top 32 bits go to
// sincospi.
#include "serving.cuh"

namespace bsa {
namespace {

// The angle's sine and cosine; false for a pair that is copied.
__device__ __forceinline__ bool pair_turn(const RopeArgs &a, int p, int b, int t, float &c, float &s) {
  c = 1.f;
  s = 0.f;
  if (!a.rotate || p >= a.n_pairs) return false;
  const int ax = a.axis[p];
  if (static_cast<unsigned>(ax) >= static_cast<unsigned>(a.n_axes)) return false;
  const int64_t pos = a.pos[ax * a.pos_s[0] + b * a.pos_s[1] + t];
  double f = a.inv_freq[p] * 0.15915494309189535;  // 1 / (2 pi)
  f -= floor(f);
  const uint64_t frac = f >= 0.0 && f < 1.0 ? static_cast<uint64_t>(f * 18446744073709551616.0) : 0ull;
  const uint64_t turn = static_cast<uint64_t>(pos) * frac;
  const int32_t top = static_cast<int32_t>((turn + 0x80000000ull) >> 32);
  sincospif(static_cast<float>(top) * 4.656612873077393e-10f /* 2^-31 */, &s, &c);
  if (a.inverse) s = -s;
  return true;
}

// Eight rotated elements as four pairs side by side.
template <bool FP16>
__device__ __forceinline__ int4 turn_interleaved(int4 v, const float (&c)[4], const float (&s)[4], uint32_t rot) {
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

template <bool FP16>
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
    // a copied pair keeps its bits (0 * infinity would make it NaN)
    const uint32_t m = ((rot >> (2 * i)) & 1u ? 0xffffu : 0u) | ((rot >> (2 * i + 1)) & 1u ? 0xffff0000u : 0u);
    x[i] = (u & m) | (x[i] & ~m);
    y[i] = (w & m) | (y[i] & ~m);
  }
  v0 = make_int4(x[0], x[1], x[2], x[3]);
  v1 = make_int4(y[0], y[1], y[2], y[3]);
}

struct HeadPtr {
  const uint16_t *src;
  uint16_t *dst;
  bool turn;
};

// Where head i of the list [q heads, k heads, v heads (append)] of a token lies;
// dst null: nothing to do.
__device__ __forceinline__ HeadPtr head_ptr(const RopeArgs &a, int i, int b, int t, int64_t k_off, int64_t v_off) {
  HeadPtr r{nullptr, nullptr, true};
  const int nq = a.q != nullptr ? a.H : 0;
  if (i < nq) {
    r.src = a.q + b * a.qs[0] + t * a.qs[1] + i * a.qs[2];
    r.dst = a.qo + b * a.qos[0] + t * a.qos[1] + i * a.qos[2];
    return r;
  }
  i -= nq;
  if (!a.append) {
    r.src = a.k + b * a.ks[0] + t * a.ks[1] + i * a.ks[2];
    r.dst = a.ko + b * a.kos[0] + t * a.kos[1] + i * a.kos[2];
    return r;
  }
  if (k_off < 0) return r;  // padding token, or no valid page
  if (i < a.H_kv) {
    r.src = a.k + b * a.ks[0] + t * a.ks[1] + i * a.ks[2];
    r.dst = a.cache.k + k_off + i * a.cache.ks[2];
  } else {
    i -= a.H_kv;
    r.src = a.v + b * a.vs[0] + t * a.vs[1] + i * a.vs[2];
    r.dst = a.cache.v + v_off + i * a.cache.vs[2];
    r.turn = false;
  }
  return r;
}

template <bool FP16, bool HALVES>
__global__ void __launch_bounds__(256) k_rope(const RopeArgs a, int n_heads, int n_chunks, int head_split) {
  constexpr int P = HALVES ? 8 : 4;
  const int64_t unit = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
  const int c = static_cast<int>(unit % n_chunks);
  const int64_t rest = unit / n_chunks;
  const int h0 = static_cast<int>(rest % head_split);
  const int64_t row = rest / head_split;
  if (row >= static_cast<int64_t>(a.B) * a.T) return;
  const int b = static_cast<int>(row / a.T), t = static_cast<int>(row % a.T);

  // this thread's elements: one chunk, or one of each half
  const int pair_chunks = HALVES ? a.n_pairs >> 3 : n_chunks;
  const bool both = HALVES && c < pair_chunks;
  const int e0 = HALVES && !both ? (c + pair_chunks) * 8 : c * 8;
  const int e1 = both ? a.n_pairs + c * 8 : e0;
  float cs[P], sn[P];
  uint32_t rot = 0;
#pragma unroll
  for (int i = 0; i < P; ++i) {
    cs[i] = 1.f;
    sn[i] = 0.f;
    if (!HALVES || both) rot |= (pair_turn(a, c * P + i, b, t, cs[i], sn[i]) ? 1u : 0u) << i;
  }

  int64_t k_off = -1, v_off = -1;
  if (a.append) {
    const bool report = c == 0 && h0 == 0;
    const int len = clamped_length(a.cache, b, report);
    const int n = clamped_new(a.cache, a.tok, b, len, report);
    if (t < n) {
      const int slot = len + t, page = page_of(a.cache, b, slot);
      if (page >= 0) {
        k_off = slot_offset(a.cache.ks, a.cache, page, slot, 0);
        v_off = slot_offset(a.cache.vs, a.cache, page, slot, 0);
      } else if (report) {
        record_status(a.cache.status, BSA_ERR_BAD_CACHE);
      }
    }
  }

  constexpr int U = 4;  // heads in flight
  for (int h = h0; h < n_heads; h += U * head_split) {
    HeadPtr hp[U];
    int4 v0[U], v1[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = h + u * head_split;
      hp[u] = HeadPtr{nullptr, nullptr, false};
      if (i < n_heads) hp[u] = head_ptr(a, i, b, t, k_off, v_off);
      if (hp[u].dst != nullptr) {
        v0[u] = *reinterpret_cast<const int4 *>(hp[u].src + e0);
        if (both) v1[u] = *reinterpret_cast<const int4 *>(hp[u].src + e1);
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (hp[u].dst == nullptr) continue;
      if (hp[u].turn && rot != 0u) {
        if constexpr (HALVES) turn_halves<FP16>(v0[u], v1[u], cs, sn, rot);
        else v0[u] = turn_interleaved<FP16>(v0[u], cs, sn, rot);
      }
      *reinterpret_cast<int4 *>(hp[u].dst + e0) = v0[u];
      if (both) *reinterpret_cast<int4 *>(hp[u].dst + e1) = v1[u];
    }
  }
}

template <bool FP16, bool HALVES>
cudaError_t launch(const RopeArgs &a, cudaStream_t s) {
  const int n_heads = (a.q != nullptr ? a.H : 0) + (a.append ? 2 * a.H_kv : a.k != nullptr ? a.H_kv : 0);
  const int chunks = HALVES ? a.D / 8 - a.n_pairs / 8 : a.D / 8;
  const int64_t rows = static_cast<int64_t>(a.B) * a.T;
  // heads shared out over threads until the GPU is full (148 SMs x 2048
  // threads), at most 16 heads a thread
  const int64_t full = 148 * 2048;
  int64_t split = (full + rows * chunks - 1) / (rows * chunks);
  split = std::max<int64_t>(split, (n_heads + 15) / 16);
  split = std::min<int64_t>(split, n_heads);
  const int64_t units = rows * chunks * split;
  const int64_t blocks = (units + 255) / 256;
  if (blocks > 0x7fffffff) return cudaErrorInvalidConfiguration;
  count_launch();
  k_rope<FP16, HALVES><<<static_cast<unsigned>(blocks), 256, 0, s>>>(a, n_heads, chunks, static_cast<int>(split));
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_rope(const RopeArgs &a, bool halves, bool fp16, cudaStream_t s) {
  if (fp16) return halves ? launch<true, true>(a, s) : launch<true, false>(a, s);
  return halves ? launch<false, true>(a, s) : launch<false, false>(a, s);
}

}  // namespace bsa
