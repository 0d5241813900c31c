// Attention of a few new tokens (a tree of drafted tokens, or one) over a paged
// cache: O = softmax(scale q K^T) V and the LSE, row (token t, head h) seeing
// the slots below length and the new tokens of its tree word.
//
// One warp per row: the keys one after the other, D / 32 elements a lane, the
// running maximum and sum in registers.
#include "serving.cuh"

namespace bsa {
namespace {

template <bool FP16, int D>
__global__ void __launch_bounds__(256) k_attend(const AttendArgs a) {
  constexpr int E = D / 32;
  const int lane = threadIdx.x & 31;
  const int64_t row = (static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x) >> 5;
  const int T = a.tok.T, H = a.tok.H;
  if (row >= static_cast<int64_t>(a.cache.B) * T * H) return;
  const int h = static_cast<int>(row % H), t = static_cast<int>((row / H) % T), b = static_cast<int>(row / H / T);
  const int len = clamped_length(a.cache, b, true), n = clamped_new(a.cache, a.tok, b, len, true);
  const uint64_t word = t < n ? tree_word(a.tok, b, t, n) : 0ull;
  const int hk = h / a.tok.G;
  float q[E], o[E], m = -INFINITY, l = 0.f;
#pragma unroll
  for (int e = 0; e < E; e += 2) {
    const float2 x = unpack16<FP16>(*reinterpret_cast<const uint32_t *>(
        a.q + b * a.qs[0] + t * a.qs[1] + h * a.qs[2] + lane * E + e));
    q[e] = x.x;
    q[e + 1] = x.y;
    o[e] = o[e + 1] = 0.f;
  }
  const int end = t < n ? len + n : 0;
  for (int j = 0; j < end; ++j) {
    if (j >= len && !((word >> (j - len)) & 1ull)) continue;
    const int page = page_of(a.cache, b, j);
    if (page < 0) record_status(a.cache.status, BSA_ERR_BAD_CACHE);
    float s = 0.f, v[E];
#pragma unroll
    for (int e = 0; e < E; e += 2) {
      float2 x = make_float2(0.f, 0.f), y = x;
      if (page >= 0) {
        x = unpack16<FP16>(*reinterpret_cast<const uint32_t *>(
            a.cache.k + slot_offset(a.cache.ks, a.cache, page, j, hk) + lane * E + e));
        y = unpack16<FP16>(*reinterpret_cast<const uint32_t *>(
            a.cache.v + slot_offset(a.cache.vs, a.cache, page, j, hk) + lane * E + e));
      }
      s += q[e] * x.x + q[e + 1] * x.y;
      v[e] = y.x;
      v[e + 1] = y.y;
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
    s *= a.scale;
    const float mn = fmaxf(m, s), al = m == -INFINITY ? 0.f : expf(m - mn), p = mn == -INFINITY ? 0.f : expf(s - mn);
    l = l * al + p;
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = o[e] * al + p * v[e];
    m = mn;
  }
  const float inv = l > 0.f ? 1.f / l : (l != l ? l : 0.f);
  uint16_t *dst = a.out + b * a.os[0] + t * a.os[1] + h * a.os[2] + lane * E;
#pragma unroll
  for (int e = 0; e < E; e += 2)
    *reinterpret_cast<uint32_t *>(dst + e) = pack16<FP16>(o[e] * inv, o[e + 1] * inv);
  if (lane == 0) a.lse[(static_cast<int64_t>(b) * H + h) * T + t] = l == 0.f ? -INFINITY : m + logf(l);
}

}  // namespace

cudaError_t launch_attend(const AttendArgs &a, bool fp16, cudaStream_t s) {
  const int64_t rows = static_cast<int64_t>(a.cache.B) * a.tok.T * a.tok.H;
  const unsigned blocks = static_cast<unsigned>((rows + 7) / 8);
  count_launch();
  if (a.cache.D == 64) {
    if (fp16) k_attend<true, 64><<<blocks, 256, 0, s>>>(a);
    else k_attend<false, 64><<<blocks, 256, 0, s>>>(a);
  } else {
    if (fp16) k_attend<true, 128><<<blocks, 256, 0, s>>>(a);
    else k_attend<false, 128><<<blocks, 256, 0, s>>>(a);
  }
  return cudaGetLastError();
}

}  // namespace bsa
