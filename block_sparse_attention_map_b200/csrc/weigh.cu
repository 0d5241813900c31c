// Accumulated attention weight of a paged cache's slots:
//   score[b, hk, j] += sum over rows r = (t, h) of the group that see j of
//                      exp(scale q_r . k_j - lse_r)
//
// One warp per slot: K's row in registers, the group's rows one after the other.
#include "serving.cuh"

namespace bsa {
namespace {

template <bool FP16, int D>
__global__ void __launch_bounds__(256) k_weigh(const WeighArgs a) {
  constexpr int E = D / 32;
  const int lane = threadIdx.x & 31;
  const int64_t warps = static_cast<int64_t>(gridDim.x) * (blockDim.x >> 5);
  const int64_t per_b = static_cast<int64_t>(a.cache.H_kv) * a.cache.capacity;
  for (int64_t w = (static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x) >> 5; w < per_b * a.cache.B;
       w += warps) {
    const int b = static_cast<int>(w / per_b), hk = static_cast<int>(w % per_b / a.cache.capacity);
    const int j = static_cast<int>(w % a.cache.capacity);
    const int len = clamped_length(a.cache, b, true), n = clamped_new(a.cache, a.tok, b, len, true);
    if (j >= len + n) continue;
    const int page = page_of(a.cache, b, j);
    if (page < 0) record_status(a.cache.status, BSA_ERR_BAD_CACHE);
    float k[E], sum = 0.f;
#pragma unroll
    for (int e = 0; e < E; e += 2) {
      float2 x = make_float2(0.f, 0.f);
      if (page >= 0)
        x = unpack16<FP16>(*reinterpret_cast<const uint32_t *>(
            a.cache.k + slot_offset(a.cache.ks, a.cache, page, j, hk) + lane * E + e));
      k[e] = x.x;
      k[e + 1] = x.y;
    }
    for (int t = 0; t < n; ++t) {
      if (j >= len && !((tree_word(a.tok, b, t, n) >> (j - len)) & 1ull)) continue;
      for (int h = hk * a.tok.G; h < (hk + 1) * a.tok.G; ++h) {
        float s = 0.f;
#pragma unroll
        for (int e = 0; e < E; e += 2) {
          const float2 x = unpack16<FP16>(*reinterpret_cast<const uint32_t *>(
              a.q + b * a.qs[0] + t * a.qs[1] + h * a.qs[2] + lane * E + e));
          s += k[e] * x.x + k[e + 1] * x.y;
        }
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
        const float z = a.lse[(static_cast<int64_t>(b) * a.tok.H + h) * a.tok.T + t];
        sum += z == -INFINITY ? 0.f : expf(s * a.scale - z);
      }
    }
    if (lane == 0) a.score_out[w] = a.score_in[w] + sum;
  }
}

}  // namespace

cudaError_t launch_weigh(const WeighArgs &a, bool fp16, cudaStream_t s) {
  count_launch();
  const unsigned blocks = 148 * 8;
  if (a.cache.D == 64) {
    if (fp16) k_weigh<true, 64><<<blocks, 256, 0, s>>>(a);
    else k_weigh<false, 64><<<blocks, 256, 0, s>>>(a);
  } else {
    if (fp16) k_weigh<true, 128><<<blocks, 256, 0, s>>>(a);
    else k_weigh<false, 128><<<blocks, 256, 0, s>>>(a);
  }
  return cudaGetLastError();
}

}  // namespace bsa
