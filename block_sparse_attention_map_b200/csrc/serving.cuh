// What the paged-cache kernels share: the cache as a kernel sees it, its
// device-side checks, and the two 16-bit element types.
#pragma once

#include "internal.h"
#include <atomic>
#include <climits>

#include "ptx.cuh"

namespace bsa {

// bsa_cache with its defaults resolved.  A slot index fits 31 bits (capacity
// <= 2^30); every element offset is 64-bit.
struct CacheView {
  int n_pages, page_log, H_kv, D, B, max_pages, capacity;
  uint16_t *k, *v;
  int64_t ks[3], vs[3];  // page, slot, head
  const int32_t *table;
  int64_t table_stride;
  const int32_t *length;
  uint32_t *status;
};

// The T new tokens of a call.
struct TokenView {
  int T, H, G;  // G = H / H_kv
  const int32_t *n_new;
  const int64_t *tree;
};

__device__ __forceinline__ int clamped_length(const CacheView &c, int b, bool report) {
  const int n = c.length[b];
  const int r = min(max(n, 0), c.capacity);
  if (report && r != n) record_status(c.status, BSA_ERR_BAD_CACHE);
  return r;
}

// The sequence's real new tokens: within [0, T], and within the capacity.
__device__ __forceinline__ int clamped_new(const CacheView &c, const TokenView &t, int b, int len, bool report) {
  const int want = t.n_new != nullptr ? t.n_new[b] : t.T;
  const int r = min(min(max(want, 0), t.T), c.capacity - len);
  if (report && r != want) record_status(c.status, BSA_ERR_BAD_CACHE);
  return r;
}

// Page of slot s of sequence b, or -1.
__device__ __forceinline__ int page_of(const CacheView &c, int b, int s) {
  const int pg = c.table[b * c.table_stride + (s >> c.page_log)];
  return static_cast<unsigned>(pg) < static_cast<unsigned>(c.n_pages) ? pg : -1;
}

__device__ __forceinline__ int64_t slot_offset(const int64_t (&st)[3], const CacheView &c, int page, int s, int h) {
  return page * st[0] + static_cast<int64_t>(s & ((1 << c.page_log) - 1)) * st[1] + h * st[2];
}

// Bits of the new tokens that token t sees, those at or past n_new cleared.
__device__ __forceinline__ uint64_t tree_word(const TokenView &t, int b, int tok, int n_new) {
  uint64_t w = ~0ull;
  if (t.tree != nullptr) w = static_cast<uint64_t>(t.tree[static_cast<int64_t>(b) * t.T + tok]);
  else w = tok >= 63 ? ~0ull : (1ull << (tok + 1)) - 1;
  return n_new >= 64 ? w : w & ((1ull << n_new) - 1);
}

template <bool FP16>
__device__ __forceinline__ float2 unpack16(uint32_t x) {
  if constexpr (FP16) return unpack_f16x2(x);
  else return unpack_bf16x2(x);
}
template <bool FP16>
__device__ __forceinline__ uint32_t pack16(float lo, float hi) {
  if constexpr (FP16) return pack_f16x2(lo, hi);
  else return pack_bf16x2(lo, hi);
}

// ---------------------------------------------------------------- launchers
// Every kernel of these is launched with programmatic serialization and waits for
// the stream's preceding kernel before it touches global memory, so its set-up
// runs under that kernel's end.  (k_attend_join alone reads before its wait, and
// only the lengths and counts: k_attend, which starts it, has waited for whatever
// wrote them and writes neither.)  Only k_attend and k_evict_select let their own
// second kernel start early; no other kernel of the stream ever starts before one
// of these is done.
//
// Sets an attribute of a kernel, once per device and kernel (`done` is the caller's
// own word, a bit a device).
template <typename F>
cudaError_t allow(F *kernel, cudaFuncAttribute what, int value, std::atomic<uint64_t> &done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev < 64 ? 1ull << dev : 0ull;
  if (bit != 0 && (done.load(std::memory_order_acquire) & bit) != 0) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, what, value);
  if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_release);
  return e;
}
template <typename F>
cudaError_t allow_smem(F *kernel, int bytes, std::atomic<uint64_t> &done) {
  return allow(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes, done);
}

struct RopeArgs {
  int B, T, H, H_kv, D;
  int n_axes, n_pairs, inverse, rotate;
  const double *inv_freq;
  const int32_t *axis, *pos;
  int64_t pos_s[2];
  const uint16_t *q, *k, *v;
  uint16_t *qo, *ko;
  int64_t qs[3], ks[3], vs[3], qos[3], kos[3];
  CacheView cache;   // append: k and v go into its slots
  TokenView tok;
};
cudaError_t launch_rope(const RopeArgs &a, bool halves, bool fp16, bool append, cudaStream_t s);

struct AttendArgs {
  CacheView cache;
  TokenView tok;
  const uint16_t *q;
  uint16_t *out;
  int64_t qs[3], os[3];
  float *lse;
  float scale;
  uint8_t *scratch;  // attend_scratch_bytes(D)
};
constexpr int kMaxCtas = 160;  // runs the attention is cut into, at most (one an SM)
size_t attend_scratch_bytes(int D);
cudaError_t launch_attend(const AttendArgs &a, const CUtensorMap &tk, const CUtensorMap &tv, bool fp16, int sms,
                          cudaStream_t s);

struct WeighArgs {
  CacheView cache;
  TokenView tok;
  const uint16_t *q;
  int64_t qs[3];
  const float *lse, *score_in;
  float *score_out;
  float scale;
};
cudaError_t launch_weigh(const WeighArgs &a, const CUtensorMap &tk, bool fp16, int sms, cudaStream_t s);

struct EvictArgs {
  CacheView cache;
  int budget, sinks, recent;
  const int32_t *next_pos, *pos_in;
  const float *score_in;
  float *score_out;
  int32_t *pos_out, *length_out;
  int list_cap;              // entries of a head's lists
  int32_t *count;            // [B * H_kv] moves of each head
  int32_t *to, *from, *mpos; // [B * H_kv, list_cap]
  float *mscore;
};
cudaError_t launch_evict(const EvictArgs &a, cudaStream_t s);

}  // namespace bsa
