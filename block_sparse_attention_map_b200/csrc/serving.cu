// C ABI of the positions and the paged cache (declared in include/bsa.h):
// argument validation and the launches of bsa_rope and the bsa_cache_* calls.
#include <cmath>
#include <cstring>

#include "serving.cuh"

namespace bsa {
namespace {

constexpr size_t kHeaderBytes = 256;  // the status word's part of the workspace
constexpr int kMaxTree = 64;          // new tokens a tree word can name
constexpr int kMaxGroup = 128;
constexpr int64_t kMaxTokens = (int64_t{1} << 31) - (1 << 20);  // B * T * heads: a kernel's steps past them fit 31 bits
constexpr int kMaxSequences = 1 << 16;  // of attend and weigh, whose CTAs and joined rows each read every length

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool aligned4(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
size_t up256(size_t x) { return (x + 255) / 256 * 256; }
bsa_status of_cuda(cudaError_t e) { return e == cudaSuccess ? BSA_OK : BSA_ERR_CUDA; }

bool have_sm100() {
  int dev = -1, major = 0;
  return cudaGetDevice(&dev) == cudaSuccess &&
         cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) == cudaSuccess && major == 10;
}

bool sm_count(int *sms) {
  int dev = -1;
  return cudaGetDevice(&dev) == cudaSuccess &&
         cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev) == cudaSuccess && *sms > 0;
}

// Contiguous strides where all three are zero, then the checks every tensor gets.
bsa_status fix_strides(const int64_t *in, int64_t mid, int64_t heads, int64_t D, int64_t (&out)[3]) {
  if (in[0] == 0 && in[1] == 0 && in[2] == 0) {
    out[0] = std::max<int64_t>(mid, 1) * heads * D;
    out[1] = heads * D;
    out[2] = D;
  } else {
    for (int i = 0; i < 3; ++i) out[i] = in[i];
  }
  for (int64_t x : out) {
    if (x <= 0) return BSA_ERR_INVALID_ARG;
    if (x % 8 != 0) return BSA_ERR_UNSUPPORTED;
    if (x >= (int64_t{1} << 38)) return BSA_ERR_UNSUPPORTED;  // a tensor map's strides are below 2^40 bytes
  }
  return BSA_OK;
}

struct Tokens {
  bsa_tokens t;
  int64_t qs[3], ks[3], vs[3], qos[3], kos[3];
};

bsa_status check_tokens(const bsa_tokens *in, bool any_dim, Tokens *out) {
  if (in == nullptr) return BSA_ERR_INVALID_ARG;
  out->t = *in;
  bsa_tokens &t = out->t;
  if (t.B < 0 || t.T < 0 || t.H < 1) return BSA_ERR_INVALID_ARG;
  if (t.H_kv == 0) t.H_kv = t.H;
  if (t.H_kv < 1 || t.H % t.H_kv != 0) return BSA_ERR_INVALID_ARG;
  if (t.dtype != BSA_DTYPE_BF16 && t.dtype != BSA_DTYPE_FP16) return BSA_ERR_UNSUPPORTED;
  if (any_dim ? (t.D < 16 || t.D > 256 || t.D % 16 != 0) : (t.D != 64 && t.D != 128)) return BSA_ERR_UNSUPPORTED;
  if (t.H > (1 << 20) || static_cast<int64_t>(t.B) * t.T * t.H >= kMaxTokens) return BSA_ERR_UNSUPPORTED;
  bsa_status st;
  if ((st = fix_strides(t.q_stride, t.T, t.H, t.D, out->qs)) != BSA_OK) return st;
  if ((st = fix_strides(t.k_stride, t.T, t.H_kv, t.D, out->ks)) != BSA_OK) return st;
  if ((st = fix_strides(t.v_stride, t.T, t.H_kv, t.D, out->vs)) != BSA_OK) return st;
  if ((st = fix_strides(t.qo_stride, t.T, t.H, t.D, out->qos)) != BSA_OK) return st;
  if ((st = fix_strides(t.ko_stride, t.T, t.H_kv, t.D, out->kos)) != BSA_OK) return st;
  if (!(t.scale > 0.f) || !std::isfinite(t.scale)) t.scale = 1.0f / std::sqrt(static_cast<float>(t.D));
  return BSA_OK;
}

bsa_status check_rope(const bsa_rope_spec *r, const bsa_tokens &t, bool empty, RopeArgs *a) {
  if (r == nullptr) return BSA_ERR_INVALID_ARG;
  if (r->n_axes < 1 || r->n_axes > 8 || r->n_pairs < 1 || r->n_pairs > t.D / 2) return BSA_ERR_INVALID_ARG;
  if (r->layout != BSA_ROPE_INTERLEAVED && r->layout != BSA_ROPE_HALVES) return BSA_ERR_INVALID_ARG;
  if (r->inverse != 0 && r->inverse != 1) return BSA_ERR_INVALID_ARG;
  if (r->layout == BSA_ROPE_HALVES && r->n_pairs % 8 != 0) return BSA_ERR_UNSUPPORTED;
  if (!empty && (r->inv_freq == nullptr || r->axis == nullptr || r->pos == nullptr)) return BSA_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(r->inv_freq) & 7u) || !aligned4(r->axis) || !aligned4(r->pos))
    return BSA_ERR_UNSUPPORTED;
  a->rotate = 1;
  a->n_axes = r->n_axes;
  a->n_pairs = r->n_pairs;
  a->inverse = r->inverse;
  a->inv_freq = r->inv_freq;
  a->axis = r->axis;
  a->pos = r->pos;
  a->pos_s[0] = r->pos_stride[0];
  a->pos_s[1] = r->pos_stride[1];
  if (a->pos_s[0] == 0 && a->pos_s[1] == 0) {
    a->pos_s[0] = static_cast<int64_t>(t.B) * t.T;
    a->pos_s[1] = t.T;
  }
  if (a->pos_s[0] < 0 || a->pos_s[1] < 0) return BSA_ERR_INVALID_ARG;
  return BSA_OK;
}

// Where the workspace's parts lie (list_cap < 0: no lists).
struct CacheWs {
  size_t scratch;                        // attend's pieces
  size_t count, to, from, mpos, mscore;  // evict's lists (they share the space: the calls follow one another)
  size_t total;
};

// The entries of a head's lists: it moves at most min(budget, slots past the budget) slots.
int moves_of(const CacheView &c, int budget) { return std::min(budget, std::max(c.capacity - budget, 0)); }

// The most of any budget up to the given one.
int most_moves(const CacheView &c, int budget) { return std::min(budget, c.capacity / 2); }

CacheWs cache_ws(const CacheView &c, int list_cap) {
  CacheWs w{};
  const size_t heads = static_cast<size_t>(c.B) * c.H_kv;
  w.scratch = kHeaderBytes;
  const size_t attend_end = kHeaderBytes + up256(attend_scratch_bytes(c.D));
  size_t off = kHeaderBytes;
  auto take = [&](size_t bytes) {
    const size_t o = off;
    off += up256(bytes);
    return o;
  };
  if (list_cap >= 0) {
    w.count = take(4 * heads);
    const size_t list = 4 * heads * static_cast<size_t>(list_cap);
    w.to = take(list);
    w.from = take(list);
    w.mpos = take(list);
    w.mscore = take(list);
  }
  w.total = std::max(off, attend_end);
  return w;
}

bsa_status check_cache(const bsa_cache *in, CacheView *c) {
  if (in == nullptr) return BSA_ERR_INVALID_ARG;
  if (in->B < 0 || in->H_kv < 1 || in->n_pages < 1 || in->max_pages < 1 || in->page_size < 1) return BSA_ERR_INVALID_ARG;
  if (in->D != 64 && in->D != 128) return BSA_ERR_UNSUPPORTED;
  if (in->dtype != BSA_DTYPE_BF16 && in->dtype != BSA_DTYPE_FP16) return BSA_ERR_UNSUPPORTED;
  if (in->page_size < 8 || in->page_size > 65536 || (in->page_size & (in->page_size - 1)) != 0)
    return BSA_ERR_UNSUPPORTED;
  if (in->n_pages > (1 << 30) || static_cast<int64_t>(in->max_pages) * in->page_size > (int64_t{1} << 30))
    return BSA_ERR_UNSUPPORTED;
  if (static_cast<int64_t>(in->B) * in->H_kv > (1 << 24)) return BSA_ERR_UNSUPPORTED;
  bsa_status st;
  if ((st = fix_strides(in->k_stride, in->page_size, in->H_kv, in->D, c->ks)) != BSA_OK) return st;
  if ((st = fix_strides(in->v_stride, in->page_size, in->H_kv, in->D, c->vs)) != BSA_OK) return st;
  if (in->table_stride < 0 || (in->table_stride > 0 && in->table_stride < in->max_pages)) return BSA_ERR_INVALID_ARG;
  c->n_pages = in->n_pages;
  c->page_log = 0;
  while ((1 << c->page_log) < in->page_size) ++c->page_log;
  c->H_kv = in->H_kv;
  c->D = in->D;
  c->B = in->B;
  c->max_pages = in->max_pages;
  c->capacity = in->max_pages * in->page_size;
  c->k = static_cast<uint16_t *>(in->k);
  c->v = static_cast<uint16_t *>(in->v);
  c->table = in->page_table;
  c->table_stride = in->table_stride > 0 ? in->table_stride : in->max_pages;
  c->length = in->length;
  c->status = nullptr;
  return BSA_OK;
}

// Pointers, workspace and device of a call that has work to do.
bsa_status check_ready(const CacheView &c, void *ws, size_t ws_bytes, size_t need) {
  if (c.k == nullptr || c.v == nullptr || c.table == nullptr || c.length == nullptr) return BSA_ERR_INVALID_ARG;
  if (!aligned16(c.k) || !aligned16(c.v) || !aligned4(c.table) || !aligned4(c.length)) return BSA_ERR_UNSUPPORTED;
  if (ws == nullptr || (reinterpret_cast<uintptr_t>(ws) & 255u) != 0) return BSA_ERR_INVALID_ARG;
  if (ws_bytes < need) return BSA_ERR_WORKSPACE_TOO_SMALL;
  return have_sm100() ? BSA_OK : BSA_ERR_NO_DEVICE;
}

bool matches(const bsa_cache &c, const bsa_tokens &t) {
  return c.B == t.B && c.H_kv == t.H_kv && c.D == t.D && c.dtype == t.dtype;
}

void copy3(int64_t *to, const int64_t *from) { std::memcpy(to, from, 3 * sizeof(int64_t)); }

TokenView token_view(const bsa_tokens &t) {
  return TokenView{t.T, t.H, t.H / t.H_kv, t.n_new, t.tree};
}

// The checks attend and weigh share.
bsa_status check_reading(const bsa_cache *cache, const bsa_tokens *tok, CacheView *c, Tokens *t) {
  bsa_status st;
  if ((st = check_cache(cache, c)) != BSA_OK) return st;
  if ((st = check_tokens(tok, false, t)) != BSA_OK) return st;
  if (!matches(*cache, t->t) || t->t.T > kMaxTree) return BSA_ERR_INVALID_ARG;
  if (t->t.H / t->t.H_kv > kMaxGroup || c->B > kMaxSequences) return BSA_ERR_UNSUPPORTED;
  // units of work of all heads and row groups (up to 3 a tile): 31 bits
  const int64_t rows = static_cast<int64_t>(t->t.T) * (t->t.H / t->t.H_kv);
  if (static_cast<int64_t>(c->B) * c->H_kv * (c->capacity / kTile + 1) >= (int64_t{1} << 29) / (rows / kTile + 1))
    return BSA_ERR_UNSUPPORTED;
  if (!aligned4(t->t.n_new) || (reinterpret_cast<uintptr_t>(t->t.tree) & 7u)) return BSA_ERR_UNSUPPORTED;
  return BSA_OK;
}

}  // namespace
}  // namespace bsa

using namespace bsa;

extern "C" {

bsa_status bsa_rope(const bsa_tokens *tok, const bsa_rope_spec *rope, const void *q, void *q_out, const void *k,
                    void *k_out, bsa_stream_t stream) {
  Tokens t;
  RopeArgs a{};
  bsa_status st;
  if ((st = check_tokens(tok, true, &t)) != BSA_OK) return st;
  const bool empty = t.t.B == 0 || t.t.T == 0;
  if ((st = check_rope(rope, t.t, empty, &a)) != BSA_OK) return st;
  if (empty) return BSA_OK;
  if ((q == nullptr) != (q_out == nullptr) || (k == nullptr) != (k_out == nullptr) || (q == nullptr && k == nullptr))
    return BSA_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(q_out) || !aligned16(k) || !aligned16(k_out)) return BSA_ERR_UNSUPPORTED;
  if (!have_sm100()) return BSA_ERR_NO_DEVICE;
  a.B = t.t.B;
  a.T = t.t.T;
  a.H = t.t.H;
  a.H_kv = t.t.H_kv;
  a.D = t.t.D;
  a.q = static_cast<const uint16_t *>(q);
  a.qo = static_cast<uint16_t *>(q_out);
  a.k = static_cast<const uint16_t *>(k);
  a.ko = static_cast<uint16_t *>(k_out);
  copy3(a.qs, t.qs);
  copy3(a.ks, t.ks);
  copy3(a.qos, t.qos);
  copy3(a.kos, t.kos);
  return of_cuda(launch_rope(a, rope->layout == BSA_ROPE_HALVES, t.t.dtype == BSA_DTYPE_FP16, false,
                             reinterpret_cast<cudaStream_t>(stream)));
}

bsa_status bsa_cache_workspace_size(const bsa_cache *cache, int32_t budget, size_t *bytes) {
  if (bytes == nullptr || budget < 0) return BSA_ERR_INVALID_ARG;
  CacheView c;
  const bsa_status st = check_cache(cache, &c);
  if (st != BSA_OK) return st;
  *bytes = cache_ws(c, budget > 0 ? most_moves(c, budget) : -1).total;
  return BSA_OK;
}

bsa_status bsa_cache_append(const bsa_cache *cache, const bsa_tokens *tok, const bsa_rope_spec *rope, const void *q,
                            void *q_out, const void *k, const void *v, void *ws, size_t ws_bytes,
                            bsa_stream_t stream) {
  CacheView c;
  Tokens t;
  RopeArgs a{};
  bsa_status st;
  if ((st = check_cache(cache, &c)) != BSA_OK) return st;
  if ((st = check_tokens(tok, false, &t)) != BSA_OK) return st;
  if (!matches(*cache, t.t)) return BSA_ERR_INVALID_ARG;
  const bool empty = t.t.B == 0 || t.t.T == 0;
  if (rope != nullptr && (st = check_rope(rope, t.t, empty, &a)) != BSA_OK) return st;
  if (empty) return BSA_OK;
  if (k == nullptr || v == nullptr || (q == nullptr) != (q_out == nullptr)) return BSA_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(q_out) || !aligned16(k) || !aligned16(v) || !aligned4(t.t.n_new))
    return BSA_ERR_UNSUPPORTED;
  if ((st = check_ready(c, ws, ws_bytes, kHeaderBytes)) != BSA_OK) return st;
  c.status = static_cast<uint32_t *>(ws);
  a.B = t.t.B;
  a.T = t.t.T;
  a.H = t.t.H;
  a.H_kv = t.t.H_kv;
  a.D = t.t.D;
  a.q = static_cast<const uint16_t *>(q);
  a.qo = static_cast<uint16_t *>(q_out);
  a.k = static_cast<const uint16_t *>(k);
  a.v = static_cast<const uint16_t *>(v);
  copy3(a.qs, t.qs);
  copy3(a.ks, t.ks);
  copy3(a.vs, t.vs);
  copy3(a.qos, t.qos);
  a.cache = c;
  a.tok = token_view(t.t);
  return of_cuda(launch_rope(a, rope != nullptr && rope->layout == BSA_ROPE_HALVES, t.t.dtype == BSA_DTYPE_FP16, true,
                             reinterpret_cast<cudaStream_t>(stream)));
}

bsa_status bsa_cache_attend(const bsa_cache *cache, const bsa_tokens *tok, const void *q, void *out, float *lse,
                            void *ws, size_t ws_bytes, bsa_stream_t stream) {
  CacheView c;
  Tokens t;
  bsa_status st;
  if ((st = check_reading(cache, tok, &c, &t)) != BSA_OK) return st;
  if (t.t.B == 0 || t.t.T == 0) return BSA_OK;
  if (q == nullptr || out == nullptr || lse == nullptr) return BSA_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(out) || !aligned4(lse)) return BSA_ERR_UNSUPPORTED;
  if ((st = check_ready(c, ws, ws_bytes, cache_ws(c, -1).total)) != BSA_OK) return st;
  c.status = static_cast<uint32_t *>(ws);
  AttendArgs a{};
  a.cache = c;
  a.tok = token_view(t.t);
  a.q = static_cast<const uint16_t *>(q);
  a.out = static_cast<uint16_t *>(out);
  copy3(a.qs, t.qs);
  copy3(a.os, t.qos);
  a.lse = lse;
  a.scale = t.t.scale;
  a.scratch = static_cast<uint8_t *>(ws) + cache_ws(c, -1).scratch;
  const bool fp16 = t.t.dtype == BSA_DTYPE_FP16;
  CUtensorMap tk, tv;
  if (!make_cache_map(&tk, c.k, c.n_pages, 1 << c.page_log, c.H_kv, c.D, c.ks, fp16) ||
      !make_cache_map(&tv, c.v, c.n_pages, 1 << c.page_log, c.H_kv, c.D, c.vs, fp16))
    return BSA_ERR_UNSUPPORTED;
  int sms = 0;
  if (!sm_count(&sms)) return BSA_ERR_NO_DEVICE;
  return of_cuda(launch_attend(a, tk, tv, fp16, sms, reinterpret_cast<cudaStream_t>(stream)));
}

bsa_status bsa_cache_weigh(const bsa_cache *cache, const bsa_tokens *tok, const void *q, const float *lse,
                           const float *score_in, float *score_out, void *ws, size_t ws_bytes,
                           bsa_stream_t stream) {
  CacheView c;
  Tokens t;
  bsa_status st;
  if ((st = check_reading(cache, tok, &c, &t)) != BSA_OK) return st;
  if (t.t.B == 0 || t.t.T == 0) return BSA_OK;
  if (q == nullptr || lse == nullptr || score_in == nullptr || score_out == nullptr) return BSA_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned4(lse) || !aligned4(score_in) || !aligned4(score_out)) return BSA_ERR_UNSUPPORTED;
  if ((st = check_ready(c, ws, ws_bytes, cache_ws(c, -1).total)) != BSA_OK) return st;
  c.status = static_cast<uint32_t *>(ws);
  WeighArgs a{};
  a.cache = c;
  a.tok = token_view(t.t);
  a.q = static_cast<const uint16_t *>(q);
  copy3(a.qs, t.qs);
  a.lse = lse;
  a.score_in = score_in;
  a.score_out = score_out;
  a.scale = t.t.scale;
  const bool fp16 = t.t.dtype == BSA_DTYPE_FP16;
  CUtensorMap tk;
  if (!make_cache_map(&tk, c.k, c.n_pages, 1 << c.page_log, c.H_kv, c.D, c.ks, fp16)) return BSA_ERR_UNSUPPORTED;
  int sms = 0;
  if (!sm_count(&sms)) return BSA_ERR_NO_DEVICE;
  return of_cuda(launch_weigh(a, tk, fp16, sms, reinterpret_cast<cudaStream_t>(stream)));
}

bsa_status bsa_cache_evict(const bsa_cache *cache, const bsa_evict_spec *e, void *ws, size_t ws_bytes,
                           bsa_stream_t stream) {
  CacheView c;
  bsa_status st;
  if ((st = check_cache(cache, &c)) != BSA_OK) return st;
  if (e == nullptr || e->budget < 1 || e->sinks < 0 || e->recent < 0) return BSA_ERR_INVALID_ARG;
  if (c.B == 0) return BSA_OK;
  if (e->next_pos == nullptr || e->score_in == nullptr || e->pos_in == nullptr || e->score_out == nullptr ||
      e->pos_out == nullptr || e->length_out == nullptr)
    return BSA_ERR_INVALID_ARG;
  if (!aligned4(e->next_pos) || !aligned4(e->score_in) || !aligned4(e->pos_in) || !aligned4(e->score_out) ||
      !aligned4(e->pos_out) || !aligned4(e->length_out))
    return BSA_ERR_UNSUPPORTED;
  const int list_cap = moves_of(c, e->budget);
  const CacheWs w = cache_ws(c, list_cap);
  if ((st = check_ready(c, ws, ws_bytes, w.total)) != BSA_OK) return st;
  uint8_t *base = static_cast<uint8_t *>(ws);
  c.status = reinterpret_cast<uint32_t *>(base);
  EvictArgs a{};
  a.cache = c;
  a.budget = e->budget;
  a.sinks = e->sinks;
  a.recent = e->recent;
  a.next_pos = e->next_pos;
  a.pos_in = e->pos_in;
  a.score_in = e->score_in;
  a.score_out = e->score_out;
  a.pos_out = e->pos_out;
  a.length_out = e->length_out;
  a.list_cap = list_cap;
  a.count = reinterpret_cast<int32_t *>(base + w.count);
  a.to = reinterpret_cast<int32_t *>(base + w.to);
  a.from = reinterpret_cast<int32_t *>(base + w.from);
  a.mpos = reinterpret_cast<int32_t *>(base + w.mpos);
  a.mscore = reinterpret_cast<float *>(base + w.mscore);
  return of_cuda(launch_evict(a, reinterpret_cast<cudaStream_t>(stream)));
}

}  // extern "C"
