// evo_seq_check.h — what the entry points of include/evo_seq.h share on the host: options, shapes,
// strides, address ranges, how a call's sequences are described to the kernels, and the query's tensor map.
#pragma once

#include <cmath>
#include <cstdint>
#include <limits>

#include "evo_seq.h"
#include "evo_seq_internal.h"

namespace evo {

constexpr uint64_t kDefaultWaitNs = 2000000000ull;
constexpr int64_t kMaxStride = int64_t(1) << 36;

inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

struct Opts {
  float scale = 0.0f;
  uint64_t wait_ns = kDefaultWaitNs;
  int* status = nullptr;
};
inline bool read_opts(const evo_seq_options_t* o, Opts* c) {
  if (!o) return true;
  if (o->size < sizeof(evo_seq_options_t) || o->flags != 0 || o->reserved != 0) return false;
  // (the kernels work with scale · log2 e, which has to be a number too)
  if (o->scale != 0.0f && !(std::isfinite(o->scale * kSeqLog2e) && o->scale > 0.0f)) return false;
  c->scale = o->scale;
  if (o->wait_limit_ns) c->wait_ns = o->wait_limit_ns < 1000 ? 1000 : o->wait_limit_ns;
  c->status = o->status;
  return true;
}

// needs_q: the call has query heads (every one but append and evict)
inline evo_status_t check_seq_shape(const evo_seq_shape_t& s, bool needs_q) {
  if (s.tokens < 0 || s.seqs < 0 || s.tokens > (int64_t(1) << 31) - 1024 || s.seqs > 65535) return EVO_ERR_BAD_SHAPE;
  if (s.kv_heads < 1 || s.kv_heads > 16384 || s.head_dim < 8 || s.head_dim > 128 || s.head_dim % 8)
    return EVO_ERR_BAD_SHAPE;
  if (!needs_q) return EVO_OK;
  if (s.q_heads < 1 || s.q_heads > 65535 || s.q_heads % s.kv_heads || s.q_heads / s.kv_heads > 128)
    return EVO_ERR_BAD_SHAPE;
  return EVO_OK;
}

inline bool page_size_ok(int64_t n) {
  return n == 16 || n == 32 || n == 64 || (n >= 128 && n <= 1024 && n % 128 == 0);
}
inline evo_status_t check_cache(const evo_cache_shape_t& c, const evo_seq_shape_t& s, int64_t* k_page, int64_t* v_page) {
  if (!page_size_ok(c.page_size) || c.num_pages < 1 || c.num_pages > (int64_t(1) << 31) - 2 || c.pages_per_seq < 1 ||
      c.pages_per_seq > (int64_t(1) << 31) - 1)
    return EVO_ERR_BAD_SHAPE;
  const int64_t packed = c.page_size * s.kv_heads * s.head_dim;
  *k_page = c.k_page_stride ? c.k_page_stride : packed;
  *v_page = c.v_page_stride ? c.v_page_stride : packed;
  for (int64_t p : {*k_page, *v_page})
    if (p < packed || p % 8 || p >= kMaxStride) return EVO_ERR_BAD_LAYOUT;
  return EVO_OK;
}

inline bool stride_ok(int64_t given, int64_t packed, long long* out) {
  *out = given ? given : packed;
  return given == 0 || (given >= packed && given % 8 == 0 && given < kMaxStride);
}

// The [tokens, heads, head_dim] tensors' token strides of one call.
struct Strides {
  long long q, k, v, out, dout, dq, dk, dv;
};
inline bool read_strides(const evo_seq_strides_t* g, const evo_seq_shape_t& s, Strides* o) {
  const evo_seq_strides_t z{};
  const evo_seq_strides_t& i = g ? *g : z;
  const int64_t nq = s.q_heads * s.head_dim, nk = s.kv_heads * s.head_dim;
  return stride_ok(i.q, nq, &o->q) && stride_ok(i.k, nk, &o->k) && stride_ok(i.v, nk, &o->v) &&
         stride_ok(i.out, nq, &o->out) && stride_ok(i.dout, nq, &o->dout) && stride_ok(i.dq, nq, &o->dq) &&
         stride_ok(i.dk, nk, &o->dk) && stride_ok(i.dv, nk, &o->dv);
}

// Address ranges: an output may overlap neither an input nor another output.  A strided
// tensor is `rows` pieces of `piece` bytes, `step` bytes apart; two with the same step may
// interleave (the parts of one projection, keys and values next to each other in a page).
struct Span {
  const void* p;
  size_t bytes;  // from the first byte to one past the last
  int64_t step, piece;
};
inline Span flat(const void* p, size_t bytes) { return {p, bytes, 0, 0}; }
inline Span strided(const void* p, int64_t rows, int64_t step, int64_t piece) {  // in elements of two bytes
  return {p, rows > 0 ? (size_t(rows - 1) * size_t(step) + size_t(piece)) * 2 : 0, step * 2, piece * 2};
}
inline bool overlap(const Span& a, const Span& b) {
  if (!a.p || !b.p || !a.bytes || !b.bytes) return false;
  const uintptr_t a0 = reinterpret_cast<uintptr_t>(a.p), b0 = reinterpret_cast<uintptr_t>(b.p);
  if (!(a0 < b0 + b.bytes && b0 < a0 + a.bytes)) return false;
  if (a.step == 0 || a.step != b.step) return true;
  const int64_t d = static_cast<int64_t>(b0 - a0), r = ((d % a.step) + a.step) % a.step;
  return !(r >= a.piece && r + b.piece <= a.step);
}
template <int NI, int NO>
inline bool aliased(const Span (&in)[NI], const Span (&out)[NO]) {
  for (int o = 0; o < NO; ++o) {
    for (int i = 0; i < NI; ++i)
      if (overlap(out[o], in[i])) return true;
    for (int p = 0; p < o; ++p)
      if (overlap(out[o], out[p])) return true;
  }
  return false;
}
inline Span pages(const void* p, const evo_cache_shape_t& c, const evo_seq_shape_t& s, int64_t stride) {
  return strided(p, c.num_pages, stride, c.page_size * s.kv_heads * s.head_dim);
}

inline SeqDesc desc(const evo_seq_shape_t& s, const int32_t* cu, const int32_t* lens, const int32_t* table,
                    const evo_cache_shape_t* c, int64_t weights_len, int* status) {
  SeqDesc d{};
  d.cu = cu;
  d.seq_lens = lens;
  d.table = table;
  d.tokens = static_cast<int>(s.tokens);
  d.seqs = static_cast<int>(s.seqs);
  d.q_heads = static_cast<int>(s.q_heads);
  d.kv_heads = static_cast<int>(s.kv_heads);
  d.group = s.kv_heads ? static_cast<int>(s.q_heads / s.kv_heads) : 0;
  d.D = static_cast<int>(s.head_dim);
  int64_t most = d.tokens;
  if (c) {
    d.page = static_cast<int>(c->page_size);
    d.pages_per_seq = static_cast<int>(c->pages_per_seq);
    d.num_pages = static_cast<int>(c->num_pages);
    most = c->page_size * c->pages_per_seq;
    if (weights_len >= 0 && weights_len < most) most = weights_len;
    const int64_t lim = std::numeric_limits<int>::max() - 1024;
    if (most > lim) most = lim;
  }
  d.max_kv = static_cast<int>(most);
  d.status = status;
  return d;
}

// CTAs of a launch: one per SM, or as many shares of a tile as the work can fill, whatever the
// lengths turn out to be.
inline int fwd_ctas(int sms, const evo_seq_shape_t& s, int64_t max_kv) {
  const double W = 2 * (kTile / (s.q_heads / s.kv_heads));
  const double units = (double(s.tokens) / W + double(s.seqs)) * (double(max_kv) + 2 * kTile) * double(s.kv_heads);
  return units < double(sms) * kTile ? static_cast<int>(units / kTile) + 1 : sms;
}

// Tensor maps of the forward.
inline bool encode16(CUtensorMap* m, const void* base, bool bf16, int rank, const cuuint64_t* dims,
                     const cuuint64_t* strides, const cuuint32_t* box, int64_t D) {
  // a head's row of more than 64 features is two boxes next to each other: one 256-byte line request
  return host_encode(m, base, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, rank, dims,
                     strides, box, CU_TENSOR_MAP_SWIZZLE_128B,
                     D > 64 ? CU_TENSOR_MAP_L2_PROMOTION_L2_256B : CU_TENSOR_MAP_L2_PROMOTION_L2_128B);
}
// [tokens, kv_heads * group, D] as (D, group, kv_heads, tokens), box (64, group, 1, TQ).
inline bool map_q(CUtensorMap* m, const void* p, bool bf16, const evo_seq_shape_t& s, int64_t stride, int TQ) {
  const int64_t G = s.q_heads / s.kv_heads;
  cuuint64_t dims[4] = {cuuint64_t(s.head_dim), cuuint64_t(G), cuuint64_t(s.kv_heads), cuuint64_t(s.tokens)};
  cuuint64_t st[3] = {cuuint64_t(s.head_dim * 2), cuuint64_t(G * s.head_dim * 2), cuuint64_t(stride * 2)};
  cuuint32_t box[4] = {64, cuuint32_t(G), 1, cuuint32_t(TQ)};
  return encode16(m, p, bf16, 4, dims, st, box, s.head_dim);
}
inline float scale_of(const Opts& o, const evo_seq_shape_t& s) {
  return o.scale != 0.0f ? o.scale : static_cast<float>(1.0 / std::sqrt(static_cast<double>(s.head_dim)));
}

}  // namespace evo
