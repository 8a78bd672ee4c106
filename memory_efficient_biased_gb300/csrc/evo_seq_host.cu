// evo_seq_host.cu — the C ABI of the causal-sequence operators (include/evo_seq.h):
// argument validation, workspace sizes and dispatch to the kernels.
#include "evo_seq_check.h"

namespace evo {
namespace {

// CTAs of the prompt's backward, as fwd_ctas.
int bwd_ctas(int sms, const evo_seq_shape_t& s) {
  const double TQ = kTile / (s.q_heads / s.kv_heads), T = double(s.tokens);
  const double units = (T / TQ + double(s.seqs)) * (T + 3 * kTile) * double(s.kv_heads);  // dQ's, the more
  return units < double(sms) * kTile ? static_cast<int>(units / kTile) + 1 : sms;
}

// dK/dV and dQ of the prompt's backward: one behind the other in each CTA (1), or at the same time in two
// rows of half as many CTAs (2).  Two rows save one phase's start and end, some 7 us, and leave the faster
// row idle at the end, some 4 % to 8 %.  So: two up to 30 tiles an SM, each item counted with the tiles
// that sequences of equal lengths would give it.  Measured, one row / two: 496 tokens (0.8 tiles) 27 / 20 us,
// 2048 tokens, one kv head of 128 (5) 54 / 41, 1800 tokens, 8 (20) 92 / 88, 2500 tokens, 4 (27) 113 / 111,
// 6000 tokens, 4 (33) 138 / 142, 8000 tokens, 2 (113) 371 / 401.
int bwd_rows(int sms, const evo_seq_shape_t& s) {
  const double T = double(s.tokens), B = double(s.seqs);
  const double items = (T / (kTile / (s.q_heads / s.kv_heads)) + B) * double(s.kv_heads);
  return items * (T / B / (2 * kTile) + 3) <= 30.0 * sms ? 2 : 1;
}

// Scores left behind by the forward for the weights (0: they are formed again).  A row's score is
// written and read once, 8 bytes a key; forming it again reads 2 head_dim bytes a key, whatever
// the number of rows.  So: up to 16 rows a key on the average, and only while the
// scores, sized by the longest length the table can hold, stay below a quarter of the cache.
long long scores_row(const evo_cache_shape_t& c, int64_t weights_len) {
  const int64_t most = c.page_size * c.pages_per_seq < weights_len ? c.page_size * c.pages_per_seq : weights_len;
  return (most + kTile - 1) / kTile * kTile;
}
size_t scores_bytes(const evo_seq_shape_t& s, const evo_cache_shape_t& c, int64_t weights_len) {
  if (weights_len <= 0 || s.tokens * (s.q_heads / s.kv_heads) > 16 * s.seqs) return 0;
  const double bytes = 4.0 * double(s.tokens) * double(s.q_heads) * double(scores_row(c, weights_len));
  const double cache = 4.0 * double(c.num_pages) * double(c.page_size) * double(s.kv_heads) * double(s.head_dim);
  return bytes <= cache / 4 ? (static_cast<size_t>(bytes) + 255) & ~size_t(255) : 0;
}

// [tokens, kv_heads, D] as (D, kv_heads, tokens), box (64, 1, 128).
bool map_rows(CUtensorMap* m, const void* p, bool bf16, const evo_seq_shape_t& s, int64_t stride) {
  cuuint64_t dims[3] = {cuuint64_t(s.head_dim), cuuint64_t(s.kv_heads), cuuint64_t(s.tokens)};
  cuuint64_t st[2] = {cuuint64_t(s.head_dim * 2), cuuint64_t(stride * 2)};
  cuuint32_t box[3] = {64, 1, kTile};
  return encode16(m, p, bf16, 3, dims, st, box, s.head_dim);
}
// [num_pages, page, kv_heads, D] as (D, kv_heads, page, num_pages), box (64, 1, min(page, 128), 1).
bool map_pages(CUtensorMap* m, const void* p, bool bf16, const evo_seq_shape_t& s, const evo_cache_shape_t& c,
               int64_t stride) {
  cuuint64_t dims[4] = {cuuint64_t(s.head_dim), cuuint64_t(s.kv_heads), cuuint64_t(c.page_size), cuuint64_t(c.num_pages)};
  cuuint64_t st[3] = {cuuint64_t(s.head_dim * 2), cuuint64_t(s.kv_heads * s.head_dim * 2), cuuint64_t(stride * 2)};
  cuuint32_t box[4] = {64, 1, cuuint32_t(c.page_size < kTile ? c.page_size : kTile), 1};
  return encode16(m, p, bf16, 4, dims, st, box, s.head_dim);
}

// Fills what both forwards share and launches; K and V maps are the caller's.
evo_status_t run_fwd(SeqFwdArgs& a, const void* q, const void* v, void* out, float* lse, void* workspace, int ctas,
                     const evo_seq_shape_t& s, bool bf16, const Strides& t, const Opts& o, cudaStream_t st) {
  const int G = static_cast<int>(s.q_heads / s.kv_heads);
  a.TQ = kTile / G;
  a.W = 2 * a.TQ;
  if (!map_q(&a.tq, q, bf16, s, t.q, a.TQ)) return EVO_ERR_CUDA;
  a.out32 = aligned(out, 32) && t.out % 16 == 0 && s.head_dim % 16 == 0;
  a.scale_log2 = scale_of(o, s) * kSeqLog2e;
  a.v = static_cast<const uint16_t*>(v);
  a.out = static_cast<uint16_t*>(out);
  a.out_stride = t.out;
  a.lse = lse;
  a.wait_ns = o.wait_ns;
  seq_fwd_workspace(ctas, static_cast<int>(s.head_dim), &a, static_cast<uint8_t*>(workspace));
  const cudaError_t e = launch_seq_fwd(a, ctas, bf16, st);
  return e == cudaSuccess ? EVO_OK : cuda_fail("sequence forward launch", e);
}

}  // namespace
}  // namespace evo

using namespace evo;

extern "C" {

size_t evo_prompt_fwd_workspace_bytes(evo_seq_shape_t shape) {
  if (check_seq_shape(shape, true) != EVO_OK) return 0;
  return seq_fwd_workspace(fwd_ctas(num_sms(), shape, shape.tokens), static_cast<int>(shape.head_dim), nullptr, nullptr);
}

size_t evo_prompt_bwd_workspace_bytes(evo_seq_shape_t shape) {
  if (check_seq_shape(shape, true) != EVO_OK) return 0;
  return prompt_bwd_workspace(bwd_ctas(num_sms(), shape), desc(shape, nullptr, nullptr, nullptr, nullptr, -1, nullptr),
                              nullptr, nullptr);
}

size_t evo_paged_fwd_workspace_bytes(evo_seq_shape_t shape, evo_cache_shape_t cache, int64_t weights_len) {
  int64_t a, b;
  if (check_seq_shape(shape, true) != EVO_OK || check_cache(cache, shape, &a, &b) != EVO_OK || weights_len < 0) return 0;
  return seq_fwd_workspace(fwd_ctas(num_sms(), shape, cache.page_size * cache.pages_per_seq),
                           static_cast<int>(shape.head_dim), nullptr, nullptr) +
         scores_bytes(shape, cache, weights_len);
}

evo_status_t evo_prompt_fwd(const void* q, const void* k, const void* v, const int32_t* cu_seqlens, void* out,
                            float* lse, void* workspace, size_t workspace_bytes, evo_seq_shape_t shape,
                            evo_dtype_t dtype, const evo_seq_strides_t* strides, const evo_seq_options_t* opts,
                            void* stream) {
  Opts o;
  if (!read_opts(opts, &o)) return EVO_ERR_BAD_ARGUMENT;
  if (dtype != EVO_F16 && dtype != EVO_BF16) return EVO_ERR_BAD_DTYPE;
  evo_status_t st = check_seq_shape(shape, true);
  if (st != EVO_OK) return st;
  Strides t;
  if (!read_strides(strides, shape, &t)) return EVO_ERR_BAD_LAYOUT;
  if (shape.tokens == 0 || shape.seqs == 0) return EVO_OK;
  if (!q || !k || !v || !cu_seqlens || !out || !lse || !workspace) return EVO_ERR_NULL_POINTER;
  if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(out, 16) || !aligned(cu_seqlens, 4) ||
      !aligned(lse, 4) || !aligned(workspace, 256) || !aligned(o.status, 4))
    return EVO_ERR_MISALIGNED;
  if (workspace_bytes < evo_prompt_fwd_workspace_bytes(shape)) return EVO_ERR_WORKSPACE_TOO_SMALL;
  const int64_t T = shape.tokens, nq = shape.q_heads * shape.head_dim, nk = shape.kv_heads * shape.head_dim;
  const Span in[] = {strided(q, T, t.q, nq), strided(k, T, t.k, nk), strided(v, T, t.v, nk),
                     flat(cu_seqlens, size_t(shape.seqs + 1) * 4)};
  const Span outs[] = {strided(out, T, t.out, nq), flat(lse, size_t(T) * shape.q_heads * 4),
                       flat(workspace, workspace_bytes)};
  if (aliased(in, outs)) return EVO_ERR_ALIASING;
  int sms = 0;
  int* fallback = nullptr;
  if ((st = host_device(&sms, &fallback)) != EVO_OK) return st;
  SeqFwdArgs a{};
  a.s = desc(shape, cu_seqlens, nullptr, nullptr, nullptr, -1, o.status ? o.status : fallback);
  const bool bf16 = dtype == EVO_BF16;
  if (!map_rows(&a.tk, k, bf16, shape, t.k) || !map_rows(&a.tv, v, bf16, shape, t.v)) return EVO_ERR_CUDA;
  a.v_stride = t.v;
  return run_fwd(a, q, v, out, lse, workspace, fwd_ctas(sms, shape, shape.tokens), shape, bf16, t, o,
                 static_cast<cudaStream_t>(stream));
}

evo_status_t evo_prompt_bwd(const void* q, const void* k, const void* v, const int32_t* cu_seqlens, const void* out,
                            const float* lse, const void* dout, void* dq, void* dk, void* dv, void* workspace,
                            size_t workspace_bytes, evo_seq_shape_t shape, evo_dtype_t dtype,
                            const evo_seq_strides_t* strides, const evo_seq_options_t* opts, void* stream) {
  Opts o;
  if (!read_opts(opts, &o)) return EVO_ERR_BAD_ARGUMENT;
  if (dtype != EVO_F16 && dtype != EVO_BF16) return EVO_ERR_BAD_DTYPE;
  evo_status_t st = check_seq_shape(shape, true);
  if (st != EVO_OK) return st;
  Strides t;
  if (!read_strides(strides, shape, &t)) return EVO_ERR_BAD_LAYOUT;
  if (shape.tokens == 0 || shape.seqs == 0) return EVO_OK;
  if (!q || !k || !v || !cu_seqlens || !out || !lse || !dout || !dq || !dk || !dv || !workspace)
    return EVO_ERR_NULL_POINTER;
  for (const void* p : {q, k, v, out, dout, static_cast<const void*>(dq), static_cast<const void*>(dk),
                        static_cast<const void*>(dv)})
    if (!aligned(p, 16)) return EVO_ERR_MISALIGNED;
  if (!aligned(cu_seqlens, 4) || !aligned(lse, 4) || !aligned(workspace, 256) || !aligned(o.status, 4))
    return EVO_ERR_MISALIGNED;
  if (workspace_bytes < evo_prompt_bwd_workspace_bytes(shape)) return EVO_ERR_WORKSPACE_TOO_SMALL;
  const int64_t T = shape.tokens, nq = shape.q_heads * shape.head_dim, nk = shape.kv_heads * shape.head_dim;
  const Span in[] = {strided(q, T, t.q, nq),       strided(k, T, t.k, nk),
                     strided(v, T, t.v, nk),       flat(cu_seqlens, size_t(shape.seqs + 1) * 4),
                     strided(out, T, t.out, nq),   flat(lse, size_t(T) * shape.q_heads * 4),
                     strided(dout, T, t.dout, nq)};
  const Span outs[] = {strided(dq, T, t.dq, nq), strided(dk, T, t.dk, nk), strided(dv, T, t.dv, nk),
                       flat(workspace, workspace_bytes)};
  if (aliased(in, outs)) return EVO_ERR_ALIASING;
  int sms = 0;
  int* fallback = nullptr;
  if ((st = host_device(&sms, &fallback)) != EVO_OK) return st;
  SeqBwdArgs a{};
  a.s = desc(shape, cu_seqlens, nullptr, nullptr, nullptr, -1, o.status ? o.status : fallback);
  a.TQ = kTile / a.s.group;
  const bool bf16 = dtype == EVO_BF16;
  if (!map_q(&a.tq, q, bf16, shape, t.q, a.TQ) || !map_q(&a.tdo, dout, bf16, shape, t.dout, a.TQ) ||
      !map_rows(&a.tk, k, bf16, shape, t.k) || !map_rows(&a.tv, v, bf16, shape, t.v))
    return EVO_ERR_CUDA;
  auto wide = [&](const void* p, long long stride) { return aligned(p, 32) && stride % 16 == 0 && shape.head_dim % 16 == 0; };
  a.dq32 = wide(dq, t.dq), a.dk32 = wide(dk, t.dk), a.dv32 = wide(dv, t.dv);
  a.scale = scale_of(o, shape);
  a.scale_log2 = a.scale * kSeqLog2e;
  a.out = static_cast<const uint16_t*>(out);
  a.dout = static_cast<const uint16_t*>(dout);
  a.lse = lse;
  a.dq = static_cast<uint16_t*>(dq);
  a.dk = static_cast<uint16_t*>(dk);
  a.dv = static_cast<uint16_t*>(dv);
  a.out_stride = t.out, a.dout_stride = t.dout, a.dq_stride = t.dq, a.dk_stride = t.dk, a.dv_stride = t.dv;
  a.wait_ns = o.wait_ns;
  const int rows = bwd_rows(sms, shape);
  const int most = bwd_ctas(sms, shape), ctas = rows * most > sms ? sms / rows : most;
  prompt_bwd_workspace(most, a.s, &a, static_cast<uint8_t*>(workspace));
  const cudaError_t e = launch_prompt_bwd(a, ctas, rows, bf16, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? EVO_OK : cuda_fail("prompt backward launch", e);
}

evo_status_t evo_cache_append(const void* k, const void* v, const int32_t* cu_seqlens, const int32_t* seq_lens,
                              const int32_t* block_table, void* k_pages, void* v_pages, evo_seq_shape_t shape,
                              evo_cache_shape_t cache, evo_dtype_t dtype, const evo_seq_strides_t* strides,
                              const evo_seq_options_t* opts, void* stream) {
  Opts o;
  if (!read_opts(opts, &o)) return EVO_ERR_BAD_ARGUMENT;
  if (dtype != EVO_F16 && dtype != EVO_BF16) return EVO_ERR_BAD_DTYPE;
  evo_status_t st = check_seq_shape(shape, false);
  if (st != EVO_OK) return st;
  shape.q_heads = shape.kv_heads;
  Strides t;
  int64_t kp, vp;
  if ((st = check_cache(cache, shape, &kp, &vp)) != EVO_OK) return st;
  evo_seq_strides_t only{};
  if (strides) only.k = strides->k, only.v = strides->v;
  if (!read_strides(&only, shape, &t)) return EVO_ERR_BAD_LAYOUT;
  if (shape.tokens == 0 || shape.seqs == 0) return EVO_OK;
  if (!k || !v || !cu_seqlens || !seq_lens || !block_table || !k_pages || !v_pages) return EVO_ERR_NULL_POINTER;
  if (!aligned(k, 16) || !aligned(v, 16) || !aligned(k_pages, 16) || !aligned(v_pages, 16) ||
      !aligned(cu_seqlens, 4) || !aligned(seq_lens, 4) || !aligned(block_table, 4) || !aligned(o.status, 4))
    return EVO_ERR_MISALIGNED;
  const int64_t nk = shape.kv_heads * shape.head_dim;
  const Span in[] = {strided(k, shape.tokens, t.k, nk), strided(v, shape.tokens, t.v, nk),
                     flat(cu_seqlens, size_t(shape.seqs + 1) * 4), flat(seq_lens, size_t(shape.seqs) * 4),
                     flat(block_table, size_t(shape.seqs) * size_t(cache.pages_per_seq) * 4)};
  const Span ks[] = {pages(k_pages, cache, shape, kp)}, vs[] = {pages(v_pages, cache, shape, vp)};
  if (aliased(in, ks) || aliased(in, vs) || overlap(ks[0], vs[0]))
    return EVO_ERR_ALIASING;
  int sms = 0;
  int* fallback = nullptr;
  if ((st = host_device(&sms, &fallback)) != EVO_OK) return st;
  AppendArgs a{};
  a.s = desc(shape, cu_seqlens, seq_lens, block_table, &cache, -1, o.status ? o.status : fallback);
  a.k = static_cast<const uint16_t*>(k);
  a.v = static_cast<const uint16_t*>(v);
  a.k_pages = static_cast<uint16_t*>(k_pages);
  a.v_pages = static_cast<uint16_t*>(v_pages);
  a.k_stride = t.k, a.v_stride = t.v, a.k_page = kp, a.v_page = vp;
  const cudaError_t e = launch_cache_append(a, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? EVO_OK : cuda_fail("cache append launch", e);
}

evo_status_t evo_paged_fwd(const void* q, const void* k_pages, const void* v_pages, const int32_t* cu_seqlens,
                           const int32_t* seq_lens, const int32_t* block_table, void* out, float* lse,
                           float* weights, int64_t weights_len, void* workspace, size_t workspace_bytes,
                           evo_seq_shape_t shape, evo_cache_shape_t cache, evo_dtype_t dtype,
                           const evo_seq_strides_t* strides, const evo_seq_options_t* opts, void* stream) {
  Opts o;
  if (!read_opts(opts, &o)) return EVO_ERR_BAD_ARGUMENT;
  if (dtype != EVO_F16 && dtype != EVO_BF16) return EVO_ERR_BAD_DTYPE;
  evo_status_t st = check_seq_shape(shape, true);
  if (st != EVO_OK) return st;
  int64_t kp, vp;
  if ((st = check_cache(cache, shape, &kp, &vp)) != EVO_OK) return st;
  if (weights && (weights_len < 1 || weights_len > (int64_t(1) << 40))) return EVO_ERR_BAD_SHAPE;
  evo_seq_strides_t only{};
  if (strides) only.q = strides->q, only.out = strides->out;
  Strides t;
  if (!read_strides(&only, shape, &t)) return EVO_ERR_BAD_LAYOUT;
  if (shape.tokens == 0 || shape.seqs == 0) return EVO_OK;
  if (!q || !k_pages || !v_pages || !cu_seqlens || !seq_lens || !block_table || !out || !lse || !workspace)
    return EVO_ERR_NULL_POINTER;
  if (!aligned(q, 16) || !aligned(k_pages, 16) || !aligned(v_pages, 16) || !aligned(out, 16) ||
      !aligned(cu_seqlens, 4) || !aligned(seq_lens, 4) || !aligned(block_table, 4) || !aligned(lse, 4) ||
      !aligned(weights, 4) || !aligned(workspace, 256) || !aligned(o.status, 4))
    return EVO_ERR_MISALIGNED;
  if (workspace_bytes < evo_paged_fwd_workspace_bytes(shape, cache, weights ? weights_len : 0)) return EVO_ERR_WORKSPACE_TOO_SMALL;
  const int64_t T = shape.tokens, nq = shape.q_heads * shape.head_dim;
  const Span in[] = {strided(q, T, t.q, nq),
                     pages(k_pages, cache, shape, kp),
                     pages(v_pages, cache, shape, vp),
                     flat(cu_seqlens, size_t(shape.seqs + 1) * 4),
                     flat(seq_lens, size_t(shape.seqs) * 4),
                     flat(block_table, size_t(shape.seqs) * size_t(cache.pages_per_seq) * 4)};
  const Span outs[] = {strided(out, T, t.out, nq), flat(lse, size_t(T) * shape.q_heads * 4),
                       flat(weights, weights ? size_t(shape.seqs) * shape.kv_heads * size_t(weights_len) * 4 : 0),
                       flat(workspace, workspace_bytes)};
  if (aliased(in, outs)) return EVO_ERR_ALIASING;
  int sms = 0;
  int* fallback = nullptr;
  if ((st = host_device(&sms, &fallback)) != EVO_OK) return st;
  SeqFwdArgs a{};
  a.s = desc(shape, cu_seqlens, seq_lens, block_table, &cache, weights ? weights_len : -1,
             o.status ? o.status : fallback);
  const bool bf16 = dtype == EVO_BF16;
  if (!map_pages(&a.tk, k_pages, bf16, shape, cache, kp) || !map_pages(&a.tv, v_pages, bf16, shape, cache, vp))
    return EVO_ERR_CUDA;
  a.v_page = vp;
  const int ctas = fwd_ctas(sms, shape, cache.page_size * cache.pages_per_seq);
  if (weights && scores_bytes(shape, cache, weights_len)) {
    a.scores = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) +
                                        seq_fwd_workspace(ctas, static_cast<int>(shape.head_dim), nullptr, nullptr));
    a.scores_ld = scores_row(cache, weights_len);
  }
  st = run_fwd(a, q, v_pages, out, lse, workspace, ctas, shape, bf16, t, o, static_cast<cudaStream_t>(stream));
  if (st != EVO_OK || !weights) return st;
  SeqWeightsArgs w{};
  w.tq = a.tq, w.tk = a.tk;
  w.s = a.s;
  w.TQ = a.TQ;
  w.scale_log2 = a.scale_log2;
  w.lse = lse;
  w.weights = weights;
  w.weights_len = weights_len;
  w.scores = a.scores;
  w.scores_ld = a.scores_ld;
  w.records = a.records;
  w.part = a.part_o;
  w.wait_ns = o.wait_ns;
  const cudaError_t e = launch_seq_weights(w, ctas, bf16, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? EVO_OK : cuda_fail("weight sums launch", e);
}

evo_status_t evo_cache_evict(void* k_pages, void* v_pages, const int32_t* block_table, int32_t* seq_lens,
                             float* weights, int64_t weights_len, int32_t* kept, int64_t budget, int64_t recent,
                             evo_seq_shape_t shape, evo_cache_shape_t cache, evo_dtype_t dtype,
                             const evo_seq_options_t* opts, void* stream) {
  Opts o;
  if (!read_opts(opts, &o)) return EVO_ERR_BAD_ARGUMENT;
  if (dtype != EVO_F16 && dtype != EVO_BF16) return EVO_ERR_BAD_DTYPE;
  shape.tokens = 0;
  evo_status_t st = check_seq_shape(shape, false);
  if (st != EVO_OK) return st;
  int64_t kp, vp;
  if ((st = check_cache(cache, shape, &kp, &vp)) != EVO_OK) return st;
  if (weights_len < 1 || weights_len > (int64_t(1) << 40)) return EVO_ERR_BAD_SHAPE;
  if (budget < 1 || budget > (int64_t(1) << 30) || recent < 0 || recent > budget) return EVO_ERR_BAD_ARGUMENT;
  if (shape.seqs == 0) return EVO_OK;
  if (!k_pages || !v_pages || !block_table || !seq_lens || !weights || !kept) return EVO_ERR_NULL_POINTER;
  if (!aligned(k_pages, 16) || !aligned(v_pages, 16) || !aligned(block_table, 4) || !aligned(seq_lens, 4) ||
      !aligned(weights, 4) || !aligned(kept, 4) || !aligned(o.status, 4))
    return EVO_ERR_MISALIGNED;
  const Span in[] = {flat(block_table, size_t(shape.seqs) * size_t(cache.pages_per_seq) * 4)};
  const Span small[] = {flat(seq_lens, size_t(shape.seqs) * 4),
                        flat(weights, size_t(shape.seqs) * shape.kv_heads * size_t(weights_len) * 4),
                        flat(kept, size_t(shape.seqs) * shape.kv_heads * size_t(budget) * 4)};
  const Span ks[] = {pages(k_pages, cache, shape, kp)}, vs[] = {pages(v_pages, cache, shape, vp)};
  if (aliased(in, small) || aliased(in, ks) || aliased(in, vs) || aliased(small, ks) || aliased(small, vs) ||
      overlap(ks[0], vs[0]))
    return EVO_ERR_ALIASING;
  int sms = 0;
  int* fallback = nullptr;
  if ((st = host_device(&sms, &fallback)) != EVO_OK) return st;
  EvictArgs a{};
  a.s = desc(shape, nullptr, seq_lens, block_table, &cache, weights_len, o.status ? o.status : fallback);
  a.k_pages = static_cast<uint16_t*>(k_pages);
  a.v_pages = static_cast<uint16_t*>(v_pages);
  a.k_page = kp, a.v_page = vp;
  a.seq_lens = seq_lens;
  a.weights = weights;
  a.weights_len = weights_len;
  a.kept = kept;
  a.budget = static_cast<int>(budget);
  a.recent = static_cast<int>(recent);
  const cudaError_t e = launch_cache_evict(a, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? EVO_OK : cuda_fail("cache evict launch", e);
}

}  // extern "C"
