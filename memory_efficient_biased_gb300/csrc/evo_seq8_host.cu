// evo_seq8_host.cu — the C ABI of the 8-bit cache (include/evo_seq.h): argument validation,
// workspace sizes and dispatch to the kernels.
#include "evo_seq8_internal.h"
#include "evo_seq_check.h"

namespace evo {
namespace {

// The cache's pages as bytes, its scales, and the same as the 16-bit cache's shape (for desc).
struct Checked {
  int64_t k_page, v_page, scales;  // strides of the pages; scales of each of k and v
  evo_cache_shape_t as16;
};
evo_status_t check_cache8(const evo_cache8_shape_t& c, const evo_seq_shape_t& s, Checked* o) {
  const bool block_ok = c.scale_block == 16 || c.scale_block == 32 || c.scale_block == 64 || c.scale_block == 128;
  if (s.head_dim % 16 || !page_size_ok(c.page_size) || !block_ok || c.page_size % c.scale_block || c.num_pages < 1 ||
      c.num_pages > (int64_t(1) << 31) - 2 || c.pages_per_seq < 1 || c.pages_per_seq > (int64_t(1) << 31) - 1)
    return EVO_ERR_BAD_SHAPE;
  const int64_t packed = c.page_size * s.kv_heads * s.head_dim;
  o->k_page = c.k_page_stride ? c.k_page_stride : packed;
  o->v_page = c.v_page_stride ? c.v_page_stride : packed;
  for (int64_t p : {o->k_page, o->v_page})
    if (p < packed || p % 16 || p >= kMaxStride) return EVO_ERR_BAD_LAYOUT;
  o->scales = c.num_pages * s.kv_heads * (c.page_size / c.scale_block);
  o->as16 = evo_cache_shape_t{c.num_pages, c.page_size, c.pages_per_seq, 0, 0};
  return EVO_OK;
}

Span pages8(const void* p, const evo_cache8_shape_t& c, const evo_seq_shape_t& s, int64_t stride) {
  const int64_t piece = c.page_size * s.kv_heads * s.head_dim;
  return {p, size_t(c.num_pages - 1) * size_t(stride) + size_t(piece), stride, piece};
}

Cache8 cache_of(const void* k_pages, const void* v_pages, const float* k_scales, const float* v_scales,
                const evo_cache8_shape_t& c, const Checked& k) {
  Cache8 o{};
  o.k_pages = static_cast<uint8_t*>(const_cast<void*>(k_pages));
  o.v_pages = static_cast<uint8_t*>(const_cast<void*>(v_pages));
  o.k_scales = const_cast<float*>(k_scales);
  o.v_scales = const_cast<float*>(v_scales);
  o.k_page = k.k_page, o.v_page = k.v_page;
  o.block = static_cast<int>(c.scale_block);
  o.blocks = static_cast<int>(c.page_size / c.scale_block);
  return o;
}

// Pages as (D, kv_heads, page, num_pages), box (DP, 1, min(page, 128), 1): a row of codes is a swizzled row of the tile.
bool map_pages8(CUtensorMap* m, const void* p, const evo_seq_shape_t& s, const evo_cache8_shape_t& c, int64_t stride) {
  const int64_t D = s.head_dim, DP = D <= 64 ? 64 : 128;
  cuuint64_t dims[4] = {cuuint64_t(D), cuuint64_t(s.kv_heads), cuuint64_t(c.page_size), cuuint64_t(c.num_pages)};
  cuuint64_t st[3] = {cuuint64_t(D), cuuint64_t(s.kv_heads * D), cuuint64_t(stride)};
  cuuint32_t box[4] = {cuuint32_t(DP), 1, cuuint32_t(c.page_size < kTile ? c.page_size : kTile), 1};
  return host_encode(m, p, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, dims, st, box,
                     DP == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                     CU_TENSOR_MAP_L2_PROMOTION_L2_128B);
}

// Which kernels, and their launch.
//   few    up to 32 rows a sequence and kv head on the average, and a token's heads in one tile of 16.  The cache is then read
//          twice, at 6 TB/s, where the other kernel widens it once, at 1.8.  Measured, 32 rows of few / of the other:
//          16 contexts of 8192 (8 kv heads of 128) 112 / 143 us, 2 of 16,384 43 / 47, 32 of 2048 92 / 95, one of
//          100,000 89 / 112, 64 of 700 107 / 100; 48 rows 158 / 145, 52 / 48, 106 / 96, 119 / 114, 139 / 101.  The average says nothing
//          of uneven batches: one chunk of 512 tokens over 16,000 beside 128 single tokens over 2000 each goes to few and takes 814
//          us, 496 the other way, its parts by themselves 142 and 127
//   copy   many rows, and the codes are widened once, into the workspace, for the 16-bit forward; otherwise every block of 256
//          rows widens them as it needs them.  The copy costs 6 bytes a code and a launch; widening in place what it takes
//          beside the products.  So: from more than two blocks a sequence on, while the copy of all that the table can hold stays below
//          512 MB.  Measured, in place / copied, 8 kv heads with group 4 of 128 unless given: two contexts of 16,384 4 blocks each
//          155 / 164 us, 6 221 / 215, 8 286 / 266; one of 23,348 21 blocks 509 / 424, of 16,384 64 blocks 948 / 767;
//          head_dim 64, one of 12,291 3.5 blocks 63 / 63, of 5000 4 blocks 37 / 43.  Where most rows are those of few sequences,
//          the average says too little of them: 5.2 blocks, 1325 tokens over 23,348 in all, 200 / 168; hence two, not six.
//   whole  few rows, contexts of at most 1024 keys and no more items than SMs: no item is cut, nothing is joined.  An SM takes
//          0.7 us a tile, a second launch 3 and the host 4 (777 keys of 8 heads: 12 us of GPU either way, 22 and 26 a call).
size_t round_up(size_t bytes) { return (bytes + 255) & ~size_t(255); }
struct Plan {
  bool few, whole;
  int ctas, rows;  // rows: of a piece
  size_t copy;     // many rows: bytes of the keys' (and of the values') copy in 16 bits; 0: none is made
};
constexpr int64_t kWholeKeys = 1024, kCopyRows = 512;
constexpr double kCopyBytes = 512.0 * 1024 * 1024;
Plan plan(int sms, const evo_seq_shape_t& s, const evo_cache8_shape_t& c) {
  const int64_t G = s.q_heads / s.kv_heads, max_kv = c.page_size * c.pages_per_seq;
  Plan p{};
  p.few = G <= kFewRows && s.tokens * G <= 2 * kFewRows * s.seqs;
  if (!p.few) {
    p.ctas = fwd_ctas(sms, s, max_kv);
    p.rows = 256;
    const double copy = 2.0 * double(s.seqs) * double(max_kv) * double(s.kv_heads) * double(s.head_dim);
    p.copy = s.tokens * G > kCopyRows * s.seqs && 2 * copy <= kCopyBytes ? round_up(static_cast<size_t>(copy)) : 0;
    return p;
  }
  p.rows = kFewRows;
  const double items = (double(s.tokens) / double(kFewRows / G) + double(s.seqs)) * double(s.kv_heads);
  p.whole = max_kv <= kTile || (max_kv <= kWholeKeys && items <= sms);
  const double most = p.whole ? items : items * (double(max_kv) / kTile + 2);  // CTAs that the work can fill
  p.ctas = most < sms ? static_cast<int>(most) + 1 : sms;
  return p;
}
size_t table_bytes(const evo_seq_shape_t& s, const evo_cache8_shape_t& c) { return round_up(size_t(s.seqs) * size_t(c.pages_per_seq) * 4); }
evo_cache_shape_t copy_shape(const evo_seq_shape_t& s, const evo_cache8_shape_t& c) {
  return {s.seqs * c.pages_per_seq, c.page_size, c.pages_per_seq, 0, 0};
}
size_t workspace_of(const Plan& p, const evo_seq_shape_t& s, const evo_cache8_shape_t& c, SeqFwdArgs* a, void* ws) {
  if (p.copy) return 2 * p.copy + table_bytes(s, c) + evo_paged_fwd_workspace_bytes(s, copy_shape(s, c), 0);
  return p.whole ? 0 : seq_fwd_workspace(p.ctas, static_cast<int>(s.head_dim), a, static_cast<uint8_t*>(ws), p.rows);
}

// What an append and a read check alike.
evo_status_t rows_call(bool append, const void* k, const void* v, const int32_t* cu_seqlens, const int32_t* seq_lens,
                       const int32_t* block_table, const void* k_pages, const void* v_pages, const float* k_scales,
                       const float* v_scales, evo_seq_shape_t shape, const evo_cache8_shape_t& cache, evo_dtype_t dtype,
                       const evo_seq_strides_t* strides, const evo_seq_options_t* opts, void* stream) {
  Opts o;
  if (!read_opts(opts, &o)) return EVO_ERR_BAD_ARGUMENT;
  if (dtype != EVO_F16 && dtype != EVO_BF16) return EVO_ERR_BAD_DTYPE;
  evo_status_t st = check_seq_shape(shape, false);
  if (st != EVO_OK) return st;
  shape.q_heads = shape.kv_heads;
  Strides t;
  Checked c;
  if ((st = check_cache8(cache, shape, &c)) != EVO_OK) return st;
  evo_seq_strides_t only{};
  if (strides) only.k = strides->k, only.v = strides->v;
  if (!read_strides(&only, shape, &t)) return EVO_ERR_BAD_LAYOUT;
  if (shape.tokens == 0 || shape.seqs == 0) return EVO_OK;
  if (!k || !v || !cu_seqlens || !seq_lens || !block_table || !k_pages || !v_pages || !k_scales || !v_scales)
    return EVO_ERR_NULL_POINTER;
  if (!aligned(k, 16) || !aligned(v, 16) || !aligned(k_pages, 16) || !aligned(v_pages, 16) || !aligned(cu_seqlens, 4) ||
      !aligned(seq_lens, 4) || !aligned(block_table, 4) || !aligned(k_scales, 4) || !aligned(v_scales, 4) ||
      !aligned(o.status, 4))
    return EVO_ERR_MISALIGNED;
  const int64_t nk = shape.kv_heads * shape.head_dim;
  const Span plan[] = {flat(cu_seqlens, size_t(shape.seqs + 1) * 4), flat(seq_lens, size_t(shape.seqs) * 4),
                       flat(block_table, size_t(shape.seqs) * size_t(cache.pages_per_seq) * 4)};
  const Span rows[] = {strided(k, shape.tokens, t.k, nk), strided(v, shape.tokens, t.v, nk)};
  const Span held[] = {pages8(k_pages, cache, shape, c.k_page), pages8(v_pages, cache, shape, c.v_page),
                       flat(k_scales, size_t(c.scales) * 4), flat(v_scales, size_t(c.scales) * 4)};
  // what is written overlaps neither what is read nor itself
  if (append ? aliased(plan, held) || aliased(rows, held) : aliased(plan, rows) || aliased(held, rows)) return EVO_ERR_ALIASING;
  int sms = 0;
  int* fallback = nullptr;
  if ((st = host_device(&sms, &fallback)) != EVO_OK) return st;
  Cache8Args a{};
  a.s = desc(shape, cu_seqlens, seq_lens, block_table, &c.as16, -1, o.status ? o.status : fallback);
  a.c = cache_of(k_pages, v_pages, k_scales, v_scales, cache, c);
  a.k = static_cast<uint16_t*>(const_cast<void*>(k));
  a.v = static_cast<uint16_t*>(const_cast<void*>(v));
  a.k_stride = t.k, a.v_stride = t.v;
  a.wide = aligned(k, 32) && aligned(v, 32) && t.k % 16 == 0 && t.v % 16 == 0;
  const bool bf16 = dtype == EVO_BF16;
  const cudaStream_t cs = static_cast<cudaStream_t>(stream);
  const cudaError_t e = append ? launch_cache8_append(a, bf16, cs) : launch_cache8_read(a, sms, bf16, cs);
  return e == cudaSuccess ? EVO_OK : cuda_fail(append ? "8-bit cache append launch" : "8-bit cache read launch", e);
}

}  // namespace
}  // namespace evo

using namespace evo;

extern "C" {

evo_status_t evo_cache8_append(const void* k, const void* v, const int32_t* cu_seqlens, const int32_t* seq_lens,
                               const int32_t* block_table, void* k_pages, void* v_pages, float* k_scales,
                               float* v_scales, evo_seq_shape_t shape, evo_cache8_shape_t cache, evo_dtype_t dtype,
                               const evo_seq_strides_t* strides, const evo_seq_options_t* opts, void* stream) {
  return rows_call(true, k, v, cu_seqlens, seq_lens, block_table, k_pages, v_pages, k_scales, v_scales, shape, cache,
                   dtype, strides, opts, stream);
}

evo_status_t evo_cache8_read(const void* k_pages, const void* v_pages, const float* k_scales, const float* v_scales,
                             const int32_t* cu_seqlens, const int32_t* seq_lens, const int32_t* block_table, void* k,
                             void* v, evo_seq_shape_t shape, evo_cache8_shape_t cache, evo_dtype_t dtype,
                             const evo_seq_strides_t* strides, const evo_seq_options_t* opts, void* stream) {
  return rows_call(false, k, v, cu_seqlens, seq_lens, block_table, k_pages, v_pages, k_scales, v_scales, shape, cache,
                   dtype, strides, opts, stream);
}

size_t evo_paged8_fwd_workspace_bytes(evo_seq_shape_t shape, evo_cache8_shape_t cache) {
  Checked c;
  if (check_seq_shape(shape, true) != EVO_OK || check_cache8(cache, shape, &c) != EVO_OK) return 0;
  return workspace_of(plan(num_sms(), shape, cache), shape, cache, nullptr, nullptr);
}

evo_status_t evo_paged8_fwd(const void* q, const void* k_pages, const void* v_pages, const float* k_scales,
                            const float* v_scales, const int32_t* cu_seqlens, const int32_t* seq_lens,
                            const int32_t* block_table, void* out, float* lse, void* workspace, size_t workspace_bytes,
                            evo_seq_shape_t shape, evo_cache8_shape_t cache, evo_dtype_t dtype,
                            const evo_seq_strides_t* strides, const evo_seq_options_t* opts, void* stream) {
  Opts o;
  if (!read_opts(opts, &o)) return EVO_ERR_BAD_ARGUMENT;
  if (dtype != EVO_F16 && dtype != EVO_BF16) return EVO_ERR_BAD_DTYPE;
  evo_status_t st = check_seq_shape(shape, true);
  if (st != EVO_OK) return st;
  Checked c;
  if ((st = check_cache8(cache, shape, &c)) != EVO_OK) return st;
  evo_seq_strides_t only{};
  if (strides) only.q = strides->q, only.out = strides->out;
  Strides t;
  if (!read_strides(&only, shape, &t)) return EVO_ERR_BAD_LAYOUT;
  if (shape.tokens == 0 || shape.seqs == 0) return EVO_OK;
  const size_t need = evo_paged8_fwd_workspace_bytes(shape, cache);
  if (!q || !k_pages || !v_pages || !k_scales || !v_scales || !cu_seqlens || !seq_lens || !block_table || !out || !lse ||
      (need && !workspace))
    return EVO_ERR_NULL_POINTER;
  if (!aligned(q, 16) || !aligned(k_pages, 16) || !aligned(v_pages, 16) || !aligned(out, 16) || !aligned(k_scales, 4) ||
      !aligned(v_scales, 4) || !aligned(cu_seqlens, 4) || !aligned(seq_lens, 4) || !aligned(block_table, 4) ||
      !aligned(lse, 4) || !aligned(workspace, 256) || !aligned(o.status, 4))
    return EVO_ERR_MISALIGNED;
  if (workspace_bytes < need) return EVO_ERR_WORKSPACE_TOO_SMALL;
  const int64_t T = shape.tokens, nq = shape.q_heads * shape.head_dim;
  const Span in[] = {strided(q, T, t.q, nq),
                     pages8(k_pages, cache, shape, c.k_page),
                     pages8(v_pages, cache, shape, c.v_page),
                     flat(k_scales, size_t(c.scales) * 4),
                     flat(v_scales, size_t(c.scales) * 4),
                     flat(cu_seqlens, size_t(shape.seqs + 1) * 4),
                     flat(seq_lens, size_t(shape.seqs) * 4),
                     flat(block_table, size_t(shape.seqs) * size_t(cache.pages_per_seq) * 4)};
  const Span outs[] = {strided(out, T, t.out, nq), flat(lse, size_t(T) * shape.q_heads * 4),
                       flat(workspace, workspace_bytes)};
  if (aliased(in, outs)) return EVO_ERR_ALIASING;
  int sms = 0;
  int* fallback = nullptr;
  if ((st = host_device(&sms, &fallback)) != EVO_OK) return st;
  const Plan p = plan(sms, shape, cache);
  const bool bf16 = dtype == EVO_BF16;
  const cudaStream_t cs = static_cast<cudaStream_t>(stream);
  if (p.copy) {
    uint8_t* at = static_cast<uint8_t*>(workspace);
    Cache8Args w{};
    w.s = desc(shape, cu_seqlens, seq_lens, block_table, &c.as16, -1, o.status ? o.status : fallback);
    w.c = cache_of(k_pages, v_pages, k_scales, v_scales, cache, c);
    w.k = reinterpret_cast<uint16_t*>(at);
    w.v = reinterpret_cast<uint16_t*>(at + p.copy);
    int* table = reinterpret_cast<int*>(at + 2 * p.copy);
    const cudaError_t e = launch_cache8_copy(w, table, sms, bf16, cs);
    if (e != cudaSuccess) return cuda_fail("8-bit cache copy launch", e);
    const size_t used = 2 * p.copy + table_bytes(shape, cache);
    return evo_paged_fwd(q, w.k, w.v, cu_seqlens, seq_lens, table, out, lse, nullptr, 0, at + used, workspace_bytes - used,
                         shape, copy_shape(shape, cache), dtype, strides, opts, stream);
  }
  Seq8FwdArgs a{};
  a.f.s = desc(shape, cu_seqlens, seq_lens, block_table, &c.as16, -1, o.status ? o.status : fallback);
  a.c = cache_of(k_pages, v_pages, k_scales, v_scales, cache, c);
  a.q = static_cast<const uint16_t*>(q);
  a.q_stride = t.q;
  a.f.out = static_cast<uint16_t*>(out);
  a.f.out_stride = t.out;
  a.f.lse = lse;
  a.f.scale_log2 = scale_of(o, shape) * kSeqLog2e;
  a.f.wait_ns = o.wait_ns;
  a.f.TQ = kTile / a.f.s.group;
  if (!map_pages8(&a.f.tk, k_pages, shape, cache, c.k_page) || !map_pages8(&a.f.tv, v_pages, shape, cache, c.v_page))
    return EVO_ERR_CUDA;
  workspace_of(p, shape, cache, &a.f, workspace);
  a.whole = p.whole;
  cudaError_t e;
  if (p.few) {
    a.f.W = kFewRows / a.f.s.group;
    e = launch_paged8_few(a, p.ctas, bf16, cs);
  } else {
    a.f.W = 2 * a.f.TQ;
    a.f.out32 = aligned(out, 32) && t.out % 16 == 0;
    if (!map_q(&a.f.tq, q, bf16, shape, t.q, a.f.TQ)) return EVO_ERR_CUDA;
    e = launch_paged8_tiles(a, p.ctas, bf16, cs);
  }
  return e == cudaSuccess ? EVO_OK : cuda_fail("8-bit cache attention launch", e);
}

}  // extern "C"
