// evo_seq8_fwd.cu — attention of new tokens over the 8-bit cache (include/evo_seq.h).
//
// Mathematics, per row (token, head): S = (q·code_k) s_k, m the running maximum of s·log2e·S, P = 2^(s·log2e·S - m),
// l = Σ P and O = Σ P s_v code_v over the keys seen so far; at the end O / l and lse = ln2·(m + log2 l).
//
// A warp a row, four features a lane, key by key.
#include "evo_seq8_internal.h"

namespace evo {
namespace {

template <bool BF16>
__global__ void __launch_bounds__(256) evo_paged8_rows_kernel(const __grid_constant__ Seq8FwdArgs a) {
  const SeqDesc& s = a.f.s;
  const Cache8& c = a.c;
  if (blockIdx.x == 0) check_seqs(s);
  const int lane = threadIdx.x & 31, d = lane * 4;
  const long long rows = static_cast<long long>(s.tokens) * s.q_heads, warps = static_cast<long long>(gridDim.x) * 8;
  for (long long r = static_cast<long long>(blockIdx.x) * 8 + (threadIdx.x >> 5); r < rows; r += warps) {
    const int t = static_cast<int>(r / s.q_heads), h = static_cast<int>(r % s.q_heads), e = h / s.group;
    const int b = find_seq(s, t);
    if (b < 0) continue;
    const Seq q = load_seq(s, b);
    if (t < q.row0 || t >= q.row0 + q.n) continue;
    const int end = q.pos0 + (t - q.row0) + 1;  // keys that it sees
    const bool has = d < s.D;
    float x[4] = {}, o[4] = {}, m = -INFINITY, l = 0.0f;
    if (has) {
      const uint2 u = *reinterpret_cast<const uint2*>(a.q + t * a.q_stride + static_cast<long long>(h) * s.D + d);
      const float2 f0 = unpack2<BF16>(u.x), f1 = unpack2<BF16>(u.y);
      x[0] = f0.x, x[1] = f0.y, x[2] = f1.x, x[3] = f1.y;
    }
    for (int j = 0; j < end; ++j) {
      const int p = page_of(s, b, j);
      const long long at = (static_cast<long long>(j % s.page) * s.kv_heads + e) * s.D + d;
      float k[4] = {}, v[4] = {}, sk = 1.0f, sv = 1.0f;
      if (p >= 0) {
        sk = c.k_scales[scale_at(c, s, p, e, j)];
        sv = c.v_scales[scale_at(c, s, p, e, j)];
        if (has) {
          const uint32_t ku = *reinterpret_cast<const uint32_t*>(c.k_pages + p * c.k_page + at);
          const uint32_t vu = *reinterpret_cast<const uint32_t*>(c.v_pages + p * c.v_page + at);
          const uint2 k2 = f16x4_of_codes(ku), v2 = f16x4_of_codes(vu);
          const float2 k0 = unpack2<false>(k2.x), k1 = unpack2<false>(k2.y), v0 = unpack2<false>(v2.x), v1 = unpack2<false>(v2.y);
          k[0] = k0.x, k[1] = k0.y, k[2] = k1.x, k[3] = k1.y;
          v[0] = v0.x, v[1] = v0.y, v[2] = v1.x, v[3] = v1.y;
        }
      }
      float y = x[0] * k[0] + x[1] * k[1] + x[2] * k[2] + x[3] * k[3];
#pragma unroll
      for (int w = 16; w > 0; w >>= 1) y += __shfl_xor_sync(0xffffffffu, y, w);
      y *= sk * a.f.scale_log2;
      if (y == -INFINITY) continue;
      const float big = fmaxf(m, y), f = m == -INFINITY ? 0.0f : ex2(m - big), w = ex2(y - big);
      m = y != y ? y : big;  // (a NaN score makes the row NaN)
      l = l * f + w;
#pragma unroll
      for (int i = 0; i < 4; ++i) o[i] = o[i] * f + w * sv * v[i];
    }
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
    if (has)
      *reinterpret_cast<uint2*>(a.f.out + t * a.f.out_stride + static_cast<long long>(h) * s.D + d) =
          l == 0.0f ? make_uint2(0u, 0u) : make_uint2(pack2<BF16>(o[0] * inv, o[1] * inv), pack2<BF16>(o[2] * inv, o[3] * inv));
    if (lane == 0) a.f.lse[static_cast<size_t>(h) * s.tokens + t] = l == 0.0f ? -INFINITY : (m + lg2(l)) * kSeqLn2;
  }
}

}  // namespace

cudaError_t launch_paged8_rows(const Seq8FwdArgs& a, bool bf16, cudaStream_t st) {
  const long long blocks = (static_cast<long long>(a.f.s.tokens) * a.f.s.q_heads + 7) / 8;
  const unsigned grid = static_cast<unsigned>(blocks < (1 << 20) ? blocks : (1 << 20));
  if (bf16)
    evo_paged8_rows_kernel<true><<<grid, 256, 0, st>>>(a);
  else
    evo_paged8_rows_kernel<false><<<grid, 256, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace evo
