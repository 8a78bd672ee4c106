// evo_seq_simple.cu — attention over causal sequences (include/evo_seq.h), one
// warp per output row: the forward over prompts and paged caches, the sums of the
// attention weights, and the prompt's gradients.  Definitions in the header.
#include <cmath>

#include "evo_seq_internal.h"

namespace evo {
namespace {

constexpr int kMaxPerLane = 4;  // head_dim <= 128

// Row (token, head) as fp32, element lane + 32 e in x[e].
template <bool BF16>
__device__ __forceinline__ void load_row(const uint16_t* p, int D, int lane, float (&x)[kMaxPerLane]) {
#pragma unroll
  for (int e = 0; e < kMaxPerLane; ++e) {
    const int d = lane + 32 * e;
    x[e] = d < D ? to_f32<BF16>(p[d]) : 0.0f;
  }
}
template <bool BF16>
__device__ __forceinline__ void store_row(uint16_t* p, int D, int lane, const float (&x)[kMaxPerLane]) {
#pragma unroll
  for (int e = 0; e < kMaxPerLane; ++e) {
    const int d = lane + 32 * e;
    if (d < D) p[d] = static_cast<uint16_t>(pack2<BF16>(x[e], 0.0f) & 0xffffu);
  }
}
__device__ __forceinline__ float dot(const float (&x)[kMaxPerLane], const float (&y)[kMaxPerLane]) {
  float s = 0.0f;
#pragma unroll
  for (int e = 0; e < kMaxPerLane; ++e) s = fmaf(x[e], y[e], s);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  return s;
}
__device__ __forceinline__ const uint16_t* key_row(const SeqAttnArgs& a, const uint16_t* base, long long stride,
                                                   long long page_stride, const Seq& q, int b, int j, int h) {
  const SeqDesc& s = a.s;
  if (!s.table) return base + (q.row0 + j) * stride + static_cast<long long>(h) * s.D;
  const int p = page_of(s, b, j);
  if (p < 0) return nullptr;
  return base + p * page_stride + (static_cast<long long>(j % s.page) * s.kv_heads + h) * s.D;
}
template <bool BF16>
__device__ __forceinline__ void load_key(const SeqAttnArgs& a, const uint16_t* base, long long stride,
                                         long long page_stride, const Seq& q, int b, int j, int h, int lane,
                                         float (&x)[kMaxPerLane]) {
  const uint16_t* p = key_row(a, base, stride, page_stride, q, b, j, h);
  if (p)
    load_row<BF16>(p, a.s.D, lane, x);
  else
    for (int e = 0; e < kMaxPerLane; ++e) x[e] = 0.0f;
}

// weights[b][h][j] += Σ P: one warp per (b, h, j), rows in order.
template <bool BF16>
__global__ void seq_weights_simple(const SeqAttnArgs a) {
  const SeqDesc& s = a.s;
  const int lane = threadIdx.x & 31, hk = blockIdx.y, b = blockIdx.z;
  const Seq q = load_seq(s, b);
  for (int j = blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5); j < q.kv; j += gridDim.x * (blockDim.x >> 5)) {
    float kr[kMaxPerLane], qr[kMaxPerLane];
    load_key<BF16>(a, a.k, a.k_stride, a.k_page, q, b, j, hk, lane, kr);
    float sum = 0.0f;
    for (int i = j > q.pos0 ? j - q.pos0 : 0; i < q.n; ++i) {
      for (int g = 0; g < s.group; ++g) {
        const int h = hk * s.group + g, t = q.row0 + i;
        load_row<BF16>(a.q + t * a.q_stride + h * s.D, s.D, lane, qr);
        const float z = a.lse[static_cast<size_t>(h) * s.tokens + t];
        sum += z == -INFINITY ? 0.0f : expf(dot(qr, kr) * a.scale - z);
      }
    }
    if (lane == 0) a.weights[(static_cast<size_t>(b) * s.kv_heads + hk) * a.weights_len + j] += sum;
  }
}

constexpr int kWarps = 8;

}  // namespace

cudaError_t launch_seq_weights(const SeqAttnArgs& a, bool bf16, cudaStream_t st) {
  const dim3 grid(256, a.s.kv_heads, a.s.seqs);
  if (bf16)
    seq_weights_simple<true><<<grid, kWarps * 32, 0, st>>>(a);
  else
    seq_weights_simple<false><<<grid, kWarps * 32, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace evo
