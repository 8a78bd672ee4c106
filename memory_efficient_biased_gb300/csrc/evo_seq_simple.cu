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

template <bool BF16>
__global__ void prompt_delta_simple(const SeqAttnArgs a) {
  const SeqDesc& s = a.s;
  if (blockIdx.x == 0 && blockIdx.y == 0) check_seqs(s);
  const int lane = threadIdx.x & 31, h = blockIdx.y;
  const int t = blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
  if (t >= s.tokens) return;
  float x[kMaxPerLane], y[kMaxPerLane];
  load_row<BF16>(a.out + t * a.out_stride + h * s.D, s.D, lane, x);
  load_row<BF16>(a.dout + t * a.dout_stride + h * s.D, s.D, lane, y);
  const float d = dot(x, y);
  if (lane == 0) a.delta[static_cast<size_t>(h) * s.tokens + t] = d;
}

template <bool BF16>
__global__ void prompt_dq_simple(const SeqAttnArgs a) {
  const SeqDesc& s = a.s;
  if (blockIdx.x == 0 && blockIdx.y == 0) check_seqs(s);
  const int lane = threadIdx.x & 31, h = blockIdx.y;
  const int t = blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
  if (t >= s.tokens) return;
  const int b = find_seq(s, t);
  if (b < 0) return;
  const Seq q = load_seq(s, b);
  if (t < q.row0 || t >= q.row0 + q.n) return;
  const int hk = h / s.group;
  float qr[kMaxPerLane], dor[kMaxPerLane], kr[kMaxPerLane], vr[kMaxPerLane], g[kMaxPerLane] = {};
  load_row<BF16>(a.q + t * a.q_stride + h * s.D, s.D, lane, qr);
  load_row<BF16>(a.dout + t * a.dout_stride + h * s.D, s.D, lane, dor);
  const size_t at = static_cast<size_t>(h) * s.tokens + t;
  const float z = a.lse[at], delta = a.delta[at];
  for (int j = 0; j <= t - q.row0; ++j) {
    load_key<BF16>(a, a.k, a.k_stride, a.k_page, q, b, j, hk, lane, kr);
    load_key<BF16>(a, a.v, a.v_stride, a.v_page, q, b, j, hk, lane, vr);
    const float p = z == -INFINITY ? 0.0f : expf(dot(qr, kr) * a.scale - z);
    const float ds = p * (dot(dor, vr) - delta) * a.scale;
#pragma unroll
    for (int e = 0; e < kMaxPerLane; ++e) g[e] = fmaf(ds, kr[e], g[e]);
  }
  store_row<BF16>(a.dq + t * a.dq_stride + h * s.D, s.D, lane, g);
}

template <bool BF16>
__global__ void prompt_dkv_simple(const SeqAttnArgs a) {
  const SeqDesc& s = a.s;
  const int lane = threadIdx.x & 31, hk = blockIdx.y;
  const int t = blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
  if (t >= s.tokens) return;
  const int b = find_seq(s, t);
  if (b < 0) return;
  const Seq q = load_seq(s, b);
  if (t < q.row0 || t >= q.row0 + q.n) return;
  float qr[kMaxPerLane], dor[kMaxPerLane], kr[kMaxPerLane], vr[kMaxPerLane], gk[kMaxPerLane] = {}, gv[kMaxPerLane] = {};
  load_row<BF16>(a.k + t * a.k_stride + hk * s.D, s.D, lane, kr);
  load_row<BF16>(a.v + t * a.v_stride + hk * s.D, s.D, lane, vr);
  for (int i = t; i < q.row0 + q.n; ++i) {
    for (int g = 0; g < s.group; ++g) {
      const int h = hk * s.group + g;
      load_row<BF16>(a.q + i * a.q_stride + h * s.D, s.D, lane, qr);
      load_row<BF16>(a.dout + i * a.dout_stride + h * s.D, s.D, lane, dor);
      const size_t at = static_cast<size_t>(h) * s.tokens + i;
      const float z = a.lse[at], delta = a.delta[at];
      const float p = z == -INFINITY ? 0.0f : expf(dot(qr, kr) * a.scale - z);
      const float ds = p * (dot(dor, vr) - delta) * a.scale;
#pragma unroll
      for (int e = 0; e < kMaxPerLane; ++e) {
        gk[e] = fmaf(ds, qr[e], gk[e]);
        gv[e] = fmaf(p, dor[e], gv[e]);
      }
    }
  }
  store_row<BF16>(a.dk + t * a.dk_stride + hk * s.D, s.D, lane, gk);
  store_row<BF16>(a.dv + t * a.dv_stride + hk * s.D, s.D, lane, gv);
}

constexpr int kWarps = 8;
dim3 rows_grid(const SeqDesc& s, int heads) { return dim3((s.tokens + kWarps - 1) / kWarps, heads); }

}  // namespace

cudaError_t launch_seq_weights(const SeqAttnArgs& a, bool bf16, cudaStream_t st) {
  const dim3 grid(256, a.s.kv_heads, a.s.seqs);
  if (bf16)
    seq_weights_simple<true><<<grid, kWarps * 32, 0, st>>>(a);
  else
    seq_weights_simple<false><<<grid, kWarps * 32, 0, st>>>(a);
  return cudaGetLastError();
}

template <bool BF16>
static cudaError_t bwd_t(const SeqAttnArgs& a, cudaStream_t st) {
  prompt_delta_simple<BF16><<<rows_grid(a.s, a.s.q_heads), kWarps * 32, 0, st>>>(a);
  prompt_dq_simple<BF16><<<rows_grid(a.s, a.s.q_heads), kWarps * 32, 0, st>>>(a);
  prompt_dkv_simple<BF16><<<rows_grid(a.s, a.s.kv_heads), kWarps * 32, 0, st>>>(a);
  return cudaGetLastError();
}
cudaError_t launch_prompt_bwd(const SeqAttnArgs& a, bool bf16, cudaStream_t st) {
  return bf16 ? bwd_t<true>(a, st) : bwd_t<false>(a, st);
}

}  // namespace evo
