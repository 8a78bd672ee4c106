// evo_seq8_cache.cu — rows into and out of the 8-bit cache of include/evo_seq.h.
#include "evo_seq8_internal.h"

namespace evo {
namespace {

// ------------------------------------------------------------------ append
// One CTA per block of tokens that a sequence's new tokens reach and eight, or fewer, of its
// (keys or values, head) units: a warp per 16 tokens of a unit, the loads of its rows all under way
// together, the largest magnitude joined over the unit's warps.
//
// How many blocks the sequences reach is known on the device only.  n tokens reach at most
// floor(n / B) + 2 blocks of B, so sequence b is given the numbers from floor(cu[b] / B) + 2 b
// on, which the CTAs search; the numbers that are left over have no block.  (The search, not the
// bytes, is what a step of single tokens waits for.)
//
// Bound by the bytes: two read and one written an element, and nothing else where the scale does not grow.
constexpr int kAppendThreads = 256;

__device__ __forceinline__ long long block_number(const SeqDesc& s, int block, int b) {
  return static_cast<long long>(s.cu[b] / block) + 2 * static_cast<long long>(b);
}

// The last sequence whose numbers begin at or before i, looked for by a whole warp; -1: none.
__device__ __forceinline__ int find_block(const SeqDesc& s, int block, long long i) {
  const int lane = threadIdx.x & 31;
  int lo = 0, n = s.seqs;  // it is in [lo, lo + n), if any
  while (n > 0) {
    const int step = (n + 31) / 32, at = lo + lane * step;
    const bool below = lane * step < n && block_number(s, block, at) <= i;
    const uint32_t m = __ballot_sync(0xffffffffu, below);
    // (offsets out of order: any answer, looked over below)
    const int last = 31 - __clz(m);
    if (last < 0) return -1;
    if (step == 1) return lo + last;
    n = n - last * step < step ? n - last * step : step;
    lo += last * step;
  }
  return -1;
}

// The least power of two s >= 2^-64 with most <= 448 s (448 = 1.75 · 2^8).
__device__ __forceinline__ float scale_for(float most) {
  const uint32_t u = __float_as_uint(most);
  int e = static_cast<int>(u >> 23) - 8 + ((u & 0x7fffffu) > 0x600000u);
  if (e < 127 - 64) e = 127 - 64;
  return __uint_as_float(static_cast<uint32_t>(e) << 23);
}

template <bool BF16>
__global__ void __launch_bounds__(kAppendThreads) evo_append8_kernel(const __grid_constant__ Cache8Args a) {
  __shared__ float warp_most[8];
  const SeqDesc& s = a.s;
  const Cache8& c = a.c;
  if (blockIdx.x == 0 && blockIdx.y == 0) check_seqs(s);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int b = find_block(s, c.block, blockIdx.x);
  if (b < 0) return;
  const Seq q = load_seq(s, b);
  if (q.n == 0) return;
  const int p0 = q.pos0 > 0 ? q.pos0 : 0;  // first position that is written
  const long long index = p0 / c.block + (static_cast<long long>(blockIdx.x) - block_number(s, c.block, b));
  if (index * c.block >= q.kv) return;
  const int start = static_cast<int>(index) * c.block;
  const int lo = start > p0 ? start : p0, hi = q.kv - start < c.block ? q.kv : start + c.block;
  if (lo >= hi) return;
  const int p = page_of(s, b, start);
  if (p < 0) return;
  // (up to here every thread of the block went the same way)
  const int team = c.block / 16, unit = blockIdx.y * (8 / team) + warp / team;
  const bool work = unit < 2 * s.kv_heads;
  const int kv = unit >= s.kv_heads, h = kv ? unit - s.kv_heads : unit;
  const int per = s.D / 8, first = start + (warp % team) * 16;  // 16-byte pieces a row; first token of this warp's 16
  const uint16_t* rows = (kv ? a.v : a.k) + static_cast<long long>(h) * s.D;
  const long long stride = kv ? a.v_stride : a.k_stride;
  uint8_t* page = (kv ? c.v_pages + p * c.v_page : c.k_pages + p * c.k_page) + h * s.D;
  float* scale = (kv ? c.v_scales : c.k_scales) + scale_at(c, s, p, work ? h : 0, start);
  const bool older = start < lo;
  const float before = work && older ? *scale : 0.0f;
  uint4 x[8];
  float most = 0.0f;
#pragma unroll
  for (int r = 0; r < 8; ++r) {
    const int i = lane + 32 * r, j = first + i / per;
    x[r] = make_uint4(0u, 0u, 0u, 0u);
    if (work && i < 16 * per && j >= lo && j < hi)
      x[r] = *reinterpret_cast<const uint4*>(rows + (q.row0 + static_cast<long long>(j - q.pos0)) * stride + i % per * 8);
  }
#pragma unroll
  for (int r = 0; r < 8; ++r) {
    const uint32_t w[4] = {x[r].x, x[r].y, x[r].z, x[r].w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float2 f = unpack2<BF16>(w[e]);
      most = fmaxf(most, fabsf(f.x) < INFINITY ? fabsf(f.x) : 0.0f);
      most = fmaxf(most, fabsf(f.y) < INFINITY ? fabsf(f.y) : 0.0f);
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
  if (team > 1) {
    if (lane == 0) warp_most[warp] = most;
    __syncthreads();
    for (int i = 0; i < team; ++i) most = fmaxf(most, warp_most[warp / team * team + i]);
  }
  if (!work) return;
  float now = scale_for(most);
  if (before > now && before < INFINITY) now = before;  // (a block without tokens from before has 0 there)
  const int row = s.kv_heads * s.D;
  if (older && now != before) {
    const float shrink = before > 0.0f && before < INFINITY ? before / now : 1.0f;
    for (int i = lane; i < 16 * per; i += 32) {
      const int j = first + i / per;
      if (j >= lo) break;
      uint2* at = reinterpret_cast<uint2*>(page + static_cast<long long>(j % s.page) * row + i % per * 8);
      float y[8];
      f32_of_codes(*at, y);
#pragma unroll
      for (int e = 0; e < 8; ++e) y[e] *= shrink;
      *at = codes_of_f32(y);
    }
  }
  const float inv = 1.0f / now;  // (exact for a power of two)
#pragma unroll
  for (int r = 0; r < 8; ++r) {
    const int i = lane + 32 * r, j = first + i / per;
    if (i >= 16 * per || j < lo || j >= hi) continue;
    const uint32_t w[4] = {x[r].x, x[r].y, x[r].z, x[r].w};
    float y[8];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float2 f = unpack2<BF16>(w[e]);
      y[2 * e] = fabsf(f.x) < INFINITY ? f.x * inv : NAN;
      y[2 * e + 1] = fabsf(f.y) < INFINITY ? f.y * inv : NAN;
    }
    *reinterpret_cast<uint2*>(page + static_cast<long long>(j % s.page) * row + i % per * 8) = codes_of_f32(y);
  }
  if (lane == 0 && warp % team == 0 && now != before) *scale = now;
}

// ------------------------------------------------------------------ read
// One thread per 16 codes of a row of keys (blockIdx.y = 0) or values.  Bound by the bytes: one read
// and two written an element.
template <bool BF16>
__global__ void __launch_bounds__(256) evo_read8_kernel(const __grid_constant__ Cache8Args a) {
  const SeqDesc& s = a.s;
  const Cache8& c = a.c;
  if (blockIdx.x == 0 && blockIdx.y == 0) check_seqs(s);
  const int per = s.D / 16, chunks = s.kv_heads * per;
  const long long i = static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x;
  if (i >= static_cast<long long>(s.tokens) * chunks) return;
  const int t = static_cast<int>(i / chunks), n = static_cast<int>(i % chunks), kv = blockIdx.y;
  const int b = find_seq(s, t);
  if (b < 0) return;
  const Seq q = load_seq(s, b);
  if (t < q.row0 || t >= q.row0 + q.n) return;
  const int j = q.pos0 + (t - q.row0);
  const int p = j < 0 ? -1 : page_of(s, b, j);
  uint32_t o[8] = {};
  if (p >= 0) {
    const uint8_t* page = kv ? c.v_pages + p * c.v_page : c.k_pages + p * c.k_page;
    const uint4 x = *reinterpret_cast<const uint4*>(page + (static_cast<long long>(j % s.page) * chunks + n) * 16);
    const float scale = (kv ? c.v_scales : c.k_scales)[scale_at(c, s, p, n / per, j)];
    constexpr float most = BF16 ? 3.38953139e38f : 65504.0f;
    const uint2 w[4] = {f16x4_of_codes(x.x), f16x4_of_codes(x.y), f16x4_of_codes(x.z), f16x4_of_codes(x.w)};
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      float2 f = unpack2<false>((e & 1) ? w[e >> 1].y : w[e >> 1].x);
      f = make_float2(f.x * scale, f.y * scale);
      // (comparisons that a NaN passes unchanged)
      f.x = f.x > most ? most : (f.x < -most ? -most : f.x);
      f.y = f.y > most ? most : (f.y < -most ? -most : f.y);
      o[e] = pack2<BF16>(f.x, f.y);
    }
  }
  uint16_t* to = (kv ? a.v : a.k) + t * (kv ? a.v_stride : a.k_stride) + static_cast<long long>(n) * 16;
  *reinterpret_cast<uint4*>(to) = make_uint4(o[0], o[1], o[2], o[3]);
  *reinterpret_cast<uint4*>(to + 8) = make_uint4(o[4], o[5], o[6], o[7]);
}

}  // namespace

cudaError_t launch_cache8_append(const Cache8Args& a, bool bf16, cudaStream_t st) {
  const long long blocks = static_cast<long long>(a.s.tokens) / a.c.block + 2ll * a.s.seqs;
  const int units = 8 / (a.c.block / 16);  // a CTA
  const dim3 grid(static_cast<unsigned>(blocks), static_cast<unsigned>((2 * a.s.kv_heads + units - 1) / units));
  if (bf16)
    evo_append8_kernel<true><<<grid, kAppendThreads, 0, st>>>(a);
  else
    evo_append8_kernel<false><<<grid, kAppendThreads, 0, st>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_cache8_read(const Cache8Args& a, bool bf16, cudaStream_t st) {
  const long long n = static_cast<long long>(a.s.tokens) * (a.s.kv_heads * a.s.D / 16);
  const dim3 grid(static_cast<unsigned>((n + 255) / 256), 2);
  if (bf16)
    evo_read8_kernel<true><<<grid, 256, 0, st>>>(a);
  else
    evo_read8_kernel<false><<<grid, 256, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace evo
