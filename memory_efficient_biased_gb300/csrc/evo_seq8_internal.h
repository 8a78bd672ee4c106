// evo_seq8_internal.h — what the kernels of the 8-bit cache (include/evo_seq.h) share: its
// layout, its scales, and conversions of e4m3 codes.
#pragma once

#include "evo_seq_internal.h"

namespace evo {

struct Cache8 {
  uint8_t *k_pages, *v_pages;
  float *k_scales, *v_scales;
  long long k_page, v_page;  // elements, which are bytes, between pages
  int block, blocks;         // tokens a scale, scales a page and head
};

struct Cache8Args {  // append, read and copy
  SeqDesc s;
  Cache8 c;
  uint16_t *k, *v;    // rows: read by an append, written by a read; a copy's pages
  long long k_stride, v_stride;
  int tokens_a_warp;  // read
  int wide;           // read: rows start at multiples of 32 bytes
};

constexpr int kFewRows = 16;  // rows of a tile of the kernel for few rows a key

struct Seq8FwdArgs {
  SeqFwdArgs f;  // tk, tv: pages of bytes as (D, kv_heads, page, num_pages); TQ = 128 / group, W: tokens of an item
  Cache8 c;
  const uint16_t* q;   // few rows
  long long q_stride;
  int whole;           // few rows: no item is cut, and nothing is joined
};

// Place of the scale of token j (of page p) and head h.
__device__ __forceinline__ long long scale_at(const Cache8& c, const SeqDesc& s, int p, int h, int j) {
  return (static_cast<long long>(p) * s.kv_heads + h) * c.blocks + (j % s.page) / c.block;
}

// log2 of a scale of values, -64 at the least (a block of zeros may have a scale of 0); NaN stays NaN.
__device__ __forceinline__ float log2_value_scale(float s) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(lg2(s)), "f"(-64.0f));
  return r;
}

// ln2 (m + log2 l): l is a sum of weights over the scales of values, so both may be large and cancel.  The whole part of log2 l
// is added to m by itself, which loses nothing then (lg2 alone would be 2^-22 of it off).
__device__ __forceinline__ float whole_log2(float l) {  // 0 for what is no normal number below 2^126
  const uint32_t u = __float_as_uint(l);
  return u - 0x00800000u < 0x7e000000u ? static_cast<float>(static_cast<int>(u >> 23) - 127) : 0.0f;
}
__device__ __forceinline__ float power_of_two(float d) {  // d whole, -126 to 127
  return __uint_as_float(static_cast<uint32_t>(127 + static_cast<int>(d)) << 23);
}
__device__ __forceinline__ float lse_of(float m, float l) {
  if (l == 0.0f) return -INFINITY;
  const float e = whole_log2(l);
  return ((m + e) + lg2(l * power_of_two(-e))) * kSeqLn2;
}

// Four codes as two pairs of f16 (bytes 0 and 1, bytes 2 and 3), exactly; NaN stays NaN.
__device__ __forceinline__ uint2 f16x4_of_codes(uint32_t codes) {
  uint2 r;
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
      : "=r"(r.x), "=r"(r.y)
      : "r"(codes));
  return r;
}
// A pair of codes in f16 as a pair of bf16, exactly (a bf16 is the upper half of an f32); NaN stays NaN.
__device__ __forceinline__ uint32_t bf16x2_of_codes(uint32_t f16) {
  const float2 f = unpack2<false>(f16);
  return __byte_perm(__float_as_uint(f.x), __float_as_uint(f.y), 0x7632);
}
__device__ __forceinline__ uint32_t mul_f16x2(uint32_t x, uint32_t y) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(y));
  return r;
}
// x (lower byte) and y rounded to e4m3, nearest even; NaN stays NaN, what is beyond 448 becomes 448.
__device__ __forceinline__ uint32_t e4m3x2_of_f32(float x, float y) {
  uint32_t r;
  asm("{\n\t.reg .b16 c;\n\tcvt.rn.satfinite.e4m3x2.f32 c, %2, %1;\n\tcvt.u32.u16 %0, c;\n\t}" : "=r"(r) : "f"(x), "f"(y));
  return r;
}
// Eight codes as numbers.
__device__ __forceinline__ void f32_of_codes(uint2 codes, float (&x)[8]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint2 w = f16x4_of_codes(i ? codes.y : codes.x);
    const float2 f = unpack2<false>(w.x), h = unpack2<false>(w.y);
    x[4 * i] = f.x, x[4 * i + 1] = f.y, x[4 * i + 2] = h.x, x[4 * i + 3] = h.y;
  }
}
__device__ __forceinline__ uint2 codes_of_f32(const float (&x)[8]) {
  return make_uint2(e4m3x2_of_f32(x[0], x[1]) | e4m3x2_of_f32(x[2], x[3]) << 16,
                    e4m3x2_of_f32(x[4], x[5]) | e4m3x2_of_f32(x[6], x[7]) << 16);
}

cudaError_t launch_cache8_append(const Cache8Args& a, bool bf16, cudaStream_t st);
cudaError_t launch_cache8_read(const Cache8Args& a, int sms, bool bf16, cudaStream_t st);
cudaError_t launch_cache8_copy(const Cache8Args& a, int* table, int sms, bool bf16, cudaStream_t st);
cudaError_t launch_paged8_few(const Seq8FwdArgs& a, int ctas, bool bf16, cudaStream_t st);
cudaError_t launch_paged8_tiles(const Seq8FwdArgs& a, int ctas, bool bf16, cudaStream_t st);

}  // namespace evo
