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

struct Cache8Args {  // append and read
  SeqDesc s;
  Cache8 c;
  uint16_t *k, *v;   // rows: read by an append, written by a read
  long long k_stride, v_stride;
};

struct Seq8FwdArgs {
  SeqFwdArgs f;  // tk, tv: pages of bytes as (D, kv_heads, page, num_pages); W, TQ: the kernel's own, TQ as the join
                 // takes it (128 / group)
  Cache8 c;
  const uint16_t* q;
  long long q_stride;
};

// Place of the scale of token j (of page p) and head h.
__device__ __forceinline__ long long scale_at(const Cache8& c, const SeqDesc& s, int p, int h, int j) {
  return (static_cast<long long>(p) * s.kv_heads + h) * c.blocks + (j % s.page) / c.block;
}

// Two codes (the lower byte first) as a pair of f16, exactly; NaN stays NaN.
__device__ __forceinline__ uint32_t f16x2_of_e4m3x2(uint32_t codes) {
  uint32_t r;
  asm("{\n\t.reg .b16 c;\n\tcvt.u16.u32 c, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, c;\n\t}" : "=r"(r) : "r"(codes));
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
  for (int i = 0; i < 4; ++i) {
    const uint32_t w = i < 2 ? codes.x : codes.y;
    const float2 f = unpack2<false>(f16x2_of_e4m3x2((i & 1) ? w >> 16 : w));
    x[2 * i] = f.x;
    x[2 * i + 1] = f.y;
  }
}
__device__ __forceinline__ uint2 codes_of_f32(const float (&x)[8]) {
  return make_uint2(e4m3x2_of_f32(x[0], x[1]) | e4m3x2_of_f32(x[2], x[3]) << 16,
                    e4m3x2_of_f32(x[4], x[5]) | e4m3x2_of_f32(x[6], x[7]) << 16);
}

cudaError_t launch_cache8_append(const Cache8Args& a, bool bf16, cudaStream_t st);
cudaError_t launch_cache8_read(const Cache8Args& a, bool bf16, cudaStream_t st);
cudaError_t launch_paged8_few(const Seq8FwdArgs& a, int ctas, bool bf16, cudaStream_t st);
cudaError_t launch_paged8_rows(const Seq8FwdArgs& a, bool bf16, cudaStream_t st);

}  // namespace evo
