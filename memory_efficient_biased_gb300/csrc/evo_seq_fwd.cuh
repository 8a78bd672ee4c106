// evo_seq_fwd.cuh — what the two tcgen05 forwards over causal sequences share (16-bit rows and pages,
// evo_seq_fwd.cu; 8-bit pages, evo_seq8_tiles.cu): where the accumulators lie, how two tiles of queries divide an item's
// key tiles, and moves of the softmax's reference.
#pragma once

#include "evo_seq_internal.h"
#include "evo_seq_sched.cuh"

namespace evo {

constexpr float kMoveLog2 = 8.0f;  // the reference moves only past this margin

// Tensor memory: scores of query tile g (P in place of them), and its O.
__device__ __forceinline__ uint32_t col_s(uint32_t g) { return g * 128u; }
__device__ __forceinline__ uint32_t col_o(uint32_t g) { return 256u + g * 128u; }

// One tile of queries: its key tiles alternate between the warpgroups.
__device__ __forceinline__ bool single(const Work& w, int TQ) { return w.nt <= TQ; }
// The key tiles of this piece that warpgroup g works on: from, from + step, ... below to.
struct Share {
  int from, to, step;
};
__device__ __forceinline__ Share share_of(const Work& w, int g, int TQ) {
  if (single(w, TQ)) return Share{w.j0 + g, w.j1, 2};
  int kt = w.kt;
  if (g == 0) {
    const int end = w.pos + TQ;
    kt = end > 0 ? (end + kTile - 1) / kTile : 1;
  }
  return Share{w.j0, kt < w.j1 ? kt : w.j1, 1};
}

// This thread's row of an accumulator times alpha.  Warp-collective.
template <int DP>
__device__ __forceinline__ void rescale(uint32_t ocol, float alpha) {
#pragma unroll 1
  for (int c = 0; c < DP / 16; ++c) {
    uint32_t x[16];
    tmem_ld16(ocol + c * 16, x);
    tmem_wait_ld(x);
#pragma unroll
    for (int e = 0; e < 16; ++e) x[e] = __float_as_uint(__uint_as_float(x[e]) * alpha);
    tmem_st16(ocol + c * 16, x);
  }
  tmem_wait_st();
}

}  // namespace evo
