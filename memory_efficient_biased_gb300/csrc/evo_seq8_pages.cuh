// evo_seq8_pages.cuh — the pages and the scales of an item's key tiles, as the 8-bit cache's kernels look them up.
#pragma once

#include "evo_seq8_internal.h"
#include "evo_seq_sched.cuh"

namespace evo {

// The pages of an item's tiles, looked up a batch of tiles at a time, a page a lane, and a batch ahead, and
// looked over only when their turn comes: looked up tile by tile, the table's latency under load was what a tile took.
struct Pages {
  const SeqDesc& s;
  const int* table;
  int pages, j1, kv_end;   // pages of a tile
  int now, next, in;       // in: tiles of the batch that are done

  __device__ __forceinline__ Pages(const SeqDesc& s, const Work& w, int pages)
      : s(s), table(s.table + static_cast<size_t>(w.b) * s.pages_per_seq), pages(pages), j1(w.j1), kv_end(w.kv_end), in(0) {
    now = look_up(w.j0);
    next = look_up(w.j0 + 32 / pages);
    now = look_over(w.j0, now);
  }
  __device__ __forceinline__ int place(int j) const {  // of this lane's page in the batch that begins at tile j
    const int lane = threadIdx.x & 31;
    j += lane / pages;
    return j < j1 ? j * kTile + lane % pages * s.page : kv_end;
  }
  __device__ __forceinline__ int look_up(int j) const {
    const int at = place(j);
    return at < kv_end ? table[at / s.page] : s.num_pages;
  }
  __device__ __forceinline__ int look_over(int j, int p) const {  // (a page past the keys, or a bad one, reads as zeros)
    if (p >= 0 && p < s.num_pages) return p;
    if (place(j) < kv_end) report_bad_index(s.status);
    return s.num_pages;
  }
  __device__ __forceinline__ int of(int i) const { return __shfl_sync(0xffffffffu, now, in * pages + i); }  // page i of the tile
  __device__ __forceinline__ void step(int j) {  // tile j is done
    if (++in == 32 / pages) {
      in = 0;
      now = look_over(j + 1, next);
      next = look_up(j + 1 + 32 / pages);
    }
  }
};

// Where the scale lies that a lane fetches of a tile: lanes 0-7 those of the keys, 8-15 of the values, 16 tokens each.
struct ScaleLane {
  const float* scales;
  int page, token, part, shift;  // page of the tile and token in it; which 16 tokens of the tile
  __device__ __forceinline__ ScaleLane(const SeqDesc& s, const Cache8& c, int lane) {
    const int pages = s.page < kTile ? kTile / s.page : 1;
    part = lane & 7;
    shift = __ffs(c.block) - 1;
    page = part * pages / 8;
    token = pages == 1 ? part * 16 : part % (8 / pages) * 16;
    scales = lane & 8 ? c.v_scales : c.k_scales;
  }
  // p: the page; first: row of it that the tile begins at
  __device__ __forceinline__ const float* at(const SeqDesc& s, const Cache8& c, int kvh, int p, int first) const {
    return scales + (static_cast<long long>(p) * s.kv_heads + kvh) * c.blocks + ((first + token) >> shift);
  }
};

}  // namespace evo
