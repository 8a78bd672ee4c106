// evo_seq_sched.cuh — how the attention of include/evo_seq.h is shared out over the CTAs
// of one launch, all of it on the device (the lengths are device data).
//
// A work item is a block of W query tokens of one sequence with all the heads of one
// group, over the keys it sees; items are laid out one behind the other (sequence, kv head,
// block), and each counts as many units as it has keys, plus kItemCost for what every item
// costs.  CTA c takes the units [c·share, (c+1)·share): every CTA has the same amount of
// work whatever the lengths are, and an item that a border cuts (at a multiple of 128 keys)
// is computed in pieces, whose results are joined in a fixed order by a second kernel.
#pragma once

#include "evo_seq_internal.h"

namespace evo {

// An item's fixed cost (its query load, first scores and output) in keys.
constexpr int kItemCost = 128;

// One item or a piece of one, as the roles of a CTA see it.
struct Work {
  int b, kvh;
  int row0;      // the sequence's first row
  int t0, nt;    // first token of the block, and how many it has
  int pos;       // position of the block's first token
  int kv_end;    // keys seen by any of its tokens (>= 0)
  int j0, j1;    // key tiles of this piece
  int kt;        // key tiles of the item (at least one, so that empty rows are written)
  int slot;      // -1: the whole item; 0 / 1: a piece, kept in this CTA's slot 0 / 1
  int stop;      // no more work
};

// Where a piece's partial results belong, for the joining kernel.
struct PieceRecord {
  int used, ends;  // slot in use; holds the item's last key tile
  int b, kvh, row0, t0, nt, pad;
};

// Units of block p (of P blocks of W tokens) of a sequence, and of all blocks before p.
struct BlockUnits {
  long long pos0c;  // position of its first new token, at least 0
  int n, W, P;
  __device__ __forceinline__ BlockUnits(const Seq& q, int w)
      : pos0c(q.pos0 > 0 ? q.pos0 : 0), n(q.n), W(w), P((q.n + w - 1) / w) {}
  __device__ __forceinline__ long long of(int p) const {
    const long long end = static_cast<long long>(p + 1) * W;
    return pos0c + (end < n ? end : n) + kItemCost;
  }
  __device__ __forceinline__ long long before(int p) const {  // p < P
    return p * (pos0c + kItemCost) + static_cast<long long>(W) * p * (p + 1) / 2;
  }
  __device__ __forceinline__ long long total() const { return P > 0 ? before(P - 1) + of(P - 1) : 0; }
  // the block that holds unit x < total()
  __device__ __forceinline__ int find(long long x) const {
    const float c = static_cast<float>(pos0c + kItemCost) + 0.5f * W;
    int p = static_cast<int>((sqrtf(c * c + 2.0f * W * static_cast<float>(x)) - c) / W);
    p = p < 0 ? 0 : (p > P - 1 ? P - 1 : p);
    while (p > 0 && before(p) > x) --p;
    while (p + 1 < P && before(p + 1) <= x) ++p;
    return p;
  }
};

// The walk of one CTA over its share; run by one whole warp (every lane holds the state).
struct Walk {
  const SeqDesc* d;
  int W, b, kvh, p;
  Seq q;
  long long off, left;  // units of the current item already passed; units of the share left
  int end_b;

  __device__ __forceinline__ void init(const SeqDesc& desc, int w, int cta, int ctas) {
    d = &desc;
    W = w;
    const int lane = threadIdx.x & 31;
    long long total = 0;
    for (int base = 0; base < desc.seqs; base += 32) {
      const int i = base + lane;
      if (i < desc.seqs) total += BlockUnits(load_seq(desc, i), w).total() * desc.kv_heads;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
    long long share = (total + ctas - 1) / ctas;
    if (share < kItemCost + 128) share = kItemCost + 128;
    const long long x0 = share * cta;
    left = total - x0 < share ? total - x0 : share;
    b = desc.seqs;
    if (left <= 0) {
      left = 0;
      return;
    }
    long long passed = 0;  // units of the sequences before `base`
    for (int base = 0; base < desc.seqs; base += 32) {
      const int i = base + lane;
      const long long mine = i < desc.seqs ? BlockUnits(load_seq(desc, i), w).total() * desc.kv_heads : 0;
      long long run = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, run, o);
        if (lane >= o) run += y;
      }
      const bool here = x0 < passed + run;
      const uint32_t any = __ballot_sync(0xffffffffu, here);
      if (any) {
        const int first = __ffs(any) - 1;
        const long long begin = __shfl_sync(0xffffffffu, passed + run - mine, first);
        b = base + first;
        q = load_seq(desc, b);
        const BlockUnits u(q, w);
        long long x = x0 - begin;
        kvh = static_cast<int>(x / u.total());
        x -= kvh * u.total();
        p = u.find(x);
        off = x - u.before(p);
        return;
      }
      passed += __shfl_sync(0xffffffffu, run, 31);
    }
  }

  // The next piece with at least one key tile, or stop.
  __device__ __forceinline__ Work next() {
    Work w{};
    while (left > 0) {
      const BlockUnits u(q, W);
      const long long units = u.of(p), to = off + left < units ? off + left : units;
      w.b = b, w.kvh = kvh, w.row0 = q.row0;
      w.t0 = p * W;
      w.nt = q.n - w.t0 < W ? q.n - w.t0 : W;
      w.pos = q.pos0 + w.t0;
      w.kv_end = w.pos + w.nt > 0 ? w.pos + w.nt : 0;
      w.kt = w.kv_end > 0 ? (w.kv_end + kTile - 1) / kTile : 1;
      auto tile = [&](long long x) {
        const long long t = x > kItemCost ? (x - kItemCost) / kTile : 0;
        return t < w.kt ? static_cast<int>(t) : w.kt;
      };
      w.j0 = tile(off);
      w.j1 = to == units ? w.kt : tile(to);
      w.slot = w.j0 > 0 ? 0 : (w.j1 < w.kt ? 1 : -1);
      left -= to - off;
      off = 0;
      if (to == units && ++p == u.P) {
        p = 0;
        if (++kvh == d->kv_heads) {
          kvh = 0;
          do {
            ++b;
            if (b >= d->seqs) {
              left = 0;
              break;
            }
            q = load_seq(*d, b);
          } while (q.n == 0);
        }
      }
      if (w.j0 < w.j1) return w;
    }
    w.stop = 1;
    return w;
  }
};

}  // namespace evo
