// evo_seq_sched.cuh — how the attention of include/evo_seq.h is shared out over the CTAs
// of one launch, all of it on the device (the lengths are device data).
//
// A work item is a block of one sequence's tokens with all the heads of one group, over
// what its tokens see (or, for a block of keys, are seen by); items are laid out one behind
// the other (sequence, kv head, block), and each counts as many units as it has tokens to
// walk over, plus cost() for what every item costs (its own loads, the first scores, the
// output).  CTA c takes the units [c·share, (c+1)·share): every CTA has the same amount of
// work whatever the lengths are, and an item that a border cuts (between two tiles) is
// computed in pieces, whose results are joined in a fixed order by a second kernel.
// Offsets out of order may give one row to many sequences; the work stays that of a call's
// rows all the same: sequences that together have more rows than the call count as empty.
#pragma once

#include "evo_seq_internal.h"

namespace evo {

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
  int q;         // forward, one tile of queries: its buffer
  int stop;      // no more work
};

// Where a piece's partial results belong, for the joining kernel.
struct PieceRecord {
  int used, ends;  // slot in use; holds the item's last key tile
  int b, kvh, row0, t0, nt, pad;
};

// How many pieces the item has that begins in slot 1 of CTA c0: it goes on in slot 0 of the next
// CTAs up to the one that ends it.  Whole warps; the records are read 32 at a time.
__device__ __forceinline__ int count_pieces(const PieceRecord* records, int c0, int ctas) {
  const int lane = threadIdx.x & 31;
  for (int base = c0 + 1; base < ctas; base += 32) {
    int used = 0, ends = 0;
    if (base + lane < ctas) {
      used = records[2 * (base + lane)].used;
      ends = records[2 * (base + lane)].ends;
    }
    const uint32_t gap = __ballot_sync(0xffffffffu, !used), last = __ballot_sync(0xffffffffu, used && ends);
    const int g = gap ? __ffs(gap) - 1 : 32, e = last ? __ffs(last) - 1 : 32;
    if (e < g) return base - c0 + e + 1;
    if (g < 32) return base - c0 + g;
  }
  return ctas - c0;
}

// How a sequence's items are laid out and cut.  An item's units are what it walks over (keys, or
// query tokens) plus cost(), in tiles: an item of the forward takes 3.4 us and a tile 1.85, of dK/dV
// 5.8 and 1.9 (its keys are loaded when the last item is done with them).  With one tile in the
// forward, CTAs that held 25 to 40 short items ended up to a third later than the others; 1, 2 and
// 3 tiles for dK/dV gave 471, 465 and 458 us at 4096 + 1031 + 2500 + 565 tokens (forward included),
// 1.25, 2 and 3 for dQ 479, 465 and 469.
//
// Blocks of W query tokens over the key tiles they see (forward, dQ).
struct QueryBlocks {
  int W;
  __device__ __forceinline__ int cost() const { return 2 * kTile; }
  __device__ __forceinline__ int count(const Seq& q) const { return (q.n + W - 1) / W; }
  // a position below 0 (more new tokens than the length) counts as 0
  __device__ __forceinline__ long long of(const Seq& q, int p) const {
    const long long end = static_cast<long long>(p + 1) * W;
    return (q.pos0 > 0 ? q.pos0 : 0) + (end < q.n ? end : q.n) + cost();
  }
  __device__ __forceinline__ long long before(const Seq& q, int p) const {  // p < count
    return p * static_cast<long long>((q.pos0 > 0 ? q.pos0 : 0) + cost()) + static_cast<long long>(W) * p * (p + 1) / 2;
  }
  __device__ __forceinline__ void place(Work& w, const Seq& q, int p) const {
    w.t0 = p * W;
    w.nt = q.n - w.t0 < W ? q.n - w.t0 : W;
    w.pos = q.pos0 + w.t0;
    w.kv_end = w.pos + w.nt > 0 ? w.pos + w.nt : 0;
    w.kt = w.kv_end > 0 ? (w.kv_end + kTile - 1) / kTile : 1;
  }
  __device__ __forceinline__ int first(const Work&) const { return 0; }
  __device__ __forceinline__ int tile(const Work&, long long keys) const { return static_cast<int>(keys / kTile); }
};

// The same blocks, none of them cut: each counts alike, and a CTA takes whole ones.
struct WholeBlocks : QueryBlocks {
  __device__ __forceinline__ int cost() const { return 0; }
  __device__ __forceinline__ long long of(const Seq&, int) const { return kTile; }
  __device__ __forceinline__ long long before(const Seq&, int p) const { return static_cast<long long>(p) * kTile; }
};

// Tiles of 128 keys under the tiles of TQ query tokens that see them (dK and dV of a prompt).
// Work: t0, nt the keys; j0, j1, kt tiles of queries.
struct KeyBlocks {
  int TQ;
  __device__ __forceinline__ int cost() const { return 3 * TQ; }
  __device__ __forceinline__ int count(const Seq& q) const { return (q.n + kTile - 1) / kTile; }
  __device__ __forceinline__ long long of(const Seq& q, int p) const { return q.n - p * kTile + cost(); }
  __device__ __forceinline__ long long before(const Seq& q, int p) const {
    return p * static_cast<long long>(q.n + cost()) - static_cast<long long>(kTile / 2) * p * (p - 1);
  }
  __device__ __forceinline__ void place(Work& w, const Seq& q, int p) const {
    w.t0 = p * kTile;
    w.nt = q.n - w.t0 < kTile ? q.n - w.t0 : kTile;
    w.pos = w.t0;
    w.kv_end = q.n;
    w.kt = (q.n + TQ - 1) / TQ;
  }
  __device__ __forceinline__ int first(const Work& w) const { return w.t0 / TQ; }
  __device__ __forceinline__ int tile(const Work& w, long long tokens) const {
    return static_cast<int>((w.t0 + tokens) / TQ);
  }
};

// A CTA's share of the units: at least a tile, or whole blocks.
template <class Blocks>
__device__ __forceinline__ long long share_of_cta(const Blocks&, long long units) {
  return units < kTile ? kTile : units;
}
__device__ __forceinline__ long long share_of_cta(const WholeBlocks&, long long units) {
  return (units + kTile - 1) / kTile * kTile;
}

// The walk of one CTA over its share; run by one whole warp (every lane holds the state).
template <class Blocks>
struct Walk {
  const SeqDesc* d;
  Blocks k;
  int b, kvh, p, P;
  Seq q;
  long long off, left;  // units of the current item already passed; units of the share left
  bool crowded;         // more rows than the call has

  __device__ __forceinline__ long long total(const Seq& s) const {
    const int n = k.count(s);
    return n > 0 ? k.before(s, n - 1) + k.of(s, n - 1) : 0;
  }

  __device__ __forceinline__ void init(const SeqDesc& desc, const Blocks& blocks, int cta, int ctas) {
    d = &desc;
    k = blocks;
    const int lane = threadIdx.x & 31;
    // the first 32 sequences stay in the lanes' registers: for most calls that is all of them,
    // and every look at device memory more costs the launch most of a microsecond
    const Seq none{0, 0, 0, 0};
    const Seq early = lane < desc.seqs ? load_seq(desc, lane) : none;
    const long long units = total(early) * desc.kv_heads;
    long long all = units, rows = early.n;
    for (int base = 32; base < desc.seqs; base += 32) {
      const int i = base + lane;
      if (i < desc.seqs) {
        const Seq one = load_seq(desc, i);
        all += total(one) * desc.kv_heads;
        rows += one.n;
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      all += __shfl_xor_sync(0xffffffffu, all, o);
      rows += __shfl_xor_sync(0xffffffffu, rows, o);
    }
    crowded = rows > desc.tokens;
    if (crowded) {
      report_bad_index(desc.status);
      all = 0;
    }
    const long long share = share_of_cta(k, (all + ctas - 1) / ctas);
    const long long x0 = share * cta;
    left = all - x0 < share ? all - x0 : share;
    b = desc.seqs;
    if (left <= 0) {
      left = 0;
      return;
    }
    long long passed = 0;  // units of the sequences before `base`
    for (int base = 0; base < desc.seqs; base += 32) {
      const int i = base + lane;
      const Seq mine_q = base == 0 ? early : (i < desc.seqs ? load_seq(desc, i) : none);
      const long long mine = base == 0 ? units : total(mine_q) * desc.kv_heads;
      long long run = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, run, o);
        if (lane >= o) run += y;
      }
      const uint32_t any = __ballot_sync(0xffffffffu, x0 < passed + run);
      if (any) {
        const int first = __ffs(any) - 1;
        const long long begin = __shfl_sync(0xffffffffu, passed + run - mine, first);
        b = base + first;
        q.row0 = __shfl_sync(0xffffffffu, mine_q.row0, first);
        q.n = __shfl_sync(0xffffffffu, mine_q.n, first);
        q.kv = __shfl_sync(0xffffffffu, mine_q.kv, first);
        q.pos0 = __shfl_sync(0xffffffffu, mine_q.pos0, first);
        P = k.count(q);
        const long long per = total(q);
        long long x = x0 - begin;
        kvh = static_cast<int>(x / per);
        x -= kvh * per;
        int lo = 0, hi = P - 1;  // the block that holds unit x
        while (lo < hi) {
          const int mid = (lo + hi + 1) >> 1;
          if (k.before(q, mid) <= x)
            lo = mid;
          else
            hi = mid - 1;
        }
        p = lo;
        off = x - k.before(q, p);
        return;
      }
      passed += __shfl_sync(0xffffffffu, run, 31);
    }
    left = 0;
  }

  // The next sequence with an item, looked for 32 at a time.
  __device__ __forceinline__ void next_sequence() {
    const int lane = threadIdx.x & 31;
    for (int base = b + 1; base < d->seqs; base += 32) {
      Seq mine{0, 0, 0, 0};
      if (base + lane < d->seqs) mine = load_seq(*d, base + lane);
      const uint32_t any = __ballot_sync(0xffffffffu, k.count(mine) > 0);
      if (any) {
        const int first = __ffs(any) - 1;
        b = base + first;
        q.row0 = __shfl_sync(0xffffffffu, mine.row0, first);
        q.n = __shfl_sync(0xffffffffu, mine.n, first);
        q.kv = __shfl_sync(0xffffffffu, mine.kv, first);
        q.pos0 = __shfl_sync(0xffffffffu, mine.pos0, first);
        P = k.count(q);
        return;
      }
    }
    b = d->seqs;
    left = 0;
  }

  // The next piece with at least one tile, or stop.
  __device__ __forceinline__ Work next() {
    Work w{};
    while (left > 0) {
      const long long units = k.of(q, p), to = off + left < units ? off + left : units;
      w.b = b, w.kvh = kvh, w.row0 = q.row0;
      k.place(w, q, p);
      const int begin = k.first(w);
      auto tile = [&](long long x) {
        const int t = x > k.cost() ? k.tile(w, x - k.cost()) : begin;
        return t < w.kt ? t : w.kt;
      };
      w.j0 = tile(off);
      w.j1 = to == units ? w.kt : tile(to);
      w.slot = w.j0 > begin ? 0 : (w.j1 < w.kt ? 1 : -1);
      left -= to - off;
      off = 0;
      if (to == units && ++p == P) {
        p = 0;
        if (++kvh == d->kv_heads) {
          kvh = 0;
          next_sequence();
        }
      }
      if (w.j0 < w.j1) return w;
    }
    w.stop = 1;
    return w;
  }
};

}  // namespace evo
