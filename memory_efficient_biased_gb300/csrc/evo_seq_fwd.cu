// evo_seq_fwd.cu — attention over causal sequences (include/evo_seq.h) on the tensor
// cores: packed prompts, and chunks of new tokens over a paged cache.
//
// Mathematics, per row (token, head): S = q·kᵀ, m the running reference of s·log2e·S,
// P = 2^(s·log2e·S - m), l = Σ P and O = Σ P v over the key tiles seen so far; at the end
// O / l and lse = ln2·(m + log2 l).  m follows a tile's maximum only when that passes it by
// more than 2^8 (P stays below 256), so O in tensor memory is rescaled rarely.
//
// Rows.  A query tile holds floor(128 / G) tokens with all G heads of their group, token by
// token: the heads of a group share the K and V tiles, single tokens fill as much of a
// tile as they can, and a causal border is as tight as with one head.  An item is two such
// tiles (tile g worked on by warpgroup g) over the key tiles of 128 that they see; items are
// shared out by evo_seq_sched.cuh.
//
// Roles (12 warps, one CTA per SM, persistent over its share of the work):
//   warps 0-3, 4-7  softmax of tile 0 and 1, one thread per row
//   warp 8          producer: Q tiles, and K and V tiles into one ring, by TMA; a cache's pages
//                   are rows of a 4-D map, one box per page (its lanes look up the table)
//   warps 9, 10     the MMAs of tile 0 and 1: S_g = Q_g Kᵀ, then O_g += P_g V in two halves of 64 keys
//                   as P comes; the two tiles alternate on the tensor core, each tile's MMAs run
//                   under the other's softmax
//   warp 11         the walk over the work (descriptors in a ring), and every V tile's release:
//                   rows that no query of the item sees are cleared in the item's last tile
//                   (whatever lies behind a sequence, NaN included, must not reach 0·V)
// Tensor memory (512 columns): S_0, S_1 (128 each, P in place of S as packed pairs), O_0, O_1.
//
// A value of V that is not finite and that only some rows of the item see (a later token of
// the same tile) is taken out of the tile and added back to the rows that see it at the end.
//
// Rounded to the input type: P as an MMA operand (what the tensor core takes) and O.
//
// What bounds it.  Single tokens: HBM, 6.7 TB/s at 1.0 GB of cache (four sequences up to 131071
// tokens, 8 kv heads of 128: 150 us).  Prompts: 16384 tokens, 16 heads of 128 take 0.84 ms, 1290
// TFLOP/s of the scores that are seen (66 % of cuBLAS).  There a pair of tiles takes 3500 cycles a key
// tile, the chain S (800), max (500), exponentials (850), P·V and back (1150); its MMAs alone take 2560
// (80 each instead of 64: both operands from shared memory ask for all of its 128 bytes a cycle).
#include "evo_seq_internal.h"
#include "evo_seq_sched.cuh"

namespace evo {
namespace {

constexpr int kThreads = 384;
constexpr int kProducerWarp = 8, kMmaWarp = 9, kWalkWarp = 11;
constexpr uint32_t kRegsLaunch = 168, kRegsSoftmax = 200, kRegsOther = 104;
static_assert(128 * kRegsOther + 256 * kRegsSoftmax <= kThreads * kRegsLaunch, "register split exceeds the launch");
constexpr float kMoveLog2 = 8.0f;  // the reference moves only past this margin
constexpr int kDescs = 4, kReady = 8, kMaxSlots = 10;
static_assert(kReady >= kMaxSlots / 2 + 1, "a V tile's release must not lap the MMA threads");

struct Bars {
  uint64_t desc_full[kDescs], desc_empty[kDescs];
  uint64_t q_full[2], q_empty[2];
  uint64_t full[kMaxSlots], empty[kMaxSlots];
  uint64_t v_ready[kReady];
  // turn: see the softmax; merge_full: the second warpgroup's share of a single tile is done
  uint64_t s_full[2], p_half[2], p_full[2], pv_done[2], o_free[2], drain[2], turn[2], merge_full;
  Work work[kDescs];
  float2 merge[kTile];  // (m, l) of the second warpgroup's share of a single tile
  int dirty[kDescs];  // a V tile of the item held values that were taken out
  uint32_t tiles, queries[2];  // K and V tiles and Q tiles that the producer asked for
  uint32_t tmem_slot;
  int abort;
};

template <int DP>
struct Layout {
  static constexpr uint32_t kHalf = kTile * 128u;            // 64 features of 128 rows
  static constexpr uint32_t kTB = kTile * DP * 2u;           // one tile
  static constexpr int kSlots = DP == 128 ? 5 : 10;          // K and V tiles in flight: 160 KB
  static constexpr uint32_t q = 0, ring = 2 * kTB, bars = ring + kSlots * kTB;
  static constexpr uint32_t total = bars + ((sizeof(Bars) + 127) & ~127u);
};
static_assert(Layout<128>::total + 1024 <= 232448, "shared memory");

__device__ __forceinline__ uint32_t col_s(uint32_t g) { return g * 128u; }
__device__ __forceinline__ uint32_t col_o(uint32_t g) { return 256u + g * 128u; }

// The next descriptor, read by every lane of a warp (or by one thread alone).
template <bool WARP>
__device__ __forceinline__ bool take(Bars* bars, uint32_t it, const WaitGuard& g, Work& w) {
  const uint32_t s = it % kDescs;
  const bool ok = WARP ? mbar_wait_warp_inl(smem_u32(&bars->desc_full[s]), (it / kDescs) & 1, g)
                       : mbar_wait_inl(smem_u32(&bars->desc_full[s]), (it / kDescs) & 1, g);
  if (!ok) return false;
  w = bars->work[s];
  return !w.stop;
}
__device__ __forceinline__ void give_back(Bars* bars, uint32_t it) {
  mbar_arrive(smem_u32(&bars->desc_empty[it % kDescs]));
}
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

// ------------------------------------------------------------ producer (one warp)
template <int DP>
__device__ __forceinline__ void producer(const SeqFwdArgs& a, uint8_t* base, Bars* bars, const WaitGuard& g, int lane) {
  using L = Layout<DP>;
  const SeqDesc& s = a.s;
  const bool paged = s.table != nullptr;
  const int box = paged ? (s.page < kTile ? s.page : kTile) : kTile;  // rows per copy
  const int boxes = kTile / box;
  const uint32_t qbytes = static_cast<uint32_t>(a.TQ * s.group) * 128u * (DP / 64);
  uint32_t use = 0, it = 0, queries[2] = {0, 0};
  Work w;
  // Two tiles of queries take a buffer each; a single one takes the buffers by turns (w.q), so that the
  // next one's load does not wait for this one's last scores.
  auto load_queries = [&]() -> bool {
    const bool one = single(w, a.TQ);
    for (int t = 0; t < (one ? 1 : 2); ++t) {
      const int b = one ? w.q : t;
      if (!mbar_wait_warp_inl(smem_u32(&bars->q_empty[b]), (queries[b] & 1) ^ 1, g)) return false;
      if (lane == 0) {
        const uint32_t full = smem_u32(&bars->q_full[b]);
        mbar_arrive_expect_tx(full, qbytes);
        for (int h = 0; h < DP / 64; ++h)
          tma_load_4d(smem_u32(base + L::q + b * L::kTB + h * L::kHalf), &a.tq, full, h * 64, 0, w.kvh,
                      w.row0 + w.t0 + t * a.TQ);
      }
      ++queries[b];
    }
    return true;
  };
  for (; take<true>(bars, it, g, w); ++it) {
    __syncwarp();
    if (lane == 0) give_back(bars, it);
    // this lane's page of a tile (a page past the keys, or a bad one, reads as zeros)
    auto page = [&](int j) -> int {
      const int key = j * kTile + lane * box;
      if (lane >= boxes || key >= w.kv_end) return s.num_pages;
      const int p = page_of(s, w.b, key);
      return p < 0 ? s.num_pages : p;
    };
    int mine = paged ? page(w.j0) : 0;
    bool ok = load_queries();
    for (int j = w.j0; ok && j < w.j1; ++j) {
      const int cur = mine;
      if (paged && j + 1 < w.j1) mine = page(j + 1);
#pragma unroll
      for (int kv = 0; kv < 2; ++kv, ++use) {
        const uint32_t slot = use % L::kSlots;
        if (!mbar_wait_warp_inl(smem_u32(&bars->empty[slot]), ((use / L::kSlots) & 1) ^ 1, g)) { ok = false; break; }
        const uint32_t full = smem_u32(&bars->full[slot]), dst = smem_u32(base + L::ring + slot * L::kTB);
        if (lane == 0) mbar_arrive_expect_tx(full, L::kTB);
        __syncwarp();
        const CUtensorMap* m = kv ? &a.tv : &a.tk;
        if (paged) {
          if (lane < boxes)
            for (int h = 0; h < DP / 64; ++h)
              tma_load_4d(dst + h * L::kHalf + lane * box * 128, m, full, h * 64, w.kvh, (j * kTile) % s.page * (boxes == 1),
                          cur);
        } else if (lane < DP / 64) {
          tma_load_3d(dst + lane * L::kHalf, m, full, lane * 64, w.kvh, w.row0 + j * kTile);
        }
      }
    }
    if (!ok) break;
  }
  if (lane == 0) bars->tiles = use, bars->queries[0] = queries[0], bars->queries[1] = queries[1];
}

// ------------------------------------------------------------ MMA (one warp per tile, one of its threads issuing)
template <int DP, bool BF16>
__device__ __forceinline__ void mma(const SeqFwdArgs& a, uint8_t* base, Bars* bars, uint32_t tmem, uint32_t gq,
                                    const WaitGuard& g) {
  using L = Layout<DP>;
  const int steps = (a.s.D + 15) / 16;  // of 16 features
  const uint32_t id_s = idesc_f16(128, 128, BF16, false, false);
  const uint32_t id_o = idesc_f16(128, steps * 16, BF16, false, true);
  uint32_t n = 0, u = 0, it = 0, own = 0, queries[2] = {0, 0};
  bool ok = true;
  Work w;
  for (; ok && take<true>(bars, it, g, w); ++it) {
    __syncwarp();
    if (elect_one()) give_back(bars, it);
    const int j0 = uniform(w.j0), j1 = uniform(w.j1);
    const bool one = uniform(single(w, a.TQ)) != 0;
    const Share sh = share_of(w, static_cast<int>(gq), a.TQ);
    const int from = uniform(sh.from), to = uniform(sh.to), step = one ? 2 : 1;
    const uint32_t qb = one ? static_cast<uint32_t>(uniform(w.q)) : gq;
    const uint64_t qd = smem_desc(smem_u32(base + L::q + qb * L::kTB), 16, 1024, kSwizzle128B);
    // (the other tile's buffer too: it is released by both)
    for (uint32_t b = 0; b < 2; ++b)
      if (!one || b == qb) {
        if (!mbar_wait_warp_inl(smem_u32(&bars->q_full[b]), queries[b] & 1, g)) ok = false;
        ++queries[b];
      }
    if (!ok) break;
    tc_fence_after();
    if (elect_one()) {
      if (!one) mbar_arrive(smem_u32(&bars->q_empty[gq ^ 1]));
      if (from >= to) mbar_arrive(smem_u32(&bars->q_empty[qb]));
    }
    __syncwarp();
    int next = from;  // this warpgroup's next key tile
    for (int j = j0; j < j1; ++j, ++n) {
      const uint32_t uk = 2 * n, uv = 2 * n + 1, ks = uk % L::kSlots, vs = uv % L::kSlots;
      if (!mbar_wait_warp_inl(smem_u32(&bars->full[ks]), (uk / L::kSlots) & 1, g)) { ok = false; break; }
      if (j != next || j >= to) {  // the other warpgroup's
        if (elect_one()) mbar_arrive(smem_u32(&bars->empty[ks]));
        if (!mbar_wait_warp_inl(smem_u32(&bars->v_ready[n % kReady]), (n / kReady) & 1, g)) { ok = false; break; }
        if (elect_one()) mbar_arrive(smem_u32(&bars->empty[vs]));
        __syncwarp();
        continue;
      }
      next += step;
      // S takes the place of the previous P, which its P·V must have read
      if (u > 0 && !mbar_wait_warp_inl(smem_u32(&bars->pv_done[gq]), (u - 1) & 1, g)) { ok = false; break; }
      tc_fence_after();
      const uint64_t kd = smem_desc(smem_u32(base + L::ring + ks * L::kTB), 16, 1024, kSwizzle128B);
      if (elect_one()) {
#pragma unroll
        for (int k = 0; k < DP / 16; ++k) {
          const uint64_t o = (k & 3) * 2 + (k >> 2) * (L::kHalf / 16);
          if (k < steps) umma_ss(tmem + col_s(gq), qd + o, kd + o, id_s, k > 0);
        }
        umma_commit(smem_u32(&bars->s_full[gq]));
        umma_commit(smem_u32(&bars->empty[ks]));
        if (next >= to) umma_commit(smem_u32(&bars->q_empty[qb]));
      }
      __syncwarp();
      if (!mbar_wait_warp_inl(smem_u32(&bars->v_ready[n % kReady]), (n / kReady) & 1, g)) { ok = false; break; }
      if (!mbar_wait_warp_inl(smem_u32(&bars->full[vs]), (uv / L::kSlots) & 1, g)) { ok = false; break; }
      if (j == from && !mbar_wait_warp_inl(smem_u32(&bars->o_free[gq]), (own & 1) ^ 1, g)) { ok = false; break; }
      const uint64_t vd = smem_desc(smem_u32(base + L::ring + vs * L::kTB), L::kHalf, 1024, kSwizzle128B);
      // the first 64 keys while the softmax works on the others
      if (!mbar_wait_warp_inl(smem_u32(&bars->p_half[gq]), u & 1, g)) { ok = false; break; }
      tc_fence_after();
      if (elect_one()) {
#pragma unroll
        for (int k = 0; k < 4; ++k)  // steps of 16 keys (8 columns of packed pairs)
          umma_ts(tmem + col_o(gq), tmem + col_s(gq) + k * 8, vd + k * (2048 / 16), id_o, (j > from || k > 0) ? 1u : 0u);
      }
      __syncwarp();
      if (!mbar_wait_warp_inl(smem_u32(&bars->p_full[gq]), u & 1, g)) { ok = false; break; }
      tc_fence_after();
      if (elect_one()) {
#pragma unroll
        for (int k = 4; k < 8; ++k)
          umma_ts(tmem + col_o(gq), tmem + col_s(gq) + k * 8, vd + k * (2048 / 16), id_o, 1u);
        umma_commit(smem_u32(&bars->pv_done[gq]));
        umma_commit(smem_u32(&bars->empty[vs]));
      }
      __syncwarp();
      ++u;
    }
    if (from < to) ++own;
  }
  __syncwarp();
  if (elect_one()) umma_commit(smem_u32(&bars->drain[gq]));
}

// ------------------------------------------------------------ the walk, and V's release (one warp)
template <bool BF16>
__device__ __forceinline__ uint32_t not_finite2(uint32_t x) {  // a mask of the halves that are not finite
  constexpr uint32_t e = BF16 ? 0x7F80u : 0x7C00u;
  return ((x & e) == e ? 0xffffu : 0u) | ((x & (e << 16)) == (e << 16) ? 0xffff0000u : 0u);
}

// Rows [from, to) of a V tile: values that are not finite become 0; true if there were any.
template <int DP, bool BF16>
__device__ __forceinline__ bool take_out(uint8_t* tile, int from, int to, int lane) {
  constexpr int per = DP / 8;  // 16-byte chunks a row
  bool found = false;
#pragma unroll 4
  for (int i = from * per + lane; i < to * per; i += 32) {
    const int r = i / per, c = i % per;
    uint4* p = reinterpret_cast<uint4*>(tile + (c >> 3) * Layout<DP>::kHalf + r * 128 + (c & 7) * 16);
    // (the swizzle permutes the chunks of a row among themselves: any order covers them)
    uint4 x = *p;
    const uint32_t m0 = not_finite2<BF16>(x.x), m1 = not_finite2<BF16>(x.y), m2 = not_finite2<BF16>(x.z),
                   m3 = not_finite2<BF16>(x.w);
    if (m0 | m1 | m2 | m3) {
      x.x &= ~m0, x.y &= ~m1, x.z &= ~m2, x.w &= ~m3;
      *p = x;
      found = true;
    }
  }
  return found;
}

template <int DP, bool BF16>
__device__ __forceinline__ void walk(const SeqFwdArgs& a, uint8_t* base, Bars* bars, const WaitGuard& g, int lane) {
  using L = Layout<DP>;
  Walk<QueryBlocks> walk;
  walk.init(a.s, QueryBlocks{a.W}, blockIdx.x, gridDim.x);
  PieceRecord* rec = a.records + 2 * blockIdx.x;
  if (lane < 2) rec[lane].used = 0;
  // (for the sums of the scores, which do not walk)
  if (a.scores && blockIdx.x == 0 && lane == 0) a.records[2 * gridDim.x].used = walk.crowded;
  __syncwarp();
  Work ring[2];  // published, V tiles not yet released: the current item and the one after it
  uint32_t pub = 0, n = 0;
  bool more = true;
  int turn = 0;  // buffer of the next single tile of queries
  auto publish = [&](Work& w) -> bool {
    w = walk.next();
    if (!w.stop && single(w, a.TQ)) {
      w.q = turn;
      turn ^= 1;
    }
    const uint32_t s = pub % kDescs;
    if (!mbar_wait_warp_inl(smem_u32(&bars->desc_empty[s]), ((pub / kDescs) & 1) ^ 1, g)) return false;
    if (lane == 0) {
      bars->work[s] = w;
      bars->dirty[s] = 0;
      if (!w.stop && w.slot >= 0) rec[w.slot] = PieceRecord{1, w.j1 == w.kt, w.b, w.kvh, w.row0, w.t0, w.nt, 0};
      mbar_arrive(smem_u32(&bars->desc_full[s]));
    }
    ++pub;
    more = !w.stop;
    return true;
  };
  if (!publish(ring[0])) return;
  for (uint32_t it = 0; !ring[0].stop; ++it) {
    ring[1].stop = 1;
    if (more && !publish(ring[1])) return;
    const Work w = ring[0];
    for (int j = w.j0; j < w.j1; ++j, ++n) {
      // A wait by parity has to see every phase of its barrier: keys and values take turns in a
      // slot, so K's arrival is waited for too, and no slot is refilled before this warp has let go.
      const uint32_t uk = 2 * n, uv = 2 * n + 1, slot = uv % L::kSlots;
      if (!mbar_wait_warp_inl(smem_u32(&bars->full[uk % L::kSlots]), (uk / L::kSlots) & 1, g)) return;
      if (lane == 0) mbar_arrive(smem_u32(&bars->empty[uk % L::kSlots]));
      if (!mbar_wait_warp_inl(smem_u32(&bars->full[slot]), (uv / L::kSlots) & 1, g)) return;
      const int last = w.kv_end - j * kTile;      // rows of the tile that some query sees
      const int all = w.pos + 1 - j * kTile;      // ... that every query sees
      if (last < kTile || all < last) {
        uint8_t* tile = base + L::ring + slot * L::kTB;
        if (all < (last < kTile ? last : kTile)) {
          const bool found = take_out<DP, BF16>(tile, all > 0 ? all : 0, last < kTile ? last : kTile, lane);
          if (__any_sync(0xffffffffu, found) && lane == 0) bars->dirty[it % kDescs] = 1;
        }
        for (int i = (last > 0 ? last : 0) * (DP / 8) + lane; i < kTile * (DP / 8); i += 32) {
          const int r = i / (DP / 8), c = i % (DP / 8);
          *reinterpret_cast<uint4*>(tile + (c >> 3) * L::kHalf + r * 128 + (c & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
        }
        fence_proxy_async_smem();
        __syncwarp();
      }
      if (lane == 0) {
        mbar_arrive(smem_u32(&bars->v_ready[n % kReady]));
        mbar_arrive(smem_u32(&bars->empty[slot]));
      }
    }
    ring[0] = ring[1];
  }
}

// ------------------------------------------------------------ softmax (warps 0..7)
__device__ __forceinline__ void st_global_32(void* p, const uint32_t (&x)[8]) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(x[0]), "r"(x[1]), "r"(x[2]),
               "r"(x[3]), "r"(x[4]), "r"(x[5]), "r"(x[6]), "r"(x[7])
               : "memory");
}

// Max of 32 scores (columns c0..), those past column `lim` taken out when MASK.
template <bool MASK>
__device__ __forceinline__ void chunk_max(uint32_t (&y)[32], int lim, float& mt) {
  float mx[4] = {mt, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
  for (int x = 0; x < 32; x += 2) {
    if (MASK) {
      if (x > lim) y[x] = 0xff800000u;
      if (x + 1 > lim) y[x + 1] = 0xff800000u;
    }
    mx[(x >> 1) & 3] = max3(mx[(x >> 1) & 3], __uint_as_float(y[x]), __uint_as_float(y[x + 1]));
  }
  mt = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
}

// P = 2^(y·s - m) of 32 scores, packed, and their sum.
template <bool BF16>
__device__ __forceinline__ void chunk_exp(const uint32_t (&y)[32], float2 sl2, float2 nm2, uint32_t (&pp)[16], float2& rs) {
#pragma unroll
  for (int x = 0; x < 32; x += 2) {
    const float2 t = fma2(make_float2(__uint_as_float(y[x]), __uint_as_float(y[x + 1])), sl2, nm2);
    const float p0 = ex2(t.x), p1 = ex2(t.y);
    rs = add2(rs, make_float2(p0, p1));
    pp[x >> 1] = pack2<BF16>(p0, p1);
  }
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

// 64 scores, times s·log2 e, for the sums of the weights.
__device__ __forceinline__ void leave_scores(const uint32_t (&y)[64], float scale_log2, float* to) {
#pragma unroll
  for (int x = 0; x < 64; x += 8) {
    uint32_t o[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) o[e] = __float_as_uint(__uint_as_float(y[x + e]) * scale_log2);
    st_global_32(to + x, o);
  }
}

// The values of V that were taken out of the item's tiles, added to a row that sees them
// (features c0 .. c0 + 63 of the unscaled O; what is added is an infinity or a NaN).
template <bool BF16>
__device__ __forceinline__ void add_back(const SeqFwdArgs& a, const Work& w, int pos, int c0, uint32_t (&out)[64]) {
  uint32_t x[64];  // indexed by a run-time column: kept apart from the caller's registers
#pragma unroll
  for (int c = 0; c < 64; ++c) x[c] = out[c];
  const SeqDesc& s = a.s;
  int from = w.pos + 1 > w.j0 * kTile ? w.pos + 1 : w.j0 * kTile;
  if (from < 0) from = 0;
  const int to = pos + 1 < w.j1 * kTile ? pos + 1 : w.j1 * kTile;
  for (int j = from; j < to; ++j) {
    const uint16_t* row;
    if (s.table) {
      const int p = page_of(s, w.b, j);
      if (p < 0) continue;
      row = a.v + p * a.v_page + (static_cast<long long>(j % s.page) * s.kv_heads + w.kvh) * s.D;
    } else {
      row = a.v + static_cast<long long>(w.row0 + j) * a.v_stride + static_cast<long long>(w.kvh) * s.D;
    }
#pragma unroll 1
    for (int c = 0; c < 64 && c0 + c < s.D; ++c) {
      const uint16_t v = row[c0 + c];
      if (not_finite2<BF16>(v) & 0xffffu) x[c] = __float_as_uint(__uint_as_float(x[c]) + to_f32<BF16>(v));
    }
  }
#pragma unroll
  for (int c = 0; c < 64; ++c) out[c] = x[c];
}

// SCORES: leave the scores behind for the sums of the weights (a kernel of its own: as a branch in
// the loop it cost prompts 3 %).
template <int DP, bool BF16, bool SCORES>
__device__ __forceinline__ void softmax(const SeqFwdArgs& a, uint8_t* base, Bars* bars, uint32_t tmem,
                                        const WaitGuard& g) {
  const SeqDesc& s = a.s;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int gq = warp >> 2, wq = warp & 3, r = wq * 32 + lane;
  const uint32_t trow = tmem + (static_cast<uint32_t>(wq * 32) << 16);
  const uint32_t scol = trow + col_s(gq), ocol = trow + col_o(gq);
  const int dt = r / s.group, head = r % s.group;  // token within the tile, head within the group
  const float scale_log2 = a.scale_log2;
  const float2 sl2 = make_float2(scale_log2, scale_log2);
  uint32_t u = 0, it = 0, merges = 0, turns = 0;
  bool ok = true;
  Work w;
  for (; ok && take<true>(bars, it, g, w); ++it) {
    const bool one = single(w, a.TQ);
    const Share sh = share_of(w, gq, a.TQ);
    const int both = one ? 0 : share_of(w, gq ^ 1, a.TQ).to;  // below it the other tile works too
    const int first = one ? 0 : gq * a.TQ;       // the tile's first token within the block
    const int tok = first + dt;
    const bool live = dt < a.TQ && tok < w.nt;
    const bool any = __any_sync(0xffffffffu, live);
    const int pos = w.pos + tok;
    float m = 0.0f, l = 0.0f;
    bool have = false;
    if (!any) {  // no row of this warp is anybody's: P may be what it is
      for (int j = sh.from; j < sh.to; j += sh.step, ++u) {
        if (!mbar_wait_warp_inl(smem_u32(&bars->s_full[gq]), u & 1, g)) { ok = false; break; }
        if (j < both) {
          if (!mbar_wait_warp_inl(smem_u32(&bars->turn[gq]), (turns & 1) ^ (gq ^ 1), g)) { ok = false; break; }
          ++turns;
          if (lane == 0) mbar_arrive(smem_u32(&bars->turn[gq ^ 1]));
        }
        if (lane == 0) {
          mbar_arrive(smem_u32(&bars->p_half[gq]));
          mbar_arrive(smem_u32(&bars->p_full[gq]));
        }
      }
    } else {
      for (int j = sh.from; j < sh.to; j += sh.step) {
        if (!mbar_wait_warp_inl(smem_u32(&bars->s_full[gq]), u & 1, g)) { ok = false; break; }
        tc_fence_after();
        uint32_t ya[64], yb[64];
        uint32_t(&y0)[32] = *reinterpret_cast<uint32_t(*)[32]>(&ya[0]);
        uint32_t(&y1)[32] = *reinterpret_cast<uint32_t(*)[32]>(&ya[32]);
        uint32_t(&y2)[32] = *reinterpret_cast<uint32_t(*)[32]>(&yb[0]);
        uint32_t(&y3)[32] = *reinterpret_cast<uint32_t(*)[32]>(&yb[32]);
        float mt = -INFINITY;
        tmem_ld64(scol, ya);
        tmem_wait_ld(ya);
        tmem_ld64(scol + 64, yb);
        if (w.pos + first >= j * kTile + kTile - 1) {
          // the tile's first token sees the whole key tile: no row needs its mask
          chunk_max<false>(y0, 0, mt);
          chunk_max<false>(y1, 0, mt);
          tmem_wait_ld(yb);
          chunk_max<false>(y2, 0, mt);
          chunk_max<false>(y3, 0, mt);
        } else {
          const int lim = pos - j * kTile;
          chunk_max<true>(y0, lim, mt);
          chunk_max<true>(y1, lim - 32, mt);
          tmem_wait_ld(yb);
          chunk_max<true>(y2, lim - 64, mt);
          chunk_max<true>(y3, lim - 96, mt);
        }
        if constexpr (SCORES) {
          if (live) {
            const size_t at = (static_cast<size_t>(w.row0) + w.t0 + tok) * s.q_heads + w.kvh * s.group + head;
            float* to = a.scores + at * a.scores_ld + static_cast<size_t>(j) * kTile;
            leave_scores(ya, scale_log2, to);
            leave_scores(yb, scale_log2, to + 64);
          }
          __syncwarp();
        }
        mt *= scale_log2;  // (a positive factor keeps the max)
        bool moved = false;
        float alpha = 1.0f;
        if (mt != -INFINITY && (!have || mt > m + kMoveLog2)) {
          moved = have;
          alpha = have ? ex2(m - mt) : 1.0f;
          m = mt;
          have = true;
        }
        // O so far is complete: this tile's S was issued behind the previous P·V
        if (__any_sync(0xffffffffu, moved)) {
          rescale<DP>(ocol, alpha);
          l *= alpha;
        }
        const float2 nm2 = make_float2(-m, -m);
        float2 rs = make_float2(0.0f, 0.0f);
        // Two tiles take turns for the exponentials, tile 0 first: without that their phases fall into
        // step, and the tensor core idles while both compute (16384 tokens, 16 heads of 128: 1085 us
        // without turns, 891 with).
        if (j < both && !mbar_wait_warp_inl(smem_u32(&bars->turn[gq]), (turns & 1) ^ (gq ^ 1), g)) { ok = false; break; }
        uint32_t pp[32];
        uint32_t(&p0)[16] = *reinterpret_cast<uint32_t(*)[16]>(&pp[0]);
        uint32_t(&p1)[16] = *reinterpret_cast<uint32_t(*)[16]>(&pp[16]);
        chunk_exp<BF16>(y0, sl2, nm2, p0, rs);
        chunk_exp<BF16>(y1, sl2, nm2, p1, rs);
        tmem_st32(scol, pp);
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(smem_u32(&bars->p_half[gq]));
        }
        chunk_exp<BF16>(y2, sl2, nm2, p0, rs);
        if (j < both) {  // handed over a little early
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&bars->turn[gq ^ 1]));
        }
        chunk_exp<BF16>(y3, sl2, nm2, p1, rs);
        if (j < both) ++turns;
        tmem_st32(scol + 32, pp);
        l += rs.x + rs.y;
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(smem_u32(&bars->p_full[gq]));
        }
        ++u;
      }
    }
    if (!ok) break;
    const bool worked = sh.from < sh.to;
    if (worked && !mbar_wait_warp_inl(smem_u32(&bars->pv_done[gq]), (u - 1) & 1, g)) break;
    tc_fence_after();
    const size_t row = static_cast<size_t>(w.row0) + w.t0 + tok;
    const int h = w.kvh * s.group + head;
    const bool two = one && w.j1 - w.j0 > 1;  // the second warpgroup has a share to add
    if (gq == 1 && one) {
      if (two) {
        bars->merge[r] = make_float2(m, l);
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&bars->merge_full));
      }
    } else {
      float f0 = 1.0f, f1 = 0.0f;
      if (two) {
        if (!mbar_wait_warp_inl(smem_u32(&bars->merge_full), merges & 1, g)) break;
        ++merges;
        tc_fence_after();
        const float2 o = bars->merge[r];
        const float big = l == 0.0f ? o.x : (o.y == 0.0f ? m : fmaxf(m, o.x));
        f0 = l == 0.0f ? 0.0f : ex2(m - big);
        f1 = o.y == 0.0f ? 0.0f : ex2(o.x - big);
        l = l * f0 + o.y * f1;
        m = big;
      }
      if (worked && any) {
        const bool dirty = bars->dirty[it % kDescs] != 0;
        const float inv = l == 0.0f ? 0.0f : 1.0f / l;
        uint16_t* out = a.out + row * a.out_stride + static_cast<size_t>(h) * s.D;
        const size_t prow = (static_cast<size_t>(blockIdx.x) * 2 + (w.slot > 0)) * 256 + gq * 128 + r;
        float* part = a.part_o + prow * DP;
#pragma unroll 1
        for (int c = 0; c < s.D; c += 64) {
          uint32_t x[64];
          tmem_ld64(ocol + c, x);
          if (two) {
            uint32_t y[64];
            tmem_ld64(trow + col_o(1) + c, y);
            tmem_wait_ld(y);
            tmem_wait_ld(x);
#pragma unroll
            for (int e = 0; e < 64; ++e)
              x[e] = __float_as_uint(__uint_as_float(x[e]) * f0 + __uint_as_float(y[e]) * f1);
          }
          tmem_wait_ld(x);
          if (live) {
            if (dirty) add_back<BF16>(a, w, pos, c, x);
            if (w.slot < 0) {
#pragma unroll
              for (int e = 0; e < 64; e += 16) {
                uint32_t o[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                  const float lo = __uint_as_float(x[e + 2 * i]) * inv, hi = __uint_as_float(x[e + 2 * i + 1]) * inv;
                  o[i] = l == 0.0f ? 0u : pack2<BF16>(lo, hi);
                }
                if (a.out32) {
                  if (c + e < s.D) st_global_32(out + c + e, o);
                } else {
                  if (c + e < s.D) *reinterpret_cast<uint4*>(out + c + e) = make_uint4(o[0], o[1], o[2], o[3]);
                  if (c + e + 8 < s.D) *reinterpret_cast<uint4*>(out + c + e + 8) = make_uint4(o[4], o[5], o[6], o[7]);
                }
              }
            } else {
#pragma unroll
              for (int e = 0; e < 64; e += 8) {
                const uint32_t(&o)[8] = *reinterpret_cast<const uint32_t(*)[8]>(&x[e]);
                st_global_32(part + c + e, o);
              }
            }
          }
          __syncwarp();  // the loads above are the whole warp's
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if (worked) mbar_arrive(smem_u32(&bars->o_free[gq]));
        if (two) mbar_arrive(smem_u32(&bars->o_free[1]));
      }
      if (live) {
        if (w.slot < 0)
          a.lse[static_cast<size_t>(h) * s.tokens + row] = l == 0.0f ? -INFINITY : (m + lg2(l)) * kSeqLn2;
        else
          a.part_ml[(static_cast<size_t>(blockIdx.x) * 2 + w.slot) * 256 + gq * 128 + r] = make_float2(m, l);
      }
    }
    __syncwarp();
    if (lane == 0) give_back(bars, it);
  }
}

template <int DP, bool BF16, bool SCORES>
__global__ void __launch_bounds__(kThreads, 1) evo_seq_fwd_kernel(const __grid_constant__ SeqFwdArgs a) {
  using L = Layout<DP>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  Bars* bars = reinterpret_cast<Bars*>(base + L::bars);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    bars->abort = 0;
    for (int i = 0; i < kDescs; ++i) {
      mbar_init(smem_u32(&bars->desc_full[i]), 1);
      mbar_init(smem_u32(&bars->desc_empty[i]), 11);  // producer, two MMA threads, eight softmax warps
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&bars->q_full[i]), 1);
      mbar_init(smem_u32(&bars->q_empty[i]), 2);  // both MMA warps
    }
    for (int i = 0; i < kMaxSlots; ++i) {
      mbar_init(smem_u32(&bars->full[i]), 1);
      mbar_init(smem_u32(&bars->empty[i]), 3);  // both MMA warps, and the one that releases V
    }
    for (int i = 0; i < kReady; ++i) mbar_init(smem_u32(&bars->v_ready[i]), 1);
    mbar_init(smem_u32(&bars->merge_full), 4);
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&bars->s_full[i]), 1);
      mbar_init(smem_u32(&bars->p_half[i]), 4);
      mbar_init(smem_u32(&bars->p_full[i]), 4);
      mbar_init(smem_u32(&bars->pv_done[i]), 1);
      mbar_init(smem_u32(&bars->o_free[i]), 4);
      mbar_init(smem_u32(&bars->drain[i]), 1);
      mbar_init(smem_u32(&bars->turn[i]), 4);
    }
    fence_barrier_init();
  }
  if (warp == kProducerWarp && lane == 0) {
    tma_prefetch_desc(&a.tq);
    tma_prefetch_desc(&a.tk);
    tma_prefetch_desc(&a.tv);
  }
  if (warp == kMmaWarp) {
    tmem_alloc(smem_u32(&bars->tmem_slot), 512);
    tmem_relinquish();
  }
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bars->tmem_slot;
  const WaitGuard g{a.wait_ns, a.s.status, &bars->abort};
  if (warp >= kProducerWarp) {
    setmaxnreg_dec<kRegsOther>();
    if (warp == kProducerWarp) {
      producer<DP>(a, base, bars, g, lane);
    } else if (warp == kWalkWarp) {
      walk<DP, BF16>(a, base, bars, g, lane);
    } else {
      mma<DP, BF16>(a, base, bars, tmem, static_cast<uint32_t>(uniform(warp) - kMmaWarp), g);
    }
    tc_fence_before();
    __syncthreads();
    if (warp == kMmaWarp) {
      const uint32_t all = bars->abort ? 0u : ~0u;  // (a CTA that gave up did not let go of every tile)
      const Owed owed[] = {{bars->full, L::kSlots, bars->tiles},
                           {bars->empty, L::kSlots, bars->tiles & all},
                           {&bars->q_full[0], 1, bars->queries[0]},
                           {&bars->q_full[1], 1, bars->queries[1]},
                           {&bars->q_empty[0], 1, bars->queries[0] & all},
                           {&bars->q_empty[1], 1, bars->queries[1] & all},
                           {&bars->drain[0], 1, 1},
                           {&bars->drain[1], 1, 1}};
      drain(owed, g);
      tc_fence_after();
      tmem_dealloc(tmem, 512);
    }
  } else {
    setmaxnreg_inc<kRegsSoftmax>();
    softmax<DP, BF16, SCORES>(a, base, bars, tmem, g);
    tc_fence_before();
    __syncthreads();
  }
}

// ------------------------------------------------------------ join
// The pieces of an item that the borders between CTAs cut: the one that begins it (slot 1 of
// CTA c), then slot 0 of c + 1, c + 2, ... up to its end, joined in that order.  Eight threads a row:
// M = max m, l = Σ l 2^(m - M), O = Σ O 2^(m - M).  Latency is what it costs (the records, then the
// (m, l), then O): 32 rows a block, so that every block of a launch is resident at once, and the
// pieces of a row read together.
constexpr int kJoinRows = 32;
template <int DP, bool BF16>
__global__ void __launch_bounds__(256) evo_seq_join_kernel(const __grid_constant__ SeqFwdArgs a, int ctas) {
  const int c0 = blockIdx.x, i = blockIdx.y * kJoinRows + (threadIdx.x >> 3), d0 = (threadIdx.x & 7) * (DP / 8);
  const PieceRecord first = a.records[2 * c0 + 1];
  const int pieces = count_pieces(a.records, c0, ctas);  // (read beside the first record)
  if (!first.used) return;
  const SeqDesc& s = a.s;
  const int gq = i >> 7, r = i & 127, dt = r / s.group, tok = gq * a.TQ + dt;
  const bool live = dt < a.TQ && tok < first.nt;
  if (!__any_sync(0xffffffffu, live)) return;
  auto at = [&](int p) { return (static_cast<size_t>(c0 + p) * 2 + (p == 0)) * 256 + i; };
  const int sub = threadIdx.x & 7;
  // (m, l) of eight pieces at a time, one a thread
  auto load_ml = [&](int base) {
    return live && base + sub < pieces ? a.part_ml[at(base + sub)] : make_float2(0.0f, 0.0f);
  };
  const float2 early = load_ml(0);
  float big = early.y != 0.0f ? early.x : -INFINITY;
  for (int base = 8; base < pieces; base += 8) {
    const float2 ml = load_ml(base);
    if (ml.y != 0.0f) big = fmaxf(big, ml.x);
  }
#pragma unroll
  for (int o = 4; o > 0; o >>= 1) big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, o));
  float o[DP / 8] = {};
  float l = 0.0f;
  for (int base = 0; base < pieces; base += 8) {
    const float2 ml = base == 0 ? early : load_ml(base);
    const float f_mine = ml.y != 0.0f ? ex2(ml.x - big) : 0.0f;
    for (int q0 = 0; q0 < 8 && base + q0 < pieces; q0 += 4) {
#pragma unroll
      for (int q = 0; q < 4; ++q) {  // the loads of four pieces under way together
        const float f = __shfl_sync(0xffffffffu, f_mine, q0 + q, 8), y = __shfl_sync(0xffffffffu, ml.y, q0 + q, 8);
        const float4* x = reinterpret_cast<const float4*>(a.part_o + at(base + q0 + q) * DP + d0);
        l += y * f;
#pragma unroll
        for (int e = 0; e < DP / 32; ++e) {
          float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
          if (y != 0.0f) v = x[e];  // (no key, or no piece: nothing is there)
          o[4 * e] = fmaf(v.x, f, o[4 * e]);
          o[4 * e + 1] = fmaf(v.y, f, o[4 * e + 1]);
          o[4 * e + 2] = fmaf(v.z, f, o[4 * e + 2]);
          o[4 * e + 3] = fmaf(v.w, f, o[4 * e + 3]);
        }
      }
    }
  }
  if (!live) return;
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;
  const size_t row = static_cast<size_t>(first.row0) + first.t0 + tok;
  const int h = first.kvh * s.group + r % s.group;
  uint16_t* out = a.out + row * a.out_stride + static_cast<size_t>(h) * s.D + d0;
#pragma unroll
  for (int e = 0; e < DP / 8; e += 8) {  // (columns past D hold nothing and are not written)
    uint32_t v[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) v[q] = l == 0.0f ? 0u : pack2<BF16>(o[e + 2 * q] * inv, o[e + 2 * q + 1] * inv);
    if (d0 + e < s.D) *reinterpret_cast<uint4*>(out + e) = make_uint4(v[0], v[1], v[2], v[3]);
  }
  if (d0 == 0) a.lse[static_cast<size_t>(h) * s.tokens + row] = l == 0.0f ? -INFINITY : (big + lg2(l)) * kSeqLn2;
}

template <int DP, bool BF16, bool SCORES>
cudaError_t launch_k(const SeqFwdArgs& a, int ctas, cudaStream_t st) {
  auto kern = evo_seq_fwd_kernel<DP, BF16, SCORES>;
  static bool limit_set[64] = {};
  cudaError_t e = ensure_smem_limit(kern, 232448, limit_set);
  if (e != cudaSuccess) return e;
  kern<<<ctas, kThreads, Layout<DP>::total + 1024, st>>>(a);
  return cudaGetLastError();
}
template <int DP, bool BF16>
cudaError_t launch_t(const SeqFwdArgs& a, int ctas, cudaStream_t st) {
  const cudaError_t e = a.scores ? launch_k<DP, BF16, true>(a, ctas, st) : launch_k<DP, BF16, false>(a, ctas, st);
  if (e != cudaSuccess || a.s.max_kv <= kTile) return e;  // one key tile: nothing is cut
  evo_seq_join_kernel<DP, BF16><<<dim3(ctas, 256 / kJoinRows), 256, 0, st>>>(a, ctas);
  return cudaGetLastError();
}

}  // namespace

size_t seq_fwd_workspace(int ctas, int D, SeqFwdArgs* a, uint8_t* ws) {
  const int DP = D <= 64 ? 64 : 128;
  size_t off = 0;
  auto take = [&](size_t bytes) {
    uint8_t* p = ws ? ws + off : nullptr;
    off += (bytes + 255) & ~size_t(255);
    return p;
  };
  uint8_t* rec = take((size_t(ctas) * 2 + 1) * sizeof(PieceRecord));
  uint8_t* ml = take(size_t(ctas) * 2 * 256 * sizeof(float2));
  uint8_t* po = take(size_t(ctas) * 2 * 256 * DP * sizeof(float));
  if (a) {
    a->records = reinterpret_cast<PieceRecord*>(rec);
    a->part_ml = reinterpret_cast<float2*>(ml);
    a->part_o = reinterpret_cast<float*>(po);
  }
  return off;
}

cudaError_t launch_seq_fwd(const SeqFwdArgs& a, int ctas, bool bf16, cudaStream_t st) {
  if (a.s.D <= 64) return bf16 ? launch_t<64, true>(a, ctas, st) : launch_t<64, false>(a, ctas, st);
  return bf16 ? launch_t<128, true>(a, ctas, st) : launch_t<128, false>(a, ctas, st);
}

}  // namespace evo
