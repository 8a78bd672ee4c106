// evo_seq8_few.cu — attention over the 8-bit cache (include/evo_seq.h) for few rows a key: single tokens,
// or a few of them, with their group's heads in 16 rows.
//
// Mathematics, per row (token, head) and block of keys with scales s_k and s_v: S = q·code_k,
// t = s_k s·log2e·S, P' = 2^(t + log2 s_v - M) with M the running maximum of t + log2 s_v, l = Σ P' / s_v and
// O = Σ P' code_v; at the end O / l and lse = ln2·(M + log2 l).  The codes are exact in fp16; so is q, for bf16 after its
// row is brought to a largest magnitude of 2^14 to 2^15 by a power of two (what falls below 2^-39 of that is lost).
//
// Range.  The weight that a value enters with is P' = P s_v, held times 2^14: fp16 has 11 bits of it down to 2^-28 of the
// largest, and loses it below 2^-39.  Among keys of like scales that loses weights below 2^-35 of the largest, less than l's own
// rounding.  (M is not rounded up to a whole number: the largest weight, a power of two, is then held exactly, which takes a fifth off
// the error of rows that few keys make.)  A key whose scale is far below another's may have a small P' and a large weight, though, and values of its own where
// the other's codes are 0.  So 16 keys whose scale is below 2^-4 of the largest so far, and some of whose P' are below 2^-14 of the row's
// largest, are held against their own largest: P' times 2^d, and O and l times 2^d before their product and 2^-d after it, d whole
// (72 at the most: O below 2^50 stays finite).  That costs such keys a second time what they take; without them nothing (a product with
// factors of its own for them beside the usual one took 7 to 14 % from all others, for the registers).
//
// Why mma.sync.  A byte of the cache has to be turned into 16 bits before a product of 16 bits
// takes it.  tcgen05 would take it from shared memory: staged, read, written twice as wide and read by the product,
// 6 to 7 bytes through shared memory for each of HBM's (128 a clock and SM, where HBM's share is 23).  Fragments
// in registers are read once from the staged tile and widened on their way into the product: 2 bytes. The
// products need 16 rows · 23 = 370 multiply-adds a clock and SM, a third of what mma.sync has.
//
// Roles (16 warps, one CTA per SM, persistent over its share of the work, evo_seq_sched.cuh):
//   warps 0-11  16 keys at a time each (they share their scales), in turns; M, l and O of their own, joined at the end of an
//               item.  Three a scheduler, for what a warp waits for between its products; that takes q out of their
//               registers, into shared memory
//   warps 12-15 the walk over the work, and keys by TMA (a page is a box); values; scales by cp.async; q, an item ahead.
//               A warp each: what one of them did for a tile, beside three busy warps, took longer than the tile
//
// What bounds it.  HBM: the 0.98 GB of four contexts of 120,000 tokens (8 kv heads of 128) take 72 to 79 us more than half
// of them, 6.2 to 6.9 TB/s by the machine.  In front of that lie 10 to 12 us until the first tiles are there (offsets, table,
// then 30 MB asked for at once on pages that no translation is held for), behind it 4 for the last tile and the joining of the
// warps, 5 of CTAs that were served later than others, and the joining launch, 3: four contexts of 245,609 tokens in all
// take 94 to 106 us (by the machine), 64 of 287,032 107 to 120, one of 777 12, one of 2000 14.  Steps: 16 keys a warp, eight warps, pages looked up
// tile by tile 119 us; page table entries a batch ahead and a second loading warp 101; the warps' shares joined
// for the live rows only 100, and the 64 contexts 136 -> 109; the join that asks for everything at once 94 (one context
// of 2000 21 -> 14).  No use: 32 keys a warp (fewer stages in flight), eight
// warps with q in registers (104), the join set up early by a programmatic launch (+1).
//
// Fragments.  Inside a product the order of the features (scores) and of the keys (P·V) is free, so a lane takes 16
// bytes next to each other: of key g for the scores (lane = 4 g + c: features 16 c .. and 64 + 16 c ..), of keys
// c, c + 4, c + 8, c + 12 for P·V (features 16 G(g) ..), whose bytes are paired by permutes.  Key (g / 2) + 4 (g % 2) stands
// in column g of the scores and G(g) = (g % 2) 4 + g / 2, so that with the tiles' 128-byte swizzle no read meets a bank twice
// (head_dim up to 64: twice).
#include <type_traits>

#include "evo_seq8_pages.cuh"

namespace evo {
namespace {

constexpr int kRows = kFewRows, kWarps = 12, kThreads = 32 * (kWarps + 4), kDescs = 4;
constexpr int kKeys = 16, kGroups = kTile / kKeys;  // keys that a warp takes at a time, times that a tile is
constexpr int kStages = 6;                          // tiles
constexpr int kJoined = 4;                          // rows whose shares are joined at a time, a warp each
// bf16 queries in fp16: log2 of what a row's largest magnitude becomes (or up to twice that).  What is below 2^-39 of it is lost
constexpr uint32_t kLift = 14;
constexpr float kHeld = 14.0f;  // log2 of what a row's largest P' is held as
constexpr float kNear = 4.0f;   // log2 of how far scales of values lie apart and need no more than that

template <int DP>
struct Layout {
  static constexpr uint32_t kTB = kTile * DP;     // codes of a tile's keys, and of its values
  static constexpr int kPitch = DP + 4;           // floats between rows of O to join: O, then M and l
  static constexpr uint32_t kQ = kRows * DP * 2;
  static constexpr uint32_t ring = 0, merge = kStages * 2 * kTB, q = merge + kWarps * kJoined * kPitch * 4;
  static constexpr uint32_t bars = q + 2 * kQ;
};

struct Bars {
  uint64_t desc_full[kDescs], desc_empty[kDescs];
  uint64_t full[kStages], empty[kStages];
  uint64_t merge_full, merge_empty, q_full[2], q_empty[2];
  alignas(8) float scales[kStages][2][8];  // of a stage: keys and values, 16 tokens each
  Work work[kDescs];
  float unit[2][kRows];           // scale · log2 e, and the power of two that q was divided by
  uint32_t tiles[3];              // that were asked for: keys, values, scales
  int abort;
};

__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint4 lds128(uint32_t addr) {
  uint4 x;
  asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w) : "r"(addr));
  return x;
}
__device__ __forceinline__ uint2 lds64(uint32_t addr) {
  uint2 x;
  asm volatile("ld.shared.v2.b32 {%0,%1}, [%2];" : "=r"(x.x), "=r"(x.y) : "r"(addr));
  return x;
}
// Bytes of four codes that are NaN, as 0xff.
__device__ __forceinline__ uint32_t nan_bytes(uint32_t w) { return __vcmpeq4(w & 0x7f7f7f7fu, 0x7f7f7f7fu); }

// Codes that are NaN taken out of the values of 16 keys, in the layout of P·V (key: the lane's first), and NaN put into
// the features of the rows that see them: the product of ones (a key that a row sees) and ones (a code that is NaN)
// counts them.
template <int COLS>
__device__ __forceinline__ void nan_values(uint32_t (&v)[4][COLS / 4], float (&o)[COLS][4], int key, int pos0, int pos1) {
  constexpr uint32_t one = 0x3c00u;  // 1 in fp16
  uint32_t seen[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const int at = key + 8 * (e >> 1), pos = (e & 1) ? pos1 : pos0;
    seen[e] = (at <= pos ? one : 0u) | (at + 4 <= pos ? one << 16 : 0u);
  }
#pragma unroll
  for (int e = 0; e < COLS / 4; ++e) {
    uint32_t bad[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      bad[i] = nan_bytes(v[i][e]);
      v[i][e] &= ~bad[i];
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      auto pair = [&](int i) {
        return ((bad[i] >> (8 * k)) & 1u ? one : 0u) | ((bad[i + 1] >> (8 * k)) & 1u ? one << 16 : 0u);
      };
      float count[4] = {};
      mma16816(count, seen, pair(0), pair(2));
#pragma unroll
      for (int x = 0; x < 4; ++x)
        if (count[x] > 0.0f) o[4 * e + k][x] = NAN;
    }
  }
}

// ------------------------------------------------------------ walk, loads, scales and q (a warp each)
// The next descriptor, for a warp that takes each one; false: no more work, or given up.
__device__ __forceinline__ bool take(Bars* bars, uint32_t it, const WaitGuard& g, Work& w) {
  const uint32_t d = it % kDescs;
  if (!mbar_wait_warp_inl(smem_u32(&bars->desc_full[d]), (it / kDescs) & 1, g)) return false;
  w = bars->work[d];
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(smem_u32(&bars->desc_empty[d]));
  return !w.stop;
}

// One item's tiles of keys, or of values, into the ring.
template <int DP>
__device__ __forceinline__ bool load_tiles(const Seq8FwdArgs& a, const CUtensorMap* map, uint32_t to, Bars* bars, const Work& w,
                                           uint32_t& use, const WaitGuard& g) {
  using L = Layout<DP>;
  const SeqDesc& s = a.f.s;
  const int box = s.page < kTile ? s.page : kTile, pages = kTile / box;  // a copy's rows, copies (and pages) of a tile
  Pages look(s, w, pages);
  int first = s.page > kTile ? (w.j0 * kTile) % s.page : 0;  // row of the page that the tile begins at
  for (int j = w.j0; j < w.j1; ++j, ++use) {
    const uint32_t st = use % kStages;
    if (!mbar_wait_warp_inl(smem_u32(&bars->empty[st]), ((use / kStages) & 1) ^ 1, g)) return false;
    const uint32_t full = smem_u32(&bars->full[st]), dst = to + st * 2 * L::kTB;
    if (elect_one()) mbar_arrive_expect_tx(full, L::kTB);
    for (int b = 0; b < pages; ++b) {
      const int p = look.of(b);
      if (elect_one()) tma_load_4d(dst + b * box * DP, map, full, 0, w.kvh, first, p);
    }
    __syncwarp();
    if (s.page > kTile && (first += kTile) == s.page) first = 0;
    look.step(j);
  }
  return true;
}

template <int DP, class Blocks>
__device__ __forceinline__ void produce(const Seq8FwdArgs& a, uint8_t* base, Bars* bars, const WaitGuard& g, int lane) {
  using L = Layout<DP>;
  Walk<Blocks> walk;
  walk.init(a.f.s, Blocks{a.f.W}, blockIdx.x, gridDim.x);
  PieceRecord* rec = a.f.records + 2 * blockIdx.x;
  if (!a.whole && lane < 2) rec[lane].used = 0;
  __syncwarp();
  uint32_t use = 0;
  for (uint32_t it = 0;; ++it) {
    const Work w = walk.next();
    const uint32_t d = it % kDescs;
    if (!mbar_wait_warp_inl(smem_u32(&bars->desc_empty[d]), ((it / kDescs) & 1) ^ 1, g)) break;
    if (lane == 0) {
      bars->work[d] = w;
      if (!w.stop && w.slot >= 0) rec[w.slot] = PieceRecord{1, w.j1 == w.kt, w.b, w.kvh, w.row0, w.t0, w.nt, 0};
      mbar_arrive(smem_u32(&bars->desc_full[d]));
    }
    if (w.stop || !load_tiles<DP>(a, &a.f.tk, smem_u32(base + L::ring), bars, w, use, g)) break;
  }
  if (lane == 0) bars->tiles[0] = use;
}

template <int DP>
__device__ __forceinline__ void load_values(const Seq8FwdArgs& a, uint8_t* base, Bars* bars, const WaitGuard& g, int lane) {
  uint32_t use = 0;
  Work w;
  for (uint32_t it = 0; take(bars, it, g, w); ++it)
    if (!load_tiles<DP>(a, &a.f.tv, smem_u32(base + Layout<DP>::ring + Layout<DP>::kTB), bars, w, use, g)) break;
  if (lane == 0) bars->tiles[1] = use;
}

__device__ __forceinline__ void fetch_scales(const Seq8FwdArgs& a, Bars* bars, const WaitGuard& g, int lane) {
  const SeqDesc& s = a.f.s;
  const Cache8& c = a.c;
  const int pages = s.page < kTile ? kTile / s.page : 1;
  const ScaleLane mine(s, c, lane);
  uint32_t use = 0;
  Work w;
  bool ok = true;
  for (uint32_t it = 0; ok && take(bars, it, g, w); ++it) {
    Pages look(s, w, pages);
    int first = s.page > kTile ? (w.j0 * kTile) % s.page : 0;
    for (int j = w.j0; j < w.j1; ++j, ++use) {
      const uint32_t st = use % kStages;
      const int p = look.of(mine.page);
      const float* from = mine.at(s, c, w.kvh, p, first);
      if (!mbar_wait_warp_inl(smem_u32(&bars->empty[st]), ((use / kStages) & 1) ^ 1, g)) { ok = false; break; }
      if (lane < 16) {
        const uint32_t full = smem_u32(&bars->full[st]);
        float* to = &bars->scales[st][lane >> 3][mine.part];
        if (p < s.num_pages && j * kTile + mine.part * 16 < w.kv_end) {
          asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(to)), "l"(from) : "memory");
          asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(full) : "memory");
        } else {
          *to = 1.0f;
          mbar_arrive(full);
        }
      }
      __syncwarp();
      if (s.page > kTile && (first += kTile) == s.page) first = 0;
      look.step(j);
    }
  }
  if (lane == 0) bars->tiles[2] = use;
}

// The items' q in fp16, an item ahead: features 64 i + 16 c + 4 k + (0, 1 | 2, 3) of row r become elements
// (2c, 2c + 1 | 2c + 8, 2c + 9) of step 4 i + k, where lane 4 (r % 8) + c takes them for its product.
template <int DP, bool BF16>
__device__ __forceinline__ void fetch_q(const Seq8FwdArgs& a, uint8_t* base, Bars* bars, const WaitGuard& g, int lane) {
  const SeqDesc& s = a.f.s;
  const int G = s.group;
  Work w;
  for (uint32_t it = 0; take(bars, it, g, w); ++it) {
    const uint32_t b = it & 1;
    if (!mbar_wait_warp_inl(smem_u32(&bars->q_empty[b]), ((it >> 1) & 1) ^ 1, g)) return;
    uint2 x[kRows];
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      x[r] = make_uint2(0u, 0u);
      if (4 * lane < s.D && r < w.nt * G)
        x[r] = *reinterpret_cast<const uint2*>(a.q + (static_cast<size_t>(w.row0) + w.t0 + r / G) * a.q_stride +
                                               static_cast<size_t>(w.kvh * G + r % G) * s.D + 4 * lane);
    }
    uint32_t* to = reinterpret_cast<uint32_t*>(base + Layout<DP>::q + b * Layout<DP>::kQ) +
                   (((lane >> 4) * 4 + (lane & 3)) * 32 + ((lane >> 2) & 3)) * 4;
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      float unit = a.f.scale_log2;
      if constexpr (BF16) {
        uint32_t most = __vmaxu2(x[r].x & 0x7fff7fffu, x[r].y & 0x7fff7fffu);  // magnitudes, as two 16-bit numbers
        most = __reduce_max_sync(0xffffffffu, max(most & 0xffffu, most >> 16));
        const uint32_t e = min(max(most >> 7, kLift + 1u), 254u);  // (an infinity stays one)
        const float down = __uint_as_float((254u + kLift - e) << 23);
        unit *= __uint_as_float((e - kLift) << 23);
        const float2 f0 = unpack2<true>(x[r].x), f1 = unpack2<true>(x[r].y);
        x[r] = make_uint2(pack2<false>(f0.x * down, f0.y * down), pack2<false>(f1.x * down, f1.y * down));
      }
      if (4 * lane < DP) {
        to[(r & 7) * 16 + (r >> 3)] = x[r].x;
        to[(r & 7) * 16 + (r >> 3) + 2] = x[r].y;
      }
      if (lane == 0) bars->unit[b][r] = unit;
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_u32(&bars->q_full[b]));
  }
}

// ------------------------------------------------------------ compute (warps 0..11)
template <int COLS>
__device__ __forceinline__ void scale_rows(float (&o)[COLS][4], float& l0, float& l1, float f0, float f1) {
  l0 *= f0, l1 *= f1;
#pragma unroll
  for (int n = 0; n < COLS; ++n) o[n][0] *= f0, o[n][1] *= f0, o[n][2] *= f1, o[n][3] *= f1;
}

// By which power of two keys are held apart whose largest t + log2 s_v of this lane is x, in a row whose maximum is m (both less kHeld): what brings the
// four lanes' largest to M, and at most 2^72, or what l allows (O is below 2^23 a key).
__device__ __forceinline__ float apart_by(float m, float x, float l) {
#pragma unroll
  for (int i = 1; i < 4; i *= 2) {
    x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, i));
    l = fmaxf(l, __shfl_xor_sync(0xffffffffu, l, i));
  }
  const float d = fminf(fminf(m - x, 72.0f), 120.0f - lg2(l));
  return x > -INFINITY && d > 0.0f ? floorf(d) : 0.0f;
}

template <int DP, bool BF16>
__device__ __forceinline__ void compute(const Seq8FwdArgs& a, uint8_t* base, Bars* bars, const WaitGuard& g) {
  using L = Layout<DP>;
  constexpr int kHalves = DP / 64, kCols = DP / 8;  // 16-byte pieces a lane of a key, tiles of eight features
  const SeqDesc& s = a.f.s;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, gr = lane >> 2, c = lane & 3;
  const int G = s.group, dt0 = gr / G, dt1 = (gr + 8) / G;  // rows gr and gr + 8: token within the item
  uint32_t use = 0, merges = 0;
  Work w;
  for (uint32_t it = 0; take(bars, it, g, w); ++it) {
    if (!mbar_wait_warp_inl(smem_u32(&bars->q_full[it & 1]), (it >> 1) & 1, g)) return;
    const float unit0 = bars->unit[it & 1][gr], unit1 = bars->unit[it & 1][gr + 8];
    const uint32_t qs = smem_u32(base + L::q + (it & 1) * L::kQ) + lane * 16;
    const int pos0 = w.pos + dt0, pos1 = w.pos + dt1;
    float o[kCols][4] = {};
    float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.0f, l1 = 0.0f;  // m: M - kHeld
    float top = -INFINITY;                                       // log2 of the largest scale of values so far
    // The 16 keys that are this warp's: every twelfth of all that the CTA walks over.  (A stage is either always one
    // of those that a warp looks at, or never: 12 times 16 keys are a tile and a half, and there are six stages.)
    const uint32_t end = (use + static_cast<uint32_t>(w.j1 - w.j0)) * kGroups;
    uint32_t n16 = use * kGroups;
    n16 += (warp + kWarps - n16 % kWarps) % kWarps;
    for (; n16 < end; n16 += kWarps) {
      const uint32_t tile = n16 / kGroups, st = tile % kStages;
      if (!mbar_wait_warp_inl(smem_u32(&bars->full[st]), (tile / kStages) & 1, g)) return;
      const int part = static_cast<int>(n16 % kGroups), key0 = (w.j0 + static_cast<int>(tile - use)) * kTile + part * kKeys;
      if (key0 >= w.kv_end) {
        if (lane == 0) mbar_arrive(smem_u32(&bars->empty[st]));
        continue;
      }
      const uint32_t kt = smem_u32(base + L::ring + 2 * st * L::kTB) + part * kKeys * DP, vt = kt + L::kTB;
      const float ks = bars->scales[st][0][part], vs = bars->scales[st][1][part];
      // ---- scores: column g of tile n is key 8 n + (g / 2) + 4 (g % 2)
      float t[2][4] = {};  // tile n: (row gr: keys 8n + c, 8n + c + 4), (row gr + 8: the same)
#pragma unroll
      for (int i = 0; i < kHalves; ++i) {
        uint32_t u[2][4];
#pragma unroll
        for (int n = 0; n < 2; ++n) {
          const int r = 8 * n + (gr >> 1) + 4 * (gr & 1);
          const uint32_t piece = DP == 128 ? static_cast<uint32_t>((c + 4 * i) ^ (r & 7)) : static_cast<uint32_t>(c ^ ((r >> 1) & 3));
          const uint4 x = lds128(kt + r * DP + piece * 16);
          u[n][0] = x.x, u[n][1] = x.y, u[n][2] = x.z, u[n][3] = x.w;
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const uint4 x = lds128(qs + (4 * i + k) * 512);
          const uint32_t q[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
          for (int n = 0; n < 2; ++n) {
            const uint2 f = f16x4_of_codes(u[n][k]);
            mma16816(t[n], q, f.x, f.y);
          }
        }
      }
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) t[n][e] *= (e < 2 ? unit0 : unit1) * ks;
      const bool edge = key0 + kKeys - 1 > w.pos;  // some row does not see some key
      if (edge) {
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (key0 + 8 * n + c + 4 * (e & 1) > (e < 2 ? pos0 : pos1)) t[n][e] = -INFINITY;
      }
      const float lv = log2_value_scale(vs), iv = ex2(-lv);
      float a0 = fmaxf(fmaxf(t[0][0], t[0][1]), fmaxf(t[1][0], t[1][1])) + (lv - kHeld);
      float a1 = fmaxf(fmaxf(t[0][2], t[0][3]), fmaxf(t[1][2], t[1][3])) + (lv - kHeld);
      // (the lanes that share rows need one M for them only where it moves)
      if (__any_sync(0xffffffffu, a0 > m0 || a1 > m1)) {
        a0 = fmaxf(a0, __shfl_xor_sync(0xffffffffu, a0, 1));
        a1 = fmaxf(a1, __shfl_xor_sync(0xffffffffu, a1, 1));
        a0 = fmaxf(a0, __shfl_xor_sync(0xffffffffu, a0, 2));
        a1 = fmaxf(a1, __shfl_xor_sync(0xffffffffu, a1, 2));
        const float n0 = fmaxf(m0, a0), n1 = fmaxf(m1, a1);
        const float f0 = m0 == -INFINITY ? 0.0f : ex2(m0 - n0), f1 = m1 == -INFINITY ? 0.0f : ex2(m1 - n1);
        m0 = n0, m1 = n1;
        scale_rows(o, l0, l1, f0, f1);
      }
      float b0 = lv - (m0 == -INFINITY ? 0.0f : m0), b1 = lv - (m1 == -INFINITY ? 0.0f : m1);
      // Keys whose scale is small, and which lie so far below M that fp16 would lose of them, are held 2^d times as large, and
      // so are O and l until their product is done (exactly: d is whole).
      top = fmaxf(top, lv);
      uint32_t apart = 0;  // d of both rows
      if (lv < top - kNear && __any_sync(0xffffffffu, (a0 < m0 - kHeld && a0 > -INFINITY) || (a1 < m1 - kHeld && a1 > -INFINITY))) {
        const float d0 = apart_by(m0, a0, l0), d1 = apart_by(m1, a1, l1);
        apart = static_cast<uint32_t>(d0) | static_cast<uint32_t>(d1) << 8;
        b0 += d0, b1 += d1;
        scale_rows(o, l0, l1, power_of_two(d0), power_of_two(d1));
      }
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) t[n][e] = ex2(t[n][e] + (e < 2 ? b0 : b1));
      l0 = fmaf((t[0][0] + t[0][1]) + (t[1][0] + t[1][1]), iv, l0);
      l1 = fmaf((t[0][2] + t[0][3]) + (t[1][2] + t[1][3]), iv, l1);
      const uint32_t p[4] = {pack2<false>(t[0][0], t[0][1]), pack2<false>(t[0][2], t[0][3]), pack2<false>(t[1][0], t[1][1]),
                             pack2<false>(t[1][2], t[1][3])};
      // ---- values: keys c, c + 4, c + 8, c + 12, features 16 G(g) .. (8 g ..)
      uint32_t v[4][kCols / 4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = c + 4 * i;
        if constexpr (DP == 128) {
          const uint32_t piece = static_cast<uint32_t>((((gr & 1) << 2) | (gr >> 1)) ^ (r & 7));
          const uint4 x = lds128(vt + r * DP + piece * 16);
          v[i][0] = x.x, v[i][1] = x.y, v[i][2] = x.z, v[i][3] = x.w;
        } else {
          const uint32_t piece = static_cast<uint32_t>((gr >> 1) ^ ((r >> 1) & 3));
          const uint2 x = lds64(vt + r * DP + piece * 16 + (gr & 1) * 8);
          v[i][0] = x.x, v[i][1] = x.y;
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&bars->empty[st]));
      if (edge) {
        // rows behind the last key that anyone sees: nothing; codes that are NaN: taken out, and put back where they are seen
        uint32_t lost = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int e = 0; e < kCols / 4; ++e) {
            if (key0 + c + 4 * i >= w.kv_end) v[i][e] = 0u;
            lost |= nan_bytes(v[i][e]);
          }
        if (__any_sync(0xffffffffu, lost != 0)) nan_values<kCols>(v, o, key0 + c, pos0, pos1);
      }
      // ---- O: bytes of keys (c, c + 4) and (c + 8, c + 12) paired, feature by feature
#pragma unroll
      for (int e = 0; e < kCols / 4; ++e) {
        const uint32_t x0 = __byte_perm(v[0][e], v[1][e], 0x5140), x1 = __byte_perm(v[0][e], v[1][e], 0x7362);
        const uint32_t y0 = __byte_perm(v[2][e], v[3][e], 0x5140), y1 = __byte_perm(v[2][e], v[3][e], 0x7362);
        const uint2 f0 = f16x4_of_codes(x0), f1 = f16x4_of_codes(x1), g0 = f16x4_of_codes(y0), g1 = f16x4_of_codes(y1);
        mma16816(o[4 * e], p, f0.x, g0.x);
        mma16816(o[4 * e + 1], p, f0.y, g0.y);
        mma16816(o[4 * e + 2], p, f1.x, g1.x);
        mma16816(o[4 * e + 3], p, f1.y, g1.y);
      }
      if (apart) scale_rows(o, l0, l1, power_of_two(-static_cast<float>(apart & 0xffu)), power_of_two(-static_cast<float>(apart >> 8)));
    }
    use += static_cast<uint32_t>(w.j1 - w.j0);
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_u32(&bars->q_empty[it & 1]));
    // ---- the warps' shares joined, four rows at a time, each by one warp; the others go on
    l0 += __shfl_xor_sync(0xffffffffu, l0, 1);
    l1 += __shfl_xor_sync(0xffffffffu, l1, 1);
    l0 += __shfl_xor_sync(0xffffffffu, l0, 2);
    l1 += __shfl_xor_sync(0xffffffffu, l1, 2);
    const int rows = w.nt * G;
    for (int first = 0; first < rows; first += kJoined, ++merges) {
      if (!mbar_wait_warp_inl(smem_u32(&bars->merge_empty), (merges & 1) ^ 1, g)) return;
      // Tile n holds, as elements 0 | 1 of a row, feature n of piece G(2 c) = c | G(2 c + 1) = 4 + c (D up to 64: of the eight
      // features 2 c | 2 c + 1).
      if ((gr & 4) == (first & 4)) {
        float* to = reinterpret_cast<float*>(base + L::merge) + (warp * kJoined + (gr & 3)) * L::kPitch;
        auto put = [&](auto upper) {
          constexpr bool up = decltype(upper)::value;
          constexpr int e = up ? 2 : 0;
#pragma unroll
          for (int x = 0; x < 2; ++x)
#pragma unroll
            for (int n = 0; n < kCols; n += 4)
              *reinterpret_cast<float4*>(to + (DP == 128 ? 16 * (c + 4 * x) : 8 * (2 * c + x)) + n) =
                  make_float4(o[n][e + x], o[n + 1][e + x], o[n + 2][e + x], o[n + 3][e + x]);
          if (c == 0) *reinterpret_cast<float2*>(to + DP) = up ? make_float2(m1, l1) : make_float2(m0, l0);
        };
        if (first < 8)
          put(std::false_type{});
        else
          put(std::true_type{});
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&bars->merge_full));
      if (warp >= kJoined) continue;
      if (!mbar_wait_warp_inl(smem_u32(&bars->merge_full), merges & 1, g)) return;
      const int r = first + warp, d = 4 * lane;  // row, four features
      if (r < rows && d < DP) {
        const float* from = reinterpret_cast<const float*>(base + L::merge) + warp * L::kPitch;
        float big = -INFINITY, l = 0.0f, f[kWarps];
#pragma unroll
        for (int i = 0; i < kWarps; ++i) {
          const float2 ml = *reinterpret_cast<const float2*>(from + i * kJoined * L::kPitch + DP);
          if (ml.y != 0.0f) big = fmaxf(big, ml.x);
        }
#pragma unroll
        for (int i = 0; i < kWarps; ++i) {
          const float2 ml = *reinterpret_cast<const float2*>(from + i * kJoined * L::kPitch + DP);
          // (a share that saw a NaN may have no maximum: its l is NaN, whatever it is scaled by)
          f[i] = ml.y == 0.0f ? 0.0f : (big == -INFINITY ? 1.0f : ex2(ml.x - big));
          if (ml.y != 0.0f) l += ml.y * f[i];
        }
        float x[4] = {};
#pragma unroll
        for (int i = 0; i < kWarps; ++i) {
          const float4 y = *reinterpret_cast<const float4*>(from + i * kJoined * L::kPitch + d);
          x[0] = fmaf(y.x, f[i], x[0]), x[1] = fmaf(y.y, f[i], x[1]), x[2] = fmaf(y.z, f[i], x[2]), x[3] = fmaf(y.w, f[i], x[3]);
        }
        const size_t row = static_cast<size_t>(w.row0) + w.t0 + r / G;
        const int h = w.kvh * G + r % G;
        if (w.slot < 0) {
          const float inv = l == 0.0f ? 0.0f : 1.0f / l;
          if (d < s.D)
            *reinterpret_cast<uint2*>(a.f.out + row * a.f.out_stride + static_cast<size_t>(h) * s.D + d) =
                l == 0.0f ? make_uint2(0u, 0u)
                          : make_uint2(pack2<BF16>(x[0] * inv, x[1] * inv), pack2<BF16>(x[2] * inv, x[3] * inv));
          if (lane == 0) a.f.lse[static_cast<size_t>(h) * s.tokens + row] = lse_of(big, l);
        } else {
          const size_t at = (static_cast<size_t>(blockIdx.x) * 2 + w.slot) * kRows + r;
          *reinterpret_cast<float4*>(a.f.part_o + at * DP + d) = make_float4(x[0], x[1], x[2], x[3]);
          if (lane == 0) a.f.part_ml[at] = make_float2(big, l);
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&bars->merge_empty));
    }
  }
}

template <int DP, bool BF16>
__global__ void __launch_bounds__(kThreads, 1) evo_paged8_few_kernel(const __grid_constant__ Seq8FwdArgs a) {
  using L = Layout<DP>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  Bars* bars = reinterpret_cast<Bars*>(base + L::bars);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    bars->abort = 0;
    bars->tiles[0] = bars->tiles[1] = bars->tiles[2] = 0;
    for (int i = 0; i < kDescs; ++i) {
      mbar_init(smem_u32(&bars->desc_full[i]), 1);
      mbar_init(smem_u32(&bars->desc_empty[i]), kWarps + 3);
    }
    for (int i = 0; i < kStages; ++i) {
      mbar_init(smem_u32(&bars->full[i]), 18);  // the copies' bytes (two warps), and a lane for each scale
      mbar_init(smem_u32(&bars->empty[i]), kGroups);
    }
    mbar_init(smem_u32(&bars->merge_full), kWarps);
    mbar_init(smem_u32(&bars->merge_empty), kJoined);
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&bars->q_full[i]), 1);
      mbar_init(smem_u32(&bars->q_empty[i]), kWarps);
    }
    fence_barrier_init();
  }
  if (warp == kWarps && lane == 0) {
    tma_prefetch_desc(&a.f.tk);
    tma_prefetch_desc(&a.f.tv);
  }
  __syncthreads();
  const WaitGuard g{a.f.wait_ns, a.f.s.status, &bars->abort};
  if (warp == kWarps) {
    if (a.whole)
      produce<DP, WholeBlocks>(a, base, bars, g, lane);
    else
      produce<DP, QueryBlocks>(a, base, bars, g, lane);
  } else if (warp == kWarps + 1) {
    load_values<DP>(a, base, bars, g, lane);
  } else if (warp == kWarps + 2) {
    fetch_scales(a, bars, g, lane);
  } else if (warp == kWarps + 3) {
    fetch_q<DP, BF16>(a, base, bars, g, lane);
  } else {
    compute<DP, BF16>(a, base, bars, g);
  }
  __syncthreads();
  if (warp == kWarps) {
    // Where a warp gave up, another may have asked for tiles more (fewer than there are stages): the arrivals that
    // are missing at their barriers, without which no wait for those copies would end before its limit.
    const uint32_t uses = max(bars->tiles[0], max(bars->tiles[1], bars->tiles[2]));
    for (int i = 0; i < 3; ++i)
      for (uint32_t use = bars->tiles[i]; use < uses; ++use)
        if (lane < (i < 2 ? 1 : 16)) mbar_arrive(smem_u32(&bars->full[use % kStages]));
    const Owed owed[] = {{bars->full, kStages, uses}};
    drain(owed, g);
  }
}

// ------------------------------------------------------------ join
// The pieces of an item that the borders between CTAs cut, as in evo_seq_fwd.cu's join: the one that begins it (slot 1 of
// CTA c), then slot 0 of c + 1, c + 2, ..., joined in that order, a warp a row.  Latency is what it costs, so the records, M and
// l of 32 pieces and O of eight are asked for together, before it is known how many there are (what lies
// behind the last is read and not used).
constexpr int kAhead = 8;
template <int DP, bool BF16>
__global__ void __launch_bounds__(32 * kRows) evo_paged8_join_kernel(const __grid_constant__ SeqFwdArgs a, int ctas) {
  constexpr int kF = DP / 32;  // features a lane
  const int c0 = blockIdx.x, lane = threadIdx.x & 31, r = threadIdx.x >> 5;
  auto at = [&](int p) { return (static_cast<size_t>(c0 + p) * 2 + (p == 0)) * kRows + r; };
  auto load_ml = [&](int p) { return c0 + p < ctas ? a.part_ml[at(p)] : make_float2(0.0f, 0.0f); };
  struct alignas(4 * kF) Features {
    float x[kF];
  };
  auto load_o = [&](int p0, Features (&o)[kAhead]) {
#pragma unroll
    for (int p = 0; p < kAhead; ++p)
      if (c0 + p0 + p < ctas) o[p] = *reinterpret_cast<const Features*>(a.part_o + at(p0 + p) * DP + lane * kF);
  };
  Features o[kAhead];
  load_o(0, o);
  float2 ml = load_ml(lane);
  const PieceRecord first = a.records[2 * c0 + 1];
  const int pieces = count_pieces(a.records, c0, ctas);
  const int G = a.s.group;
  if (!first.used || r >= first.nt * G) return;
  float big = lane < pieces && ml.y != 0.0f ? ml.x : -INFINITY;
  for (int base = 32; base < pieces; base += 32) {
    const float2 more = base + lane < pieces ? load_ml(base + lane) : make_float2(0.0f, 0.0f);
    if (more.y != 0.0f) big = fmaxf(big, more.x);
  }
#pragma unroll
  for (int x = 16; x > 0; x >>= 1) big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, x));
  float sum[kF] = {}, l = 0.0f;
  for (int p0 = 0; p0 < pieces; p0 += kAhead) {
    if (p0 > 0) {
      load_o(p0, o);
      if (p0 % 32 == 0) ml = load_ml(p0 + lane);
    }
    // (a piece that saw a NaN may have no maximum: its l is NaN, whatever it is scaled by)
    const float f_mine = p0 / 32 * 32 + lane < pieces && ml.y != 0.0f ? (big == -INFINITY ? 1.0f : ex2(ml.x - big)) : 0.0f;
#pragma unroll
    for (int p = 0; p < kAhead; ++p) {
      const float f = __shfl_sync(0xffffffffu, f_mine, (p0 + p) & 31), y = __shfl_sync(0xffffffffu, ml.y, (p0 + p) & 31);
      if (p0 + p >= pieces || y == 0.0f) continue;  // (no key: nothing is there)
      l += y * f;
#pragma unroll
      for (int e = 0; e < kF; ++e) sum[e] = fmaf(o[p].x[e], f, sum[e]);
    }
  }
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;
  const size_t row = static_cast<size_t>(first.row0) + first.t0 + r / G;
  const int h = first.kvh * G + r % G, d = lane * kF;
  if (d < a.s.D) {
    uint32_t v[kF / 2];
#pragma unroll
    for (int e = 0; e < kF / 2; ++e) v[e] = l == 0.0f ? 0u : pack2<BF16>(sum[2 * e] * inv, sum[2 * e + 1] * inv);
    uint16_t* out = a.out + row * a.out_stride + static_cast<size_t>(h) * a.s.D + d;
    if constexpr (kF == 4)
      *reinterpret_cast<uint2*>(out) = make_uint2(v[0], v[1]);
    else
      *reinterpret_cast<uint32_t*>(out) = v[0];
  }
  if (lane == 0) a.lse[static_cast<size_t>(h) * a.s.tokens + row] = lse_of(big, l);
}

template <int DP, bool BF16>
cudaError_t launch_t(const Seq8FwdArgs& a, int ctas, cudaStream_t st) {
  auto kern = evo_paged8_few_kernel<DP, BF16>;
  static bool limit_set[64] = {};
  cudaError_t e = ensure_smem_limit(kern, 232448, limit_set);
  if (e != cudaSuccess) return e;
  constexpr size_t smem = Layout<DP>::bars + sizeof(Bars) + 1024;
  static_assert(smem <= 232448, "shared memory");
  kern<<<ctas, kThreads, smem, st>>>(a);
  if ((e = cudaGetLastError()) != cudaSuccess || a.whole) return e;
  evo_paged8_join_kernel<DP, BF16><<<ctas, 32 * kRows, 0, st>>>(a.f, ctas);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_paged8_few(const Seq8FwdArgs& a, int ctas, bool bf16, cudaStream_t st) {
  if (a.f.s.D <= 64) return bf16 ? launch_t<64, true>(a, ctas, st) : launch_t<64, false>(a, ctas, st);
  return bf16 ? launch_t<128, true>(a, ctas, st) : launch_t<128, false>(a, ctas, st);
}

}  // namespace evo
