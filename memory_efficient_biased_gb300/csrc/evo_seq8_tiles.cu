// evo_seq8_tiles.cu — attention over the 8-bit cache (include/evo_seq.h) for many rows a key, on tcgen05.
//
// Mathematics, rows, items and roles as in evo_seq_fwd.cu, with scales: S = q·code_k, t = s_k s·log2e·S,
// P' = 2^(t + log2 r_v - M), M following the maximum of t + log2 r_v, l = Σ P' / r_v and O = Σ P' v'; at the end O / l and
// lse = ln2·(M + log2 l).  Operands are in q's type, which holds every code exactly, and P' is rounded to it, as in the
// 16-bit forward.  What a value enters with is P' v':
//   bf16  v' = code and r_v = s_v: bf16 holds P s_v whatever the scales
//   fp16  v' = code times the power of two in s_v, as far as fp16 goes (2^-24 to 2^7), and r_v the rest of s_v (1 to 2 in
//         that range).  With all of s_v in P', fp16 would lose keys whose scale is small beside another's, though their
//         weight be as large
//
// The tensor core takes 16 bits from shared memory, so a tile of codes arrives in a staging buffer and four warps widen
// it into the ring that the products read: 128 KB a pair of key tiles in and out of shared memory, beside the products' own 192.
//
// What bounds it: the chain scores, maximum, exponentials, P·V of a pair of tiles, as in the 16-bit forward, and the widening
// beside it, on the same schedulers and the same shared memory (bf16 / fp16).  4096 tokens over 16,384 keys, 32 heads of 128: 948 / 976 us,
// where a copy widened beforehand and the 16-bit forward take 767; 2 x 64 tokens over 16,384 each 58 / 59 us, where those take 87;
// 16 x 16 tokens over 8192 each 146 / 145 (a key tile and SM 2.2 us: the ring holds a tile and a half, and the next keys are
// widened when a tile's P·V is done).  The widening is the better for few instructions and few loads under way: codes of bf16 take three
// instructions a pair more than f16's (146 us where those took 132), fp16's product and the wait for its factor 7 us
// each; one piece of a row at a time in bf16 146, two 144, four 155, but 4096 tokens 948, 976, 993; in fp16 154, 145, 163; loops of
// their own for keys and values, 152 and 155; what only the last tiles need in a loop of its own.
// No use: four slots and two staging buffers instead of three and three, codes loaded into registers instead of a staging
// buffer (twice as long: the loads' latency, and no registers to hide it in).
//
// Roles (16 warps, one CTA per SM, persistent over its share of the work):
//   warps 0-3, 4-7  softmax of query tile 0 and 1, one thread per row
//   warp 8          producer: Q tiles, and tiles of codes into the staging ring, by TMA (a page is a box)
//   warps 9, 10     the MMAs of tile 0 and 1
//   warp 11         the walk over the work, and the tiles' scales
//   warps 12-15     widening: a thread a row of K and V (rows of V that no query of the item sees become zeros, and
//                   codes that are NaN and seen by some rows only are taken out, to be put back at the end)
// Tensor memory (512 columns): S_0, S_1 (128 each, P' in place of S as packed pairs), O_0, O_1.
#include "evo_seq8_pages.cuh"
#include "evo_seq_fwd.cuh"

namespace evo {
namespace {

constexpr int kThreads = 512;
constexpr int kProducerWarp = 8, kMmaWarp = 9, kWalkWarp = 11, kWidenWarp = 12;
constexpr uint32_t kRegsLaunch = 128, kRegsSoftmax = 192, kRegsOther = 64;
static_assert(256 * kRegsOther + 256 * kRegsSoftmax <= kThreads * kRegsLaunch, "register split exceeds the launch");
constexpr int kDescs = 4, kScaleSlots = 8, kMaxSlots = 6;

struct Bars {
  uint64_t desc_full[kDescs], desc_empty[kDescs];
  uint64_t q_full[2], q_empty[2];
  uint64_t raw_full[kMaxSlots], raw_empty[kMaxSlots], full[kMaxSlots], empty[kMaxSlots];
  uint64_t scale_full[kScaleSlots], scale_empty[kScaleSlots];
  // turn: see the softmax; merge_full: the second warpgroup's share of a single tile is done
  uint64_t s_full[2], p_half[2], p_full[2], pv_done[2], o_free[2], drain[2], turn[2], merge_full;
  // of a key tile, 16 tokens each: s_k; log2 r_v and 1 / r_v; fp16: s_v / r_v, which V's codes are multiplied by
  alignas(16) float scales[kScaleSlots][4][8];
  Work work[kDescs];
  float2 merge[kTile];       // (M, l) of the second warpgroup's share of a single tile
  int dirty[kDescs];         // a V tile of the item held codes that were taken out
  uint32_t tiles, queries[2];  // tiles of codes and Q tiles that the producer asked for
  uint32_t tmem_slot;
  int abort;
};

template <int DP>
struct Layout {
  static constexpr uint32_t kHalf = kTile * 128u;                 // 64 features of 128 rows, 16 bits
  static constexpr uint32_t kTB = kTile * DP * 2u, kRaw = kTB / 2;  // a tile, and its codes
  static constexpr int kSlots = DP == 128 ? 3 : 6;                // of either ring
  static constexpr uint32_t q = 0, ring = 2 * kTB, raw = ring + kSlots * kTB, bars = raw + kSlots * kRaw;
  static constexpr uint32_t total = bars + ((sizeof(Bars) + 127) & ~127u);
};
static_assert(Layout<128>::total + 1024 <= 232448, "shared memory");

// The next descriptor, read by every lane of a warp.
__device__ __forceinline__ bool take(Bars* bars, uint32_t it, const WaitGuard& g, Work& w) {
  const uint32_t s = it % kDescs;
  if (!mbar_wait_warp_inl(smem_u32(&bars->desc_full[s]), (it / kDescs) & 1, g)) return false;
  w = bars->work[s];
  return !w.stop;
}
__device__ __forceinline__ void give_back(Bars* bars, uint32_t it) { mbar_arrive(smem_u32(&bars->desc_empty[it % kDescs])); }

// ------------------------------------------------------------ producer (one warp)
template <int DP>
__device__ __forceinline__ void producer(const Seq8FwdArgs& a, uint8_t* base, Bars* bars, const WaitGuard& g, int lane) {
  using L = Layout<DP>;
  const SeqDesc& s = a.f.s;
  const int box = s.page < kTile ? s.page : kTile, pages = kTile / box;
  const uint32_t qbytes = static_cast<uint32_t>(a.f.TQ * s.group) * 128u * (DP / 64);
  uint32_t use = 0, queries[2] = {0, 0};
  Work w;
  for (uint32_t it = 0; take(bars, it, g, w); ++it) {
    __syncwarp();
    if (lane == 0) give_back(bars, it);
    Pages look(s, w, pages);
    int first = s.page > kTile ? (w.j0 * kTile) % s.page : 0;  // row of the page that the tile begins at
    // Two tiles of queries take a buffer each; a single one takes the buffers by turns (w.q).
    const bool one = single(w, a.f.TQ);
    bool ok = true;
    for (int t = 0; ok && t < (one ? 1 : 2); ++t) {
      const int b = one ? w.q : t;
      ok = mbar_wait_warp_inl(smem_u32(&bars->q_empty[b]), (queries[b] & 1) ^ 1, g);
      if (ok && elect_one()) {
        const uint32_t full = smem_u32(&bars->q_full[b]);
        mbar_arrive_expect_tx(full, qbytes);
        for (int h = 0; h < DP / 64; ++h)
          tma_load_4d(smem_u32(base + L::q + b * L::kTB + h * L::kHalf), &a.f.tq, full, h * 64, 0, w.kvh,
                      w.row0 + w.t0 + t * a.f.TQ);
      }
      queries[b] += ok;
    }
    for (int j = w.j0; ok && j < w.j1; ++j) {
#pragma unroll
      for (int kv = 0; kv < 2; ++kv) {
        const uint32_t slot = use % L::kSlots;
        if (!mbar_wait_warp_inl(smem_u32(&bars->raw_empty[slot]), ((use / L::kSlots) & 1) ^ 1, g)) { ok = false; break; }
        const uint32_t full = smem_u32(&bars->raw_full[slot]), dst = smem_u32(base + L::raw + slot * L::kRaw);
        if (elect_one()) mbar_arrive_expect_tx(full, L::kRaw);
        for (int b = 0; b < pages; ++b) {
          const int p = look.of(b);
          if (elect_one()) tma_load_4d(dst + b * box * DP, kv ? &a.f.tv : &a.f.tk, full, 0, w.kvh, first, p);
        }
        ++use;
      }
      __syncwarp();
      if (s.page > kTile && (first += kTile) == s.page) first = 0;
      look.step(j);
    }
    if (!ok) break;
  }
  if (lane == 0) bars->tiles = use, bars->queries[0] = queries[0], bars->queries[1] = queries[1];
}

// ------------------------------------------------------------ MMA (one warp per tile, one of its threads issuing)
template <int DP, bool BF16>
__device__ __forceinline__ void mma(const Seq8FwdArgs& a, uint8_t* base, Bars* bars, uint32_t tmem, uint32_t gq,
                                    const WaitGuard& g) {
  using L = Layout<DP>;
  const int steps = a.f.s.D / 16;  // of 16 features
  const uint32_t id_s = idesc_f16(128, 128, BF16, false, false);
  const uint32_t id_o = idesc_f16(128, steps * 16, BF16, false, true);
  uint32_t n = 0, u = 0, it = 0, own = 0, queries[2] = {0, 0};
  bool ok = true;
  Work w;
  for (; ok && take(bars, it, g, w); ++it) {
    __syncwarp();
    if (elect_one()) give_back(bars, it);
    const int j0 = uniform(w.j0), j1 = uniform(w.j1);
    const bool one = uniform(single(w, a.f.TQ)) != 0;
    const Share sh = share_of(w, static_cast<int>(gq), a.f.TQ);
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
        if (!mbar_wait_warp_inl(smem_u32(&bars->full[vs]), (uv / L::kSlots) & 1, g)) { ok = false; break; }
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

// ------------------------------------------------------------ the walk, and the scales (one warp)
// fp16: what V's codes are multiplied by, the power of two in a block's scale as far as fp16 goes: codes of 448 just fit 2^7, and
// below 2^-15 the products are rounded to steps of 2^-24, as reading rounds them.
__device__ __forceinline__ float value_part(float s) {
  const float power = __uint_as_float(__float_as_uint(s) & 0x7f800000u);
  return fminf(fmaxf(power, 0x1p-24f), 0x1p7f);
}

template <bool BF16>
__device__ __forceinline__ void walk(const Seq8FwdArgs& a, Bars* bars, const WaitGuard& g, int lane) {
  const SeqDesc& s = a.f.s;
  const Cache8& c = a.c;
  Walk<QueryBlocks> walk;
  walk.init(s, QueryBlocks{a.f.W}, blockIdx.x, gridDim.x);
  PieceRecord* rec = a.f.records + 2 * blockIdx.x;
  if (lane < 2) rec[lane].used = 0;
  __syncwarp();
  const int pages = s.page < kTile ? kTile / s.page : 1;
  const ScaleLane mine(s, c, lane);
  uint32_t n = 0;
  int turn = 0;  // buffer of the next single tile of queries
  for (uint32_t it = 0;; ++it) {
    Work w = walk.next();
    if (!w.stop && single(w, a.f.TQ)) {
      w.q = turn;
      turn ^= 1;
    }
    const uint32_t d = it % kDescs;
    if (!mbar_wait_warp_inl(smem_u32(&bars->desc_empty[d]), ((it / kDescs) & 1) ^ 1, g)) return;
    if (lane == 0) {
      bars->work[d] = w;
      bars->dirty[d] = 0;
      if (!w.stop && w.slot >= 0) rec[w.slot] = PieceRecord{1, w.j1 == w.kt, w.b, w.kvh, w.row0, w.t0, w.nt, 0};
      mbar_arrive(smem_u32(&bars->desc_full[d]));
    }
    __syncwarp();
    if (w.stop) return;
    Pages look(s, w, pages);
    int first = s.page > kTile ? (w.j0 * kTile) % s.page : 0;
    auto fetch = [&](int j) -> float {
      const int p = look.of(mine.page);
      const bool there = lane < 16 && p < s.num_pages && j * kTile + mine.part * 16 < w.kv_end;
      const float x = there ? *mine.at(s, c, w.kvh, p, first) : 1.0f;
      if (s.page > kTile && (first += kTile) == s.page) first = 0;
      look.step(j);
      return x;
    };
    float now = fetch(w.j0);
    for (int j = w.j0; j < w.j1; ++j, ++n) {
      float next = 1.0f;
      if (j + 1 < w.j1) next = fetch(j + 1);
      const uint32_t slot = n % kScaleSlots;
      if (!mbar_wait_warp_inl(smem_u32(&bars->scale_empty[slot]), ((n / kScaleSlots) & 1) ^ 1, g)) return;
      if (lane < 8) {
        bars->scales[slot][0][lane] = now;
      } else if (lane < 16) {
        const float part = BF16 ? 1.0f : value_part(now), lv = log2_value_scale(now) - lg2(part);
        bars->scales[slot][1][lane - 8] = lv;
        bars->scales[slot][2][lane - 8] = ex2(-lv);
        bars->scales[slot][3][lane - 8] = part;
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&bars->scale_full[slot]));
      now = next;
    }
  }
}

// ------------------------------------------------------------ widening (four warps)
__device__ __forceinline__ uint32_t nan_bytes(uint32_t w) { return __vcmpeq4(w & 0x7f7f7f7fu, 0x7f7f7f7fu); }

template <int DP, bool BF16>
__device__ __forceinline__ void widen(const Seq8FwdArgs& a, uint8_t* base, Bars* bars, const WaitGuard& g, int r) {
  using L = Layout<DP>;
  const int lane = r & 31;
  uint32_t use = 0, n = 0;
  Work w;
  for (uint32_t it = 0; take(bars, it, g, w); ++it) {
    for (int j = w.j0; j < w.j1; ++j, ++n) {
      const int last = w.kv_end - j * kTile;  // rows of the tile that some query sees
      const int all = w.pos + 1 - j * kTile;  // ... that every query sees
#pragma unroll 1
      for (int kv = 0; kv < 2; ++kv, ++use) {
        const uint32_t slot = use % L::kSlots;
        uint32_t times = 0x3c003c00u;  // fp16: what the codes are multiplied by, for keys 1
        if (!BF16 && kv) {
          const uint32_t sc = n % kScaleSlots;
          if (!mbar_wait_warp_inl(smem_u32(&bars->scale_full[sc]), (n / kScaleSlots) & 1, g)) return;
          const float part = bars->scales[sc][3][r >> 4];
          times = pack2<false>(part, part);
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&bars->scale_empty[sc]));
        }
        if (!mbar_wait_warp_inl(smem_u32(&bars->raw_full[slot]), (use / L::kSlots) & 1, g)) return;
        if (!mbar_wait_warp_inl(smem_u32(&bars->empty[slot]), ((use / L::kSlots) & 1) ^ 1, g)) return;
        const uint8_t* from = base + L::raw + slot * L::kRaw + r * DP;
        uint8_t* to = base + L::ring + slot * L::kTB + r * 128;
        const bool none = kv && r >= last, some = kv && r >= all;
        bool lost = false;
        auto four = [&](uint32_t codes) {
          const uint2 f = f16x4_of_codes(codes);
          return BF16 ? make_uint2(bf16x2_of_codes(f.x), bf16x2_of_codes(f.y)) : make_uint2(mul_f16x2(f.x, times), mul_f16x2(f.y, times));
        };
        auto put = [&](int i, const uint4& x) {
          const uint2 f0 = four(x.x), f1 = four(x.y), f2 = four(x.z), f3 = four(x.w);
          uint8_t* half = to + (i >> 2) * L::kHalf;
          *reinterpret_cast<uint4*>(half + (((2 * i) ^ r) & 7) * 16) = make_uint4(f0.x, f0.y, f1.x, f1.y);
          *reinterpret_cast<uint4*>(half + (((2 * i + 1) ^ r) & 7) * 16) = make_uint4(f2.x, f2.y, f3.x, f3.y);
        };
        auto piece = [&](int i) { return *reinterpret_cast<const uint4*>(from + (DP == 128 ? (i ^ r) & 7 : (i ^ (r >> 1)) & 3) * 16); };
        if (!some) {
#pragma unroll(BF16 ? 1 : 2)
          for (int i = 0; i < DP / 16; ++i) put(i, piece(i));
        } else {
#pragma unroll 1
          for (int i = 0; i < DP / 16; ++i) {
            uint4 x = piece(i);
            const uint32_t n0 = nan_bytes(x.x), n1 = nan_bytes(x.y), n2 = nan_bytes(x.z), n3 = nan_bytes(x.w);
            lost = lost || (!none && (n0 | n1 | n2 | n3));
            x = none ? make_uint4(0u, 0u, 0u, 0u) : make_uint4(x.x & ~n0, x.y & ~n1, x.z & ~n2, x.w & ~n3);
            put(i, x);
          }
        }
        if (lost) bars->dirty[it % kDescs] = 1;
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(smem_u32(&bars->full[slot]));
          mbar_arrive(smem_u32(&bars->raw_empty[slot]));
        }
      }
    }
    __syncwarp();
    if (lane == 0) give_back(bars, it);
  }
}

// ------------------------------------------------------------ softmax (warps 0..7)
// The maximum of t + log2 s_v over 32 scores (columns c0.. of the row, lim the last that it sees), 16 of which share scales:
// f = s_k · what turns the row's products into scores, lv = log2 s_v.
template <bool MASK>
__device__ __forceinline__ void chunk_max(uint32_t (&y)[32], int lim, const float* f, const float* lv, float& mt) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
    for (int x = 16 * h; x < 16 * h + 16; x += 2) {
      if (MASK) {
        if (x > lim) y[x] = 0xff800000u;
        if (x + 1 > lim) y[x + 1] = 0xff800000u;
      }
      mx[(x >> 1) & 1] = max3(mx[(x >> 1) & 1], __uint_as_float(y[x]), __uint_as_float(y[x + 1]));
    }
    mt = fmaxf(mt, fmaf(fmaxf(mx[0], mx[1]), f[h], lv[h]));
  }
}

// P' = 2^(t + log2 s_v - M) of 32 scores, packed, and the sum of P' / s_v.
template <bool BF16>
__device__ __forceinline__ void chunk_exp(const uint32_t (&y)[32], const float* f, const float* lv, const float* iv, float m,
                                          uint32_t (&pp)[16], float& l) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const float b = lv[h] - m;
    const float2 f2 = make_float2(f[h], f[h]), b2 = make_float2(b, b);
    float2 rs = make_float2(0.0f, 0.0f);
#pragma unroll
    for (int x = 16 * h; x < 16 * h + 16; x += 2) {
      const float2 t = fma2(make_float2(__uint_as_float(y[x]), __uint_as_float(y[x + 1])), f2, b2);
      const float p0 = ex2(t.x), p1 = ex2(t.y);
      rs = add2(rs, make_float2(p0, p1));
      pp[x >> 1] = pack2<BF16>(p0, p1);
    }
    l = fmaf(rs.x + rs.y, iv[h], l);
  }
}

// Codes that were taken out of the item's V tiles: NaN in the features of a row that sees them (c0 .. c0 + 63 of O).
__device__ __forceinline__ void add_back(const Seq8FwdArgs& a, const Work& w, int pos, int c0, uint32_t (&out)[64]) {
  uint32_t x[64];  // indexed by a run-time column: kept apart from the caller's registers
#pragma unroll
  for (int c = 0; c < 64; ++c) x[c] = out[c];
  const SeqDesc& s = a.f.s;
  int from = w.pos + 1 > w.j0 * kTile ? w.pos + 1 : w.j0 * kTile;
  if (from < 0) from = 0;
  const int to = pos + 1 < w.j1 * kTile ? pos + 1 : w.j1 * kTile;
  for (int j = from; j < to; ++j) {
    const int p = page_of(s, w.b, j);
    if (p < 0) continue;
    const uint8_t* row = a.c.v_pages + p * a.c.v_page + (static_cast<long long>(j % s.page) * s.kv_heads + w.kvh) * s.D;
#pragma unroll 1
    for (int c = 0; c < 64 && c0 + c < s.D; ++c)
      if ((row[c0 + c] & 0x7f) == 0x7f) x[c] = 0x7fffffffu;
  }
#pragma unroll
  for (int c = 0; c < 64; ++c) out[c] = x[c];
}

template <int DP, bool BF16>
__device__ __forceinline__ void softmax(const Seq8FwdArgs& a, Bars* bars, uint32_t tmem, const WaitGuard& g) {
  const SeqDesc& s = a.f.s;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int gq = warp >> 2, wq = warp & 3, r = wq * 32 + lane;
  const uint32_t trow = tmem + (static_cast<uint32_t>(wq * 32) << 16);
  const uint32_t scol = trow + col_s(gq), ocol = trow + col_o(gq);
  const int dt = r / s.group, head = r % s.group;  // token within the tile, head within the group
  const float scale_log2 = a.f.scale_log2;
  uint32_t u = 0, it = 0, merges = 0, turns = 0, n = 0;
  bool ok = true;
  Work w;
  for (; ok && take(bars, it, g, w); ++it) {
    const bool one = single(w, a.f.TQ);
    const Share sh = share_of(w, gq, a.f.TQ);
    const int both = one ? 0 : share_of(w, gq ^ 1, a.f.TQ).to;  // below it the other tile works too
    const int first = one ? 0 : gq * a.f.TQ;       // the tile's first token within the block
    const int tok = first + dt;
    const bool live = dt < a.f.TQ && tok < w.nt;
    const bool any = __any_sync(0xffffffffu, live);
    const int pos = w.pos + tok;
    float m = 0.0f, l = 0.0f;
    bool have = false;
    int next = sh.from;
    for (int j = w.j0; j < w.j1; ++j, ++n) {
      const uint32_t slot = n % kScaleSlots;
      const uint32_t sc_full = smem_u32(&bars->scale_full[slot]), sc_empty = smem_u32(&bars->scale_empty[slot]);
      const uint32_t sc_phase = (n / kScaleSlots) & 1;
      const bool mine = j == next && j < sh.to;
      if (!mine || !any) {  // the other warpgroup's tile, or no row of this warp is anybody's: P may be what it is
        if (mine) {
          next += sh.step;
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
          ++u;
        }
        if (!mbar_wait_warp_inl(sc_full, sc_phase, g)) { ok = false; break; }  // (every phase is seen)
        if (lane == 0) mbar_arrive(sc_empty);
        continue;
      }
      next += sh.step;
      if (!mbar_wait_warp_inl(sc_full, sc_phase, g)) { ok = false; break; }
      float f[8], lv[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] = bars->scales[slot][0][e], lv[e] = bars->scales[slot][1][e];
      const float* iv = bars->scales[slot][2];
      if (!mbar_wait_warp_inl(smem_u32(&bars->s_full[gq]), u & 1, g)) { ok = false; break; }
      tc_fence_after();
      uint32_t ya[64], yb[64];
      uint32_t(&y0)[32] = *reinterpret_cast<uint32_t(*)[32]>(&ya[0]);
      uint32_t(&y1)[32] = *reinterpret_cast<uint32_t(*)[32]>(&ya[32]);
      uint32_t(&y2)[32] = *reinterpret_cast<uint32_t(*)[32]>(&yb[0]);
      uint32_t(&y3)[32] = *reinterpret_cast<uint32_t(*)[32]>(&yb[32]);
      float mt = -INFINITY;
      tmem_ld64(scol, ya);
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] = fmaxf(f[e] * scale_log2, 1.2e-38f);  // (one that underflows would make -inf a NaN)
      tmem_wait_ld(ya);
      tmem_ld64(scol + 64, yb);
      if (w.pos + first >= j * kTile + kTile - 1) {
        // the tile's first token sees the whole key tile: no row needs its mask
        chunk_max<false>(y0, 0, f, lv, mt);
        chunk_max<false>(y1, 0, f + 2, lv + 2, mt);
        tmem_wait_ld(yb);
        chunk_max<false>(y2, 0, f + 4, lv + 4, mt);
        chunk_max<false>(y3, 0, f + 6, lv + 6, mt);
      } else {
        const int lim = pos - j * kTile;
        chunk_max<true>(y0, lim, f, lv, mt);
        chunk_max<true>(y1, lim - 32, f + 2, lv + 2, mt);
        tmem_wait_ld(yb);
        chunk_max<true>(y2, lim - 64, f + 4, lv + 4, mt);
        chunk_max<true>(y3, lim - 96, f + 6, lv + 6, mt);
      }
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
      // Two tiles take turns for the exponentials, tile 0 first, as in the 16-bit forward.
      if (j < both && !mbar_wait_warp_inl(smem_u32(&bars->turn[gq]), (turns & 1) ^ (gq ^ 1), g)) { ok = false; break; }
      uint32_t pp[32];
      uint32_t(&p0)[16] = *reinterpret_cast<uint32_t(*)[16]>(&pp[0]);
      uint32_t(&p1)[16] = *reinterpret_cast<uint32_t(*)[16]>(&pp[16]);
      chunk_exp<BF16>(y0, f, lv, iv, m, p0, l);
      chunk_exp<BF16>(y1, f + 2, lv + 2, iv + 2, m, p1, l);
      tmem_st32(scol, pp);
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&bars->p_half[gq]));
      chunk_exp<BF16>(y2, f + 4, lv + 4, iv + 4, m, p0, l);
      if (j < both) {  // handed over a little early
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&bars->turn[gq ^ 1]));
      }
      chunk_exp<BF16>(y3, f + 6, lv + 6, iv + 6, m, p1, l);
      if (j < both) ++turns;
      tmem_st32(scol + 32, pp);
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(smem_u32(&bars->p_full[gq]));
        mbar_arrive(sc_empty);
      }
      ++u;
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
        const float inv = l == 0.0f ? 0.0f : 1.0f / l, unit = power_of_two(-whole_log2(l));
        uint16_t* out = a.f.out + row * a.f.out_stride + static_cast<size_t>(h) * s.D;
        const size_t prow = (static_cast<size_t>(blockIdx.x) * 2 + (w.slot > 0)) * 256 + gq * 128 + r;
        float* part = a.f.part_o + prow * DP;
#pragma unroll 1
        for (int c = 0; c < s.D; c += 64) {
          uint32_t x[64];
          tmem_ld64(ocol + c, x);
          if (two) {
#pragma unroll
            for (int q = 0; q < 64; q += 32) {
              uint32_t y[32];
              tmem_ld32(trow + col_o(1) + c + q, y);
              tmem_wait_ld(y);
              tmem_wait_ld(x);
#pragma unroll
              for (int e = 0; e < 32; ++e)
                x[q + e] = __float_as_uint(__uint_as_float(x[q + e]) * f0 + __uint_as_float(y[e]) * f1);
            }
          }
          tmem_wait_ld(x);
          if (live) {
            if (dirty) add_back(a, w, pos, c, x);
            if (w.slot < 0) {
#pragma unroll
              for (int e = 0; e < 64; e += 16) {
                uint32_t o[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                  const float lo = __uint_as_float(x[e + 2 * i]) * inv, hi = __uint_as_float(x[e + 2 * i + 1]) * inv;
                  o[i] = l == 0.0f ? 0u : pack2<BF16>(lo, hi);
                }
                if (c + e < s.D) {  // (head_dim is a multiple of 16)
                  if (a.f.out32) {
                    st_global_32(out + c + e, o);
                  } else {
                    *reinterpret_cast<uint4*>(out + c + e) = make_uint4(o[0], o[1], o[2], o[3]);
                    *reinterpret_cast<uint4*>(out + c + e + 8) = make_uint4(o[4], o[5], o[6], o[7]);
                  }
                }
              }
            } else {
#pragma unroll
              for (int e = 0; e < 64; e += 8) {  // (a piece's l is kept as 1 to 2, so that its m is one of weights)
                uint32_t o[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) o[i] = __float_as_uint(__uint_as_float(x[e + i]) * unit);
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
          a.f.lse[static_cast<size_t>(h) * s.tokens + row] = lse_of(m, l);
        else
          a.f.part_ml[(static_cast<size_t>(blockIdx.x) * 2 + w.slot) * 256 + gq * 128 + r] =
              make_float2(m + whole_log2(l), l * power_of_two(-whole_log2(l)));
      }
    }
    __syncwarp();
    if (lane == 0) give_back(bars, it);
  }
}

template <int DP, bool BF16>
__global__ void __launch_bounds__(kThreads, 1) evo_paged8_tiles_kernel(const __grid_constant__ Seq8FwdArgs a) {
  using L = Layout<DP>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  Bars* bars = reinterpret_cast<Bars*>(base + L::bars);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    bars->abort = 0;
    bars->tiles = bars->queries[0] = bars->queries[1] = 0;
    for (int i = 0; i < kDescs; ++i) {
      mbar_init(smem_u32(&bars->desc_full[i]), 1);
      mbar_init(smem_u32(&bars->desc_empty[i]), 15);  // producer, two MMA threads, eight softmax warps, four that widen
    }
    for (int i = 0; i < kMaxSlots; ++i) {
      mbar_init(smem_u32(&bars->raw_full[i]), 1);
      mbar_init(smem_u32(&bars->raw_empty[i]), 4);
      mbar_init(smem_u32(&bars->full[i]), 4);
      mbar_init(smem_u32(&bars->empty[i]), 2);  // both MMA warps
    }
    for (int i = 0; i < kScaleSlots; ++i) {
      mbar_init(smem_u32(&bars->scale_full[i]), 1);
      mbar_init(smem_u32(&bars->scale_empty[i]), BF16 ? 8 : 12);  // eight softmax warps; fp16: those that widen
    }
    mbar_init(smem_u32(&bars->merge_full), 4);
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&bars->q_full[i]), 1);
      mbar_init(smem_u32(&bars->q_empty[i]), 2);  // both MMA warps
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
    tma_prefetch_desc(&a.f.tq);
    tma_prefetch_desc(&a.f.tk);
    tma_prefetch_desc(&a.f.tv);
  }
  if (warp == kMmaWarp) {
    tmem_alloc(smem_u32(&bars->tmem_slot), 512);
    tmem_relinquish();
  }
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bars->tmem_slot;
  const WaitGuard g{a.f.wait_ns, a.f.s.status, &bars->abort};
  if (warp >= kProducerWarp) {
    setmaxnreg_dec<kRegsOther>();
    if (warp >= kWidenWarp) {
      widen<DP, BF16>(a, base, bars, g, static_cast<int>(threadIdx.x) - 32 * kWidenWarp);
    } else if (warp == kProducerWarp) {
      producer<DP>(a, base, bars, g, lane);
    } else if (warp == kWalkWarp) {
      walk<BF16>(a, bars, g, lane);
    } else {
      mma<DP, BF16>(a, base, bars, tmem, static_cast<uint32_t>(uniform(warp) - kMmaWarp), g);
    }
    tc_fence_before();
    __syncthreads();
    if (warp == kMmaWarp) {
      const uint32_t all = bars->abort ? 0u : ~0u;  // (a CTA that gave up did not let go of every tile)
      const Owed owed[] = {{bars->raw_full, L::kSlots, bars->tiles},
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
    softmax<DP, BF16>(a, bars, tmem, g);
    tc_fence_before();
    __syncthreads();
  }
}

template <int DP, bool BF16>
cudaError_t launch_t(const Seq8FwdArgs& a, int ctas, cudaStream_t st) {
  auto kern = evo_paged8_tiles_kernel<DP, BF16>;
  static bool limit_set[64] = {};
  cudaError_t e = ensure_smem_limit(kern, 232448, limit_set);
  if (e != cudaSuccess) return e;
  kern<<<ctas, kThreads, Layout<DP>::total + 1024, st>>>(a);
  if ((e = cudaGetLastError()) != cudaSuccess || a.f.s.max_kv <= kTile) return e;  // one key tile: nothing is cut
  return launch_seq_join(a.f, ctas, BF16, st);
}

}  // namespace

cudaError_t launch_paged8_tiles(const Seq8FwdArgs& a, int ctas, bool bf16, cudaStream_t st) {
  if (a.f.s.D <= 64) return bf16 ? launch_t<64, true>(a, ctas, st) : launch_t<64, false>(a, ctas, st);
  return bf16 ? launch_t<128, true>(a, ctas, st) : launch_t<128, false>(a, ctas, st);
}

}  // namespace evo
