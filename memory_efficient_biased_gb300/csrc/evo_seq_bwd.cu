// evo_seq_bwd.cu — gradients of causal attention over packed prompts
// (include/evo_seq.h) on the tensor cores.
//
// With P = 2^(s·log2e·S - log2e·lse) rebuilt from the saved lse, dP = dO·vᵀ,
// dS = P∘(dP - delta) and delta = dO·O:
//     dV = Σ Pᵀ dO     dK = s Σ dSᵀ q     dQ = s Σ dS k.
// Five products per pair of tiles would do; here it is seven in two phases, since dQ
// gathers over key tiles what dK and dV gather over query tiles: in one walk either its
// sums (64 KB of fp32 per pair of tiles) go through L2 by atomics whose order changes the
// result, or wait for one another.  Two phases keep every sum in tensor memory, in a
// fixed order, and P and dS (the MMAs' A operands) in tensor memory too.
//
//   evo_seq_rows_kernel  (-lse·log2e, -delta) per row, [tokens][q_heads]
//   evo_seq_bwd_kernel   both phases in one launch, one behind the other in each CTA or, for little work,
//                        side by side (496 tokens of 4 heads of 64, forward included: 35 us, and 45 with a launch and a join for each)
//     dK, dV             items: 128 keys of a kv head, over the tiles of queries that see
//                        them (TQ tokens x the heads of the group, as in the forward, which sums
//                        dK and dV over a group's heads for nothing); Sᵀ = K Qᵀ, dPᵀ = V dOᵀ, a
//                        thread per key and half of the rows; dV += Pᵀ dO, dK += dSᵀ Q
//     dQ                 items: one tile of queries over its key tiles; S = Q Kᵀ, dP = dO Vᵀ, a
//                        thread per row and half of the keys; dQ += dS K
// Work is shared out and cut items joined as in the forward (evo_seq_sched.cuh); pieces are
// fp32 sums, added in order.
//
// Rounded to the input type: P and dS as MMA operands (what the tensor core takes), and the results.
// delta comes from the rounded O, the only one that the call is given: forming it again, as the sum of P dP,
// would take S and dP a third time (two products beside seven).  Errors of dQ and dK against 64 bits,
// relative to the exact result rounded once: 1.5 in sequences of 500 tokens and more, 1.6 at 128, 1.8 at 16,
// 2.0 at 8 and 2.5 at 2, where dP - delta cancels; dV 1.15 to 1.4 (bf16 and fp16, head_dim 64 and 128).
//
// What bounds it: the MMAs.  4096 + 1031 + 2500 + 565 tokens, 16 heads of 128 in groups of 4: dK/dV
// 170 us, of which 145 stay when the compute warps only hand over (timed in a copy), and dQ 150 us; the
// four (three) MMA groups of a tile take 2560 (1920) cycles at 80 an MMA, of 3400 (2670).  1.2 PFLOP/s
// of MMAs, 0.75 of what the formulas count, forward included.
#include "evo_seq_internal.h"
#include "evo_seq_sched.cuh"

#include <cstddef>
#include <type_traits>

namespace evo {
namespace {

constexpr int kThreads = 384;
constexpr int kProducerWarp = 8, kMmaWarp = 9, kRowsWarp = 10;  // and 11: the walk
constexpr uint32_t kRegsLaunch = 168, kRegsCompute = 200, kRegsOther = 104;
static_assert(128 * kRegsOther + 256 * kRegsCompute <= kThreads * kRegsLaunch, "register split exceeds the launch");
constexpr int kDescs = 4, kReady = 4;
// The streamed tiles: the one that is read twice (Q for dK, K for dQ: first by the scores, then by
// the gradient) has three buffers, the other (dO, V) two: 160 KB with head_dim 128, and the
// item's own two tiles 64 KB.
constexpr int kASlots = 3, kBSlots = 2;

struct Bars {
  uint64_t desc_full[kDescs], desc_empty[kDescs];
  uint64_t own_full, own_empty;                      // the item's own two tiles
  uint64_t a_full[kASlots], a_empty[kASlots];        // streamed: Q or K
  uint64_t b_full[kBSlots], b_empty[kBSlots];        // streamed: dO or V
  uint64_t ready[kReady];                            // a pair of streamed tiles, cleaned
  uint64_t rows_full[2], rows_empty[2];              // dK/dV: (lse, delta) of a tile of queries
  uint64_t s_full[2], dp_full, p_ready, dp_free;
  uint64_t ds_ready[2];                              // dQ: by turns; dK/dV: the first
  uint64_t second_done;                              // dS·(Q or K), and all before it, is done
  uint64_t acc_full, acc_free, drain;
  Work work[kDescs];
  uint32_t loads_a, loads_b, loads_own;  // copies that the producer asked for
  uint32_t tmem_slot;
  int abort;
  int go;  // dQ's phase begins
};

template <int DP>
struct Layout {
  static constexpr uint32_t kHalf = kTile * 128u;
  static constexpr uint32_t kTB = kTile * DP * 2u;
  static constexpr uint32_t own = 0, a = 2 * kTB, b = a + kASlots * kTB, rows = b + kBSlots * kTB,
                            bars = rows + 2 * kTile * 8u;
  static constexpr uint32_t total = bars + ((sizeof(Bars) + 127) & ~127u);
};
static_assert(Layout<128>::total <= 232448, "shared memory");

// Tensor memory columns.  P and dS, as packed pairs, take the place of the scores that they were
// made from, each warpgroup's in its own half (P its first, dS its second 32 columns).
//   dK/dV  two regions of 128 by turns: tile x has Sᵀ, then P and dS, in region x & 1, and dPᵀ in the
//          other, so Sᵀ of x + 1 (where dPᵀ of x was) waits only for dPᵀ to be loaded, and
//          dPᵀ of x + 1 for the gradients of x
//   dQ     S, then dS, in region x & 1; dP in a third
constexpr uint32_t kColV = 256, kColK = 384;    // dK/dV
constexpr uint32_t kColDp2 = 256, kColQ = 384;  // dQ
__device__ __forceinline__ uint32_t packed_col(int k) {  // 16 rows or keys from 16·k on
  return k < 4 ? k * 8 : 64 + (k - 4) * 8;
}

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

// ------------------------------------------------------------ producer (one thread)
template <int DP, bool DKV>
__device__ __forceinline__ void producer(const SeqBwdArgs& a, uint8_t* base, Bars* bars, const WaitGuard& g) {
  using L = Layout<DP>;
  constexpr int kHalves = DP / 64;
  const uint32_t qbytes = static_cast<uint32_t>(a.TQ * a.s.group) * 128u * kHalves;
  uint32_t n = 0, it = 0, own = 0, na = 0, nb = 0;
  auto queries = [&](uint32_t dst, const CUtensorMap* m, uint32_t bar, const Work& w, int token) {
    for (int h = 0; h < kHalves; ++h) tma_load_4d(dst + h * L::kHalf, m, bar, h * 64, 0, w.kvh, w.row0 + token);
  };
  auto keys = [&](uint32_t dst, const CUtensorMap* m, uint32_t bar, const Work& w, int token) {
    for (int h = 0; h < kHalves; ++h) tma_load_3d(dst + h * L::kHalf, m, bar, h * 64, w.kvh, w.row0 + token);
  };
  Work w;
  bool ok = true;
  for (; ok && take<false>(bars, it, g, w); ++it) {
    give_back(bars, it);
    for (int j = w.j0; j < w.j1; ++j, ++n) {
      const uint32_t as = n % kASlots, bs = n % kBSlots;
      if (!mbar_wait_inl(smem_u32(&bars->a_empty[as]), ((n / kASlots) & 1) ^ 1, g)) { ok = false; break; }
      uint32_t bar = smem_u32(&bars->a_full[as]), dst = smem_u32(base + L::a + as * L::kTB);
      mbar_arrive_expect_tx(bar, DKV ? qbytes : L::kTB);
      if (DKV)
        queries(dst, &a.tq, bar, w, j * a.TQ);
      else
        keys(dst, &a.tk, bar, w, j * kTile);
      ++na;
      if (j == w.j0) {  // the item's own tiles, behind the first streamed one
        if (!mbar_wait_inl(smem_u32(&bars->own_empty), (it & 1) ^ 1, g)) { ok = false; break; }
        bar = smem_u32(&bars->own_full), dst = smem_u32(base + L::own);
        mbar_arrive_expect_tx(bar, 2 * (DKV ? L::kTB : qbytes));
        if (DKV) {
          keys(dst, &a.tk, bar, w, w.t0);
          keys(dst + L::kTB, &a.tv, bar, w, w.t0);
        } else {
          queries(dst, &a.tq, bar, w, w.t0);
          queries(dst + L::kTB, &a.tdo, bar, w, w.t0);
        }
        ++own;
      }
      if (!mbar_wait_inl(smem_u32(&bars->b_empty[bs]), ((n / kBSlots) & 1) ^ 1, g)) { ok = false; break; }
      bar = smem_u32(&bars->b_full[bs]), dst = smem_u32(base + L::b + bs * L::kTB);
      mbar_arrive_expect_tx(bar, DKV ? qbytes : L::kTB);
      if (DKV)
        queries(dst, &a.tdo, bar, w, j * a.TQ);
      else
        keys(dst, &a.tv, bar, w, j * kTile);
      ++nb;
    }
  }
  bars->loads_a = na, bars->loads_b = nb, bars->loads_own = own;
}

// ------------------------------------------------------------ the walk, and the streamed tiles' release
// Rows of a streamed tile that belong to no token of the sequence are cleared: they are
// multiplied by P or dS of 0, and 0 times a NaN of a neighbouring sequence would spread.
template <int DP, bool DKV>
__device__ __forceinline__ void walk(const SeqBwdArgs& a, uint8_t* base, Bars* bars, const WaitGuard& g, int lane) {
  using L = Layout<DP>;
  Walk<typename std::conditional<DKV, KeyBlocks, QueryBlocks>::type> walk;
  if constexpr (DKV)
    walk.init(a.s, KeyBlocks{a.TQ}, blockIdx.x, gridDim.x);
  else
    walk.init(a.s, QueryBlocks{a.TQ}, blockIdx.x, gridDim.x);
  PieceRecord* rec = a.records + 2 * (blockIdx.x + (DKV ? 0 : gridDim.x));
  Work cur, ahead;
  uint32_t pub = 0, n = 0;
  bool more = true;
  auto publish = [&](Work& w) -> bool {
    w = walk.next();
    const uint32_t s = pub % kDescs;
    if (!mbar_wait_warp_inl(smem_u32(&bars->desc_empty[s]), ((pub / kDescs) & 1) ^ 1, g)) return false;
    if (lane == 0) {
      bars->work[s] = w;
      if (!w.stop && w.slot >= 0) rec[w.slot] = PieceRecord{1, w.j1 == w.kt, w.b, w.kvh, w.row0, w.t0, w.nt, 0};
      mbar_arrive(smem_u32(&bars->desc_full[s]));
    }
    ++pub;
    more = !w.stop;
    return true;
  };
  auto clear = [&](uint8_t* tile, int from) {
    for (int i = from * (DP / 8) + lane; i < kTile * (DP / 8); i += 32) {
      const int r = i / (DP / 8), c = i % (DP / 8);
      *reinterpret_cast<uint4*>(tile + (c >> 3) * L::kHalf + r * 128 + (c & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
    }
  };
  if (!publish(cur)) return;
  while (!cur.stop) {
    ahead.stop = 1;
    if (more && !publish(ahead)) return;
    for (int j = cur.j0; j < cur.j1; ++j, ++n) {
      const uint32_t as = n % kASlots, bs = n % kBSlots;
      if (!mbar_wait_warp_inl(smem_u32(&bars->a_full[as]), (n / kASlots) & 1, g)) return;
      if (!mbar_wait_warp_inl(smem_u32(&bars->b_full[bs]), (n / kBSlots) & 1, g)) return;
      const int last = DKV ? tile_rows(cur.kv_end - j * a.TQ, a.TQ, a.s.group) : cur.kv_end - j * kTile;  // rows in the sequence
      if (last < (DKV ? a.TQ * a.s.group : kTile)) {
        clear(base + L::a + as * L::kTB, last);
        if (DKV) clear(base + L::b + bs * L::kTB, last);  // (V's rows only reach masked entries of dP)
        fence_proxy_async_smem();
        __syncwarp();
      }
      if (lane == 0) mbar_arrive(smem_u32(&bars->ready[n % kReady]));
    }
    cur = ahead;
  }
}

// ------------------------------------------------------------ dK, dV: (lse, delta) of each tile of queries
// (per stage 128 of -lse·log2 e, then 128 of -delta)
__device__ __forceinline__ void rows(const SeqBwdArgs& a, float* buf, Bars* bars, const WaitGuard& g, int lane) {
  const SeqDesc& s = a.s;
  int dt[4], head[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) dt[e] = (lane + 32 * e) / s.group, head[e] = (lane + 32 * e) % s.group;
  uint32_t n = 0;
  Work w;
  for (uint32_t it = 0; take<true>(bars, it, g, w); ++it) {
    __syncwarp();
    if (lane == 0) give_back(bars, it);
    for (int j = w.j0; j < w.j1; ++j, ++n) {
      float2 x[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int t = j * a.TQ + dt[e];
        x[e] = make_float2(-INFINITY, 0.0f);  // P = 0
        if (dt[e] < a.TQ && t < w.kv_end)
          x[e] = a.rows[static_cast<size_t>(w.row0 + t) * s.q_heads + w.kvh * s.group + head[e]];
      }
      const uint32_t st = n & 1;
      if (!mbar_wait_warp_inl(smem_u32(&bars->rows_empty[st]), ((n >> 1) & 1) ^ 1, g)) return;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        buf[st * 2 * kTile + lane + 32 * e] = x[e].x;
        buf[st * 2 * kTile + kTile + lane + 32 * e] = x[e].y;
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&bars->rows_full[st]));
    }
  }
}

// ------------------------------------------------------------ MMA (one warp, one of its threads issuing)
template <int DP>
__device__ __forceinline__ uint64_t k_step(int k) {  // 16 features further in a tile, in descriptor units
  return (k & 3) * 2 + (k >> 2) * (Layout<DP>::kHalf / 16);
}
// D = A Bᵀ over the features: two tiles of 128 rows.
template <int DP>
__device__ __forceinline__ void scores(uint32_t d, uint32_t a, uint32_t b, int steps, uint32_t id) {
  const uint64_t ad = smem_desc(a, 16, 1024, kSwizzle128B), bd = smem_desc(b, 16, 1024, kSwizzle128B);
#pragma unroll
  for (int k = 0; k < DP / 16; ++k)
    if (k < steps) umma_ss(d, ad + k_step<DP>(k), bd + k_step<DP>(k), id, k > 0);
}
// D (+)= A B over 128 rows or keys, A packed in tensor memory, B a tile (features along N).
template <int DP>
__device__ __forceinline__ void gather(uint32_t d, uint32_t a, uint32_t b, uint32_t id, bool add) {
  const uint64_t bd = smem_desc(b, Layout<DP>::kHalf, 1024, kSwizzle128B);
#pragma unroll
  for (int k = 0; k < 8; ++k) umma_ts(d, a + packed_col(k), bd + k * (2048 / 16), id, (add || k > 0) ? 1u : 0u);
}

template <int DP, bool BF16>
__device__ __forceinline__ void mma_dkv(const SeqBwdArgs& a, uint8_t* base, Bars* bars, uint32_t tmem, const WaitGuard& g) {
  using L = Layout<DP>;
  const int steps = (a.s.D + 15) / 16;
  const uint32_t id_s = idesc_f16(128, 128, BF16, false, false), id_g = idesc_f16(128, steps * 16, BF16, false, true);
  const uint32_t ks = smem_u32(base + L::own), vs = ks + L::kTB;
  uint32_t n = 0, it = 0;
  bool ok = true;
  // Sᵀ of streamed tile x, and dPᵀ
  auto issue_s = [&](uint32_t x) -> bool {
    if (!mbar_wait_warp_inl(smem_u32(&bars->ready[x % kReady]), (x / kReady) & 1, g)) return false;
    if (!mbar_wait_warp_inl(smem_u32(&bars->a_full[x % kASlots]), (x / kASlots) & 1, g)) return false;
    if (x > 0 && !mbar_wait_warp_inl(smem_u32(&bars->dp_free), (x - 1) & 1, g)) return false;
    tc_fence_after();
    if (elect_one()) {
      scores<DP>(tmem + (x & 1) * 128, ks, smem_u32(base + L::a + (x % kASlots) * L::kTB), steps, id_s);
      umma_commit(smem_u32(&bars->s_full[0]));
    }
    __syncwarp();
    return true;
  };
  auto issue_dp = [&](uint32_t x) -> bool {
    if (!mbar_wait_warp_inl(smem_u32(&bars->b_full[x % kBSlots]), (x / kBSlots) & 1, g)) return false;
    if (x > 0 && !mbar_wait_warp_inl(smem_u32(&bars->second_done), (x - 1) & 1, g)) return false;
    tc_fence_after();
    if (elect_one()) {
      scores<DP>(tmem + (~x & 1) * 128, vs, smem_u32(base + L::b + (x % kBSlots) * L::kTB), steps, id_s);
      umma_commit(smem_u32(&bars->dp_full));
    }
    __syncwarp();
    return true;
  };
  Work w;
  for (; ok && take<true>(bars, it, g, w); ++it) {
    __syncwarp();
    if (elect_one()) give_back(bars, it);
    const int j0 = uniform(w.j0), j1 = uniform(w.j1);
    if (!mbar_wait_warp_inl(smem_u32(&bars->own_full), it & 1, g)) break;
    if (!issue_s(n) || !issue_dp(n)) break;
    for (int j = j0; j < j1; ++j, ++n) {
      const uint32_t as = n % kASlots, bs = n % kBSlots;
      if (!mbar_wait_warp_inl(smem_u32(&bars->p_ready), n & 1, g)) { ok = false; break; }
      if (j == j0 && !mbar_wait_warp_inl(smem_u32(&bars->acc_free), (it & 1) ^ 1, g)) { ok = false; break; }
      tc_fence_after();
      if (elect_one()) {
        gather<DP>(tmem + kColV, tmem + (n & 1) * 128, smem_u32(base + L::b + bs * L::kTB), id_g, j > j0);
        umma_commit(smem_u32(&bars->b_empty[bs]));
      }
      __syncwarp();
      if (j + 1 < j1 && !issue_s(n + 1)) { ok = false; break; }
      if (!mbar_wait_warp_inl(smem_u32(&bars->ds_ready[0]), n & 1, g)) { ok = false; break; }
      tc_fence_after();
      if (elect_one()) {
        gather<DP>(tmem + kColK, tmem + (n & 1) * 128 + 32, smem_u32(base + L::a + as * L::kTB), id_g, j > j0);
        umma_commit(smem_u32(&bars->second_done));
        umma_commit(smem_u32(&bars->a_empty[as]));
      }
      __syncwarp();
      if (j + 1 < j1 && !issue_dp(n + 1)) { ok = false; break; }
    }
    if (elect_one()) {
      umma_commit(smem_u32(&bars->own_empty));
      umma_commit(smem_u32(&bars->acc_full));
    }
    __syncwarp();
  }
  __syncwarp();
  if (elect_one()) umma_commit(smem_u32(&bars->drain));
}

template <int DP, bool BF16>
__device__ __forceinline__ void mma_dq(const SeqBwdArgs& a, uint8_t* base, Bars* bars, uint32_t tmem, const WaitGuard& g) {
  using L = Layout<DP>;
  const int steps = (a.s.D + 15) / 16;
  const uint32_t id_s = idesc_f16(128, 128, BF16, false, false), id_g = idesc_f16(128, steps * 16, BF16, false, true);
  const uint32_t qs = smem_u32(base + L::own), dos = qs + L::kTB;
  uint32_t n = 0, it = 0;
  bool ok = true;
  uint32_t gathers = 0;  // issued
  auto issue_s = [&](uint32_t x) -> bool {
    if (!mbar_wait_warp_inl(smem_u32(&bars->ready[x % kReady]), (x / kReady) & 1, g)) return false;
    if (!mbar_wait_warp_inl(smem_u32(&bars->a_full[x % kASlots]), (x / kASlots) & 1, g)) return false;
    // its buffer held dS of tile x - 2.  The wait is for the newest gather issued (a parity
    // says nothing about an older phase): x - 2's within an item, x - 1's at an item's start
    if (gathers > 0 && !mbar_wait_warp_inl(smem_u32(&bars->second_done), (gathers - 1) & 1, g)) return false;
    tc_fence_after();
    if (elect_one()) {
      scores<DP>(tmem + (x & 1) * 128, qs, smem_u32(base + L::a + (x % kASlots) * L::kTB), steps, id_s);
      umma_commit(smem_u32(&bars->s_full[x & 1]));
    }
    __syncwarp();
    return true;
  };
  auto issue_dp = [&](uint32_t x) -> bool {
    if (!mbar_wait_warp_inl(smem_u32(&bars->b_full[x % kBSlots]), (x / kBSlots) & 1, g)) return false;
    if (x > 0 && !mbar_wait_warp_inl(smem_u32(&bars->dp_free), (x - 1) & 1, g)) return false;
    tc_fence_after();
    if (elect_one()) {
      scores<DP>(tmem + kColDp2, dos, smem_u32(base + L::b + (x % kBSlots) * L::kTB), steps, id_s);
      umma_commit(smem_u32(&bars->dp_full));
      umma_commit(smem_u32(&bars->b_empty[x % kBSlots]));
    }
    __syncwarp();
    return true;
  };
  Work w;
  for (; ok && take<true>(bars, it, g, w); ++it) {
    __syncwarp();
    if (elect_one()) give_back(bars, it);
    const int j0 = uniform(w.j0), j1 = uniform(w.j1);
    if (!mbar_wait_warp_inl(smem_u32(&bars->own_full), it & 1, g)) break;
    if (!issue_s(n) || !issue_dp(n)) break;
    for (int j = j0; j < j1; ++j, ++n) {
      const uint32_t as = n % kASlots;
      if (j + 1 < j1 && (!issue_s(n + 1) || !issue_dp(n + 1))) { ok = false; break; }
      // Two barriers by turns: S and dP of tile n + 1 are on their way already, so that its dS may be
      // complete before this warp has looked for dS of n, and a wait by parity would miss a phase
      // that the next one has passed.  With two, the compute warps need S of n + 2 first, issued behind this.
      if (!mbar_wait_warp_inl(smem_u32(&bars->ds_ready[n & 1]), (n >> 1) & 1, g)) { ok = false; break; }
      if (j == j0 && !mbar_wait_warp_inl(smem_u32(&bars->acc_free), (it & 1) ^ 1, g)) { ok = false; break; }
      tc_fence_after();
      if (elect_one()) {
        gather<DP>(tmem + kColQ, tmem + (n & 1) * 128, smem_u32(base + L::a + as * L::kTB), id_g, j > j0);
        umma_commit(smem_u32(&bars->second_done));
        umma_commit(smem_u32(&bars->a_empty[as]));
      }
      __syncwarp();
      ++gathers;
    }
    if (elect_one()) {
      umma_commit(smem_u32(&bars->own_empty));
      umma_commit(smem_u32(&bars->acc_full));
    }
    __syncwarp();
  }
  __syncwarp();
  if (elect_one()) umma_commit(smem_u32(&bars->drain));
}

// ------------------------------------------------------------ compute (warps 0..7)
// Columns [c0, c1) (N at a time; stops at D) of this thread's row of an accumulator: times f in the
// result's type at `out`, or as they are at `part`.  Warp-collective.
template <int N, bool BF16>
__device__ __forceinline__ void write_row(uint32_t col, int c0, int c1, int D, bool live, bool piece, float f, uint16_t* out,
                                          bool out32, float* part) {
#pragma unroll 1
  for (int c = c0; c < c1 && c < D; c += N) {
    uint32_t x[N];
    if constexpr (N == 64) {
      tmem_ld64(col + c, x);
    } else {
      tmem_ld32(col + c, x);
    }
    tmem_wait_ld(x);
    if (live) {
      if (piece) {
#pragma unroll
        for (int e = 0; e < N; e += 8) {
          const uint32_t(&o)[8] = *reinterpret_cast<const uint32_t(*)[8]>(&x[e]);
          st_global_32(part + c + e, o);
        }
      } else {
#pragma unroll
        for (int e = 0; e < N; e += 16) {
          uint32_t o[8];
#pragma unroll
          for (int i = 0; i < 8; ++i)
            o[i] = pack2<BF16>(__uint_as_float(x[e + 2 * i]) * f, __uint_as_float(x[e + 2 * i + 1]) * f);
          if (out32) {
            if (c + e < D) st_global_32(out + c + e, o);
          } else {
            if (c + e < D) *reinterpret_cast<uint4*>(out + c + e) = make_uint4(o[0], o[1], o[2], o[3]);
            if (c + e + 8 < D) *reinterpret_cast<uint4*>(out + c + e + 8) = make_uint4(o[4], o[5], o[6], o[7]);
          }
        }
      }
    }
    __syncwarp();
  }
}

// P = 2^(S·s + nl) of 64 scores in place, nl (-lse·log2 e) per column, and packed; columns below
// `from` do not see the key.
template <bool BF16, bool MASK>
__device__ __forceinline__ void probs(uint32_t (&p)[64], uint32_t (&pp)[32], float2 sl2, const float4* nl, int from) {
#pragma unroll
  for (int x = 0; x < 64; x += 4) {
    const float4 z = nl[x >> 2];
    const float2 t0 = fma2(make_float2(__uint_as_float(p[x]), __uint_as_float(p[x + 1])), sl2, make_float2(z.x, z.y));
    const float2 t1 = fma2(make_float2(__uint_as_float(p[x + 2]), __uint_as_float(p[x + 3])), sl2, make_float2(z.z, z.w));
    float e[4] = {ex2(t0.x), ex2(t0.y), ex2(t1.x), ex2(t1.y)};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (MASK && x + i < from) e[i] = 0.0f;
      p[x + i] = __float_as_uint(e[i]);
    }
    pp[x >> 1] = pack2<BF16>(e[0], e[1]);
    pp[(x >> 1) + 1] = pack2<BF16>(e[2], e[3]);
  }
}
// dS = P (dP + nd) of 64 columns, packed; nd (-delta) per column.
template <bool BF16, bool MASK>
__device__ __forceinline__ void dscores(const uint32_t (&d)[64], const uint32_t (&p)[64], uint32_t (&pp)[32], const float4* nd,
                                        int from) {
#pragma unroll
  for (int x = 0; x < 64; x += 4) {
    const float4 z = nd[x >> 2];
    float2 s0 = mul2(add2(make_float2(__uint_as_float(d[x]), __uint_as_float(d[x + 1])), make_float2(z.x, z.y)),
                     make_float2(__uint_as_float(p[x]), __uint_as_float(p[x + 1])));
    float2 s1 = mul2(add2(make_float2(__uint_as_float(d[x + 2]), __uint_as_float(d[x + 3])), make_float2(z.z, z.w)),
                     make_float2(__uint_as_float(p[x + 2]), __uint_as_float(p[x + 3])));
    if (MASK) {
      if (x < from) s0.x = 0.0f;
      if (x + 1 < from) s0.y = 0.0f;
      if (x + 2 < from) s1.x = 0.0f;
      if (x + 3 < from) s1.y = 0.0f;
    }
    pp[x >> 1] = pack2<BF16>(s0.x, s0.y);
    pp[(x >> 1) + 1] = pack2<BF16>(s1.x, s1.y);
  }
}
// The same with one row's delta; columns past `lim` are not seen.
template <bool BF16, bool MASK>
__device__ __forceinline__ void dscores_row(const uint32_t (&d)[64], const uint32_t (&p)[64], uint32_t (&pp)[32], float2 nd,
                                            int lim) {
#pragma unroll
  for (int x = 0; x < 64; x += 2) {
    float2 ds = mul2(add2(make_float2(__uint_as_float(d[x]), __uint_as_float(d[x + 1])), nd),
                     make_float2(__uint_as_float(p[x]), __uint_as_float(p[x + 1])));
    if (MASK) {
      if (x > lim) ds.x = 0.0f;
      if (x + 1 > lim) ds.y = 0.0f;
    }
    pp[x >> 1] = pack2<BF16>(ds.x, ds.y);
  }
}

// dK, dV.  Thread: key r of the tile, rows 64·grp .. 64·grp + 63 of each tile of queries.
template <int DP, bool BF16>
__device__ __forceinline__ void compute_dkv(const SeqBwdArgs& a, const float* rowbuf, Bars* bars, uint32_t tmem,
                                            const WaitGuard& g) {
  const SeqDesc& s = a.s;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int grp = warp >> 2, r = (warp & 3) * 32 + lane;
  const uint32_t trow = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
  const float2 sl2 = make_float2(a.scale_log2, a.scale_log2);
  uint32_t n = 0, it = 0;
  bool ok = true;
  Work w;
  for (; ok && take<true>(bars, it, g, w); ++it) {
    __syncwarp();
    if (lane == 0) give_back(bars, it);
    const int key = w.t0 + r;
    for (int j = w.j0; j < w.j1; ++j, ++n) {
      const uint32_t st = n & 1, scol = trow + st * 128 + grp * 64, dcol = trow + (st ^ 1) * 128 + grp * 64;
      const float4* nl = reinterpret_cast<const float4*>(rowbuf + st * 2 * kTile + grp * 64);
      const float4* nd = reinterpret_cast<const float4*>(rowbuf + st * 2 * kTile + kTile + grp * 64);
      // rows below `from` belong to tokens in front of the key; none does once the tile lies behind the keys
      const bool mask = j * a.TQ < w.t0 + kTile - 1;
      const int from = first_row(key - j * a.TQ, a.TQ, s.group) - grp * 64;
      uint32_t p[64];
      if (!mbar_wait_warp_inl(smem_u32(&bars->rows_full[st]), (n >> 1) & 1, g)) { ok = false; break; }
      if (!mbar_wait_warp_inl(smem_u32(&bars->s_full[0]), n & 1, g)) { ok = false; break; }
      tc_fence_after();
      tmem_ld64(scol, p);
      tmem_wait_ld(p);
      {
        uint32_t pp[32];
        if (mask)
          probs<BF16, true>(p, pp, sl2, nl, from);
        else
          probs<BF16, false>(p, pp, sl2, nl, 0);
        tmem_st32(scol, pp);
      }
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&bars->p_ready));
      if (!mbar_wait_warp_inl(smem_u32(&bars->dp_full), n & 1, g)) { ok = false; break; }
      tc_fence_after();
      {
        uint32_t d[64], pp[32];
        tmem_ld64(dcol, d);
        tmem_wait_ld(d);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&bars->dp_free));
        if (mask)
          dscores<BF16, true>(d, p, pp, nd, from);
        else
          dscores<BF16, false>(d, p, pp, nd, 0);
        tmem_st32(scol + 32, pp);
      }
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(smem_u32(&bars->ds_ready[0]));
        mbar_arrive(smem_u32(&bars->rows_empty[st]));
      }
    }
    if (!ok || !mbar_wait_warp_inl(smem_u32(&bars->acc_full), it & 1, g)) break;
    tc_fence_after();
    const bool live = r < w.nt;
    const size_t row = static_cast<size_t>(w.row0) + key;
    uint16_t* out = (grp ? a.dk + row * a.dk_stride : a.dv + row * a.dv_stride) + static_cast<size_t>(w.kvh) * s.D;
    float* part = a.part + (((static_cast<size_t>(blockIdx.x) * 2 + (w.slot > 0)) * 2 + grp) * kTile + r) * DP;
    write_row<64, BF16>(trow + (grp ? kColK : kColV), 0, DP, s.D, live, w.slot >= 0, grp ? a.scale : 1.0f, out,
                    grp ? a.dk32 : a.dv32, part);
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_u32(&bars->acc_free));
  }
}

// dQ.  Thread: row r of the tile, keys 64·grp .. 64·grp + 63 of each key tile.
template <int DP, bool BF16>
__device__ __forceinline__ void compute_dq(const SeqBwdArgs& a, Bars* bars, uint32_t tmem, const WaitGuard& g) {
  const SeqDesc& s = a.s;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int grp = warp >> 2, r = (warp & 3) * 32 + lane;
  const uint32_t trow = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
  const uint32_t dcol = trow + kColDp2 + grp * 64;
  const int dt = r / s.group, head = r % s.group;
  const float2 sl2 = make_float2(a.scale_log2, a.scale_log2);
  uint32_t n = 0, it = 0;
  bool ok = true;
  Work w;
  for (; ok && take<true>(bars, it, g, w); ++it) {
    __syncwarp();
    if (lane == 0) give_back(bars, it);
    const bool live = dt < a.TQ && dt < w.nt;
    const size_t row = static_cast<size_t>(w.row0) + w.t0 + dt;
    const int h = w.kvh * s.group + head;
    float2 z = make_float2(-INFINITY, 0.0f);
    if (live) z = a.rows[row * s.q_heads + h];
    const float2 nl = make_float2(z.x, z.x), nd = make_float2(z.y, z.y);
    for (int j = w.j0; j < w.j1; ++j, ++n) {
      const uint32_t scol = trow + (n & 1) * 128 + grp * 64;
      const bool mask = w.pos < j * kTile + kTile - 1;
      const int lim = w.pos + dt - j * kTile - grp * 64;  // keys past it are not seen
      uint32_t p[64];
      if (!mbar_wait_warp_inl(smem_u32(&bars->s_full[n & 1]), (n >> 1) & 1, g)) { ok = false; break; }
      tc_fence_after();
      tmem_ld64(scol, p);
      tmem_wait_ld(p);
#pragma unroll
      for (int x = 0; x < 64; x += 2) {
        const float2 t = fma2(make_float2(__uint_as_float(p[x]), __uint_as_float(p[x + 1])), sl2, nl);
        p[x] = __float_as_uint(ex2(t.x));
        p[x + 1] = __float_as_uint(ex2(t.y));
      }
      if (!mbar_wait_warp_inl(smem_u32(&bars->dp_full), n & 1, g)) { ok = false; break; }
      tc_fence_after();
      uint32_t d[64], pp[32];
      tmem_ld64(dcol, d);
      tmem_wait_ld(d);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&bars->dp_free));
      if (mask)
        dscores_row<BF16, true>(d, p, pp, nd, lim);
      else
        dscores_row<BF16, false>(d, p, pp, nd, 0);
      tmem_st32(scol, pp);
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&bars->ds_ready[n & 1]));
    }
    if (!ok || !mbar_wait_warp_inl(smem_u32(&bars->acc_full), it & 1, g)) break;
    tc_fence_after();
    uint16_t* out = a.dq + row * a.dq_stride + static_cast<size_t>(h) * s.D;
    float* part = a.part_q + ((static_cast<size_t>(blockIdx.x) * 2 + (w.slot > 0)) * kTile + r) * DP;
    write_row<DP / 2, BF16>(trow + kColQ, grp * (DP / 2), (grp + 1) * (DP / 2), s.D, live, w.slot >= 0, a.scale, out, a.dq32, part);
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_u32(&bars->acc_free));
  }
}

__device__ __forceinline__ void init_bars(Bars* bars, bool dkv) {
  for (int i = 0; i < kDescs; ++i) {
    mbar_init(smem_u32(&bars->desc_full[i]), 1);
    mbar_init(smem_u32(&bars->desc_empty[i]), dkv ? 11 : 10);  // producer, MMA, compute warps; rows
  }
  mbar_init(smem_u32(&bars->own_full), 1);
  mbar_init(smem_u32(&bars->own_empty), 1);
  for (int i = 0; i < kASlots; ++i) {
    mbar_init(smem_u32(&bars->a_full[i]), 1);
    mbar_init(smem_u32(&bars->a_empty[i]), 1);
  }
  for (int i = 0; i < kBSlots; ++i) {
    mbar_init(smem_u32(&bars->b_full[i]), 1);
    mbar_init(smem_u32(&bars->b_empty[i]), 1);
  }
  for (int i = 0; i < kReady; ++i) mbar_init(smem_u32(&bars->ready[i]), 1);
  for (int i = 0; i < 2; ++i) {
    mbar_init(smem_u32(&bars->rows_full[i]), 1);
    mbar_init(smem_u32(&bars->rows_empty[i]), 8);
    mbar_init(smem_u32(&bars->s_full[i]), 1);
    mbar_init(smem_u32(&bars->ds_ready[i]), 8);
  }
  mbar_init(smem_u32(&bars->dp_full), 1);
  mbar_init(smem_u32(&bars->p_ready), 8);
  mbar_init(smem_u32(&bars->dp_free), 8);
  mbar_init(smem_u32(&bars->second_done), 1);
  mbar_init(smem_u32(&bars->acc_full), 1);
  mbar_init(smem_u32(&bars->acc_free), 8);
  mbar_init(smem_u32(&bars->drain), 1);
  fence_barrier_init();
}

// By one warp, when every role has ended.  (Every tile that was loaded was let go by a commit; where the
// CTA gave up some were not.)
__device__ __forceinline__ void drain_all(Bars* bars, const WaitGuard& g) {
  const uint32_t all = *g.abort ? 0u : ~0u;
  const Owed owed[] = {{bars->a_full, kASlots, bars->loads_a},       {bars->b_full, kBSlots, bars->loads_b},
                       {&bars->own_full, 1, bars->loads_own},        {bars->a_empty, kASlots, bars->loads_a & all},
                       {&bars->second_done, 1, bars->loads_a & all}, {bars->b_empty, kBSlots, bars->loads_b & all},
                       {&bars->own_empty, 1, bars->loads_own & all}, {&bars->drain, 1, 1}};
  drain(owed, g);
}

// Between dK/dV and dQ, by every thread of the CTA: nothing is under way, so nobody uses a barrier any more,
// and all of them begin anew.  False where a wait ran out: something may then still be to come, and the
// CTA does no more.
template <bool COMPUTE>
__device__ __forceinline__ bool turn_over(Bars* bars, const WaitGuard& g) {
  tc_fence_before();
  __syncthreads();
  if (!COMPUTE && threadIdx.x >> 5 == kMmaWarp) {
    drain_all(bars, g);
    if ((threadIdx.x & 31) == 0) {
      bars->go = *g.abort == 0;  // (one word that does not change: `abort` may, as soon as the first warp goes on)
      if (bars->go) {
        uint64_t* bar = reinterpret_cast<uint64_t*>(bars);
        for (uint32_t i = 0; i < offsetof(Bars, work) / 8; ++i) mbar_inval(smem_u32(bar + i));
        init_bars(bars, false);
      }
    }
  }
  __syncthreads();
  tc_fence_after();
  return bars->go != 0;
}

template <int DP, bool BF16, bool DKV>
__device__ __forceinline__ void other_warps(const SeqBwdArgs& a, uint8_t* base, Bars* bars, uint32_t tmem, const WaitGuard& g,
                                            float* rowbuf, int warp, int lane) {
  if (warp == kProducerWarp) {
    if (lane == 0) producer<DP, DKV>(a, base, bars, g);
    __syncwarp();
  } else if (warp == kMmaWarp) {
    if (DKV)
      mma_dkv<DP, BF16>(a, base, bars, tmem, g);
    else
      mma_dq<DP, BF16>(a, base, bars, tmem, g);
  } else if (warp == kRowsWarp) {
    if (DKV) rows(a, rowbuf, bars, g, lane);
  } else {
    walk<DP, DKV>(a, base, bars, g, lane);
  }
}

// With one row of CTAs each does its share of dK/dV and then its share of dQ; with two rows the first
// does dK/dV and the second dQ at the same time (bwd_rows in evo_seq_host.cu says when).
template <int DP, bool BF16>
__global__ void __launch_bounds__(kThreads, 1) evo_seq_bwd_kernel(const __grid_constant__ SeqBwdArgs a) {
  using L = Layout<DP>;
  extern __shared__ __align__(1024) uint8_t base[];
  Bars* bars = reinterpret_cast<Bars*>(base + L::bars);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const bool both = gridDim.y == 1, dkv = blockIdx.y == 0;
  // no piece yet, in either phase: the join reads every record, those of a CTA that gave up too
  if (threadIdx.x < 4 && (both || (threadIdx.x < 2) == dkv))
    a.records[2 * (blockIdx.x + (threadIdx.x < 2 ? 0 : gridDim.x)) + (threadIdx.x & 1)].used = 0;
  if (smem_u32(base) & 1023u) {  // the tiles' swizzle counts from 1 KB borders
    if (threadIdx.x == 0) atomicExch(a.s.status, kStatusTimeout);
    return;
  }
  if (threadIdx.x == 0) {
    bars->abort = 0;
    init_bars(bars, dkv);
  }
  if (warp == kProducerWarp && lane == 0) {
    tma_prefetch_desc(&a.tq);
    tma_prefetch_desc(&a.tk);
    tma_prefetch_desc(&a.tv);
    tma_prefetch_desc(&a.tdo);
  }
  if (warp == kMmaWarp) {
    tmem_alloc(smem_u32(&bars->tmem_slot), 512);
    tmem_relinquish();
  }
  if (dkv && a.TQ * a.s.group < kTile) {
    // rows that no query tile fills are read by the gradient MMAs (against P = dS = 0)
    for (uint32_t i = threadIdx.x; i < (kASlots + kBSlots) * L::kTB / 16; i += kThreads)
      reinterpret_cast<uint4*>(base + L::a)[i] = make_uint4(0u, 0u, 0u, 0u);
    fence_proxy_async_smem();
  }
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bars->tmem_slot;
  const WaitGuard g{a.wait_ns, a.s.status, &bars->abort};
  float* rowbuf = reinterpret_cast<float*>(base + L::rows);
  if (warp >= kProducerWarp) {
    setmaxnreg_dec<kRegsOther>();
    if (dkv) other_warps<DP, BF16, true>(a, base, bars, tmem, g, rowbuf, warp, lane);
    if (both ? turn_over<false>(bars, g) : !dkv) other_warps<DP, BF16, false>(a, base, bars, tmem, g, rowbuf, warp, lane);
    tc_fence_before();
    __syncthreads();
    if (warp == kMmaWarp) {
      drain_all(bars, g);
      tc_fence_after();
      tmem_dealloc(tmem, 512);
    }
  } else {
    setmaxnreg_inc<kRegsCompute>();
    if (dkv) compute_dkv<DP, BF16>(a, rowbuf, bars, tmem, g);
    if (both ? turn_over<true>(bars, g) : !dkv) compute_dq<DP, BF16>(a, bars, tmem, g);
    tc_fence_before();
    __syncthreads();
  }
}

// ------------------------------------------------------------ pieces, summed in order
// Eight threads a row, 32 rows a block.
constexpr int kJoinRows = 32;
template <int DP, bool BF16, bool DKV>
__device__ __forceinline__ void join(const SeqBwdArgs& a, int ctas, int block) {
  constexpr int kParts = DKV ? 2 : 1;
  const int c0 = blockIdx.x, i = block * kJoinRows + (threadIdx.x >> 3), d0 = (threadIdx.x & 7) * (DP / 8);
  const PieceRecord* records = a.records + (DKV ? 0 : 2 * ctas);
  const PieceRecord first = records[2 * c0 + 1];
  if (!first.used) return;
  const int pieces = count_pieces(records, c0, ctas);
  const SeqDesc& s = a.s;
  const int part = i / kTile, r = i % kTile;
  const int tok = DKV ? r : r / s.group;
  if (tok >= first.nt || (!DKV && tok >= a.TQ)) return;
  float x[DP / 8] = {};
  for (int p = 0; p < pieces; ++p) {
    const float4* y = reinterpret_cast<const float4*>(
        (DKV ? a.part : a.part_q) + (((static_cast<size_t>(c0 + p) * 2 + (p == 0)) * kParts + part) * kTile + r) * DP + d0);
#pragma unroll
    for (int e = 0; e < DP / 32; ++e) {
      const float4 v = y[e];
      x[4 * e] += v.x, x[4 * e + 1] += v.y, x[4 * e + 2] += v.z, x[4 * e + 3] += v.w;
    }
  }
  const size_t row = static_cast<size_t>(first.row0) + first.t0 + tok;
  uint16_t* out = DKV ? (part ? a.dk + row * a.dk_stride : a.dv + row * a.dv_stride) + static_cast<size_t>(first.kvh) * s.D
                      : a.dq + row * a.dq_stride + static_cast<size_t>(first.kvh * s.group + r % s.group) * s.D;
  const float f = DKV && part == 0 ? 1.0f : a.scale;
#pragma unroll
  for (int e = 0; e < DP / 8; e += 8) {  // (columns past D hold nothing and are not written)
    uint32_t v[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) v[q] = pack2<BF16>(x[e + 2 * q] * f, x[e + 2 * q + 1] * f);
    if (d0 + e < s.D) *reinterpret_cast<uint4*>(out + d0 + e) = make_uint4(v[0], v[1], v[2], v[3]);
  }
}

template <int DP, bool BF16>
__global__ void __launch_bounds__(256) evo_seq_bwd_join_kernel(const __grid_constant__ SeqBwdArgs a, int ctas) {
  constexpr int kBlocks = 2 * kTile / kJoinRows;  // dK and dV's
  if (blockIdx.y < kBlocks)
    join<DP, BF16, true>(a, ctas, blockIdx.y);
  else
    join<DP, BF16, false>(a, ctas, blockIdx.y - kBlocks);
}

// ------------------------------------------------------------ lse and delta
// 16 threads per (row, head), 16 bytes of O and of dO each, four (row, head)s one behind the other
// so that eight loads are under way.  Bound by those bytes.
constexpr int kRowsPer = 4;
template <bool BF16>
__global__ void __launch_bounds__(256) evo_seq_rows_kernel(const __grid_constant__ SeqBwdArgs a) {
  const SeqDesc& s = a.s;
  const int c = threadIdx.x & 15;
  const long long first = static_cast<long long>(blockIdx.x) * (16 * kRowsPer) + (threadIdx.x >> 4);
  const long long end = static_cast<long long>(s.tokens) * s.q_heads;
  uint4 x[kRowsPer], y[kRowsPer];
  float z[kRowsPer];
#pragma unroll
  for (int e = 0; e < kRowsPer; ++e) {
    const long long i = first + 16 * e;
    x[e] = y[e] = make_uint4(0u, 0u, 0u, 0u);
    z[e] = 0.0f;
    if (i >= end) continue;
    const int t = static_cast<int>(i / s.q_heads), h = static_cast<int>(i % s.q_heads);
    if (c * 8 < s.D) {
      x[e] = *reinterpret_cast<const uint4*>(a.out + t * a.out_stride + static_cast<long long>(h) * s.D + c * 8);
      y[e] = *reinterpret_cast<const uint4*>(a.dout + t * a.dout_stride + static_cast<long long>(h) * s.D + c * 8);
    }
    if (c == 0) z[e] = a.lse[static_cast<size_t>(h) * s.tokens + t];
  }
#pragma unroll
  for (int e = 0; e < kRowsPer; ++e) {
    const uint32_t xs[4] = {x[e].x, x[e].y, x[e].z, x[e].w}, ys[4] = {y[e].x, y[e].y, y[e].z, y[e].w};
    float d = 0.0f;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const float2 u = unpack2<BF16>(xs[q]), v = unpack2<BF16>(ys[q]);
      d = fmaf(u.x, v.x, d);
      d = fmaf(u.y, v.y, d);
    }
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) d += __shfl_xor_sync(0xffffffffu, d, o);
    const long long i = first + 16 * e;
    if (i < end && c == 0) a.rows[i] = make_float2(z[e] == -INFINITY ? -INFINITY : -z[e] * kSeqLog2e, -d);
  }
}

template <int DP, bool BF16>
cudaError_t launch_t(const SeqBwdArgs& a, int ctas, int rows, cudaStream_t st) {
  const long long n = static_cast<long long>(a.s.tokens) * a.s.q_heads;
  evo_seq_rows_kernel<BF16><<<static_cast<unsigned>((n + 16 * kRowsPer - 1) / (16 * kRowsPer)), 256, 0, st>>>(a);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  auto kern = evo_seq_bwd_kernel<DP, BF16>;
  static bool limit_set[64] = {};
  if ((e = ensure_smem_limit(kern, 232448, limit_set)) != cudaSuccess) return e;
  // more than half of an SM's shared memory: each CTA allocates all of tensor memory
  const size_t smem = Layout<DP>::total > 118784 ? Layout<DP>::total : 118784;
  kern<<<dim3(ctas, rows), kThreads, smem, st>>>(a);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  if (a.s.tokens <= a.TQ) return e;  // items of one tile: nothing is cut
  evo_seq_bwd_join_kernel<DP, BF16><<<dim3(ctas, 3 * kTile / kJoinRows), 256, 0, st>>>(a, ctas);
  return cudaGetLastError();
}

}  // namespace

size_t prompt_bwd_workspace(int ctas, const SeqDesc& s, SeqBwdArgs* a, uint8_t* ws) {
  const int DP = s.D <= 64 ? 64 : 128;
  size_t off = 0;
  auto take = [&](size_t bytes) {
    uint8_t* p = ws ? ws + off : nullptr;
    off += (bytes + 255) & ~size_t(255);
    return p;
  };
  uint8_t* rec = take(size_t(ctas) * 2 * 2 * sizeof(PieceRecord));
  uint8_t* rows = take(size_t(s.tokens) * s.q_heads * sizeof(float2));
  uint8_t* part = take(size_t(ctas) * 2 * 2 * kTile * DP * sizeof(float));
  uint8_t* part_q = take(size_t(ctas) * 2 * kTile * DP * sizeof(float));
  if (a) {
    a->records = reinterpret_cast<PieceRecord*>(rec);
    a->rows = reinterpret_cast<float2*>(rows);
    a->part = reinterpret_cast<float*>(part);
    a->part_q = reinterpret_cast<float*>(part_q);
  }
  return off;
}

cudaError_t launch_prompt_bwd(const SeqBwdArgs& a, int ctas, int rows, bool bf16, cudaStream_t st) {
  if (a.s.D <= 64) return bf16 ? launch_t<64, true>(a, ctas, rows, st) : launch_t<64, false>(a, ctas, rows, st);
  return bf16 ? launch_t<128, true>(a, ctas, rows, st) : launch_t<128, false>(a, ctas, rows, st);
}

}  // namespace evo
