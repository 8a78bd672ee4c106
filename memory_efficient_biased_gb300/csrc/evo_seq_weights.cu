// evo_seq_weights.cu — the attention weight that every cached key received
// (include/evo_seq.h): weights[b][h][j] += Σ P_ij over a call's rows i and the heads of group h,
// with P = 2^(s·log2e·S - log2e·lse) from the lse that the forward wrote.
//
// Two ways, the host's choice (evo_seq_host.cu):
//   evo_scores_sum_kernel    few rows a key (single tokens): the forward left its scores behind,
//                            8 bytes a row and key to write and read, and this pass sums them
//   evo_seq_weights_kernel   many rows: the scores are formed again, Sᵀ = K Qᵀ (a thread per key,
//                            so a key's sum stays in one register), 2 head_dim bytes a key and
//                            half of the forward's products
// The second is the dK/dV kernel (evo_seq_bwd.cu) without its gradients: items are tiles of 128
// keys over the tiles of queries that see them, cut and joined alike.
#include "evo_seq_internal.h"
#include "evo_seq_sched.cuh"

namespace evo {
namespace {

constexpr int kThreads = 384;
constexpr int kProducerWarp = 8, kMmaWarp = 9, kRowsWarp = 10;  // and 11: the walk
constexpr int kDescs = 4, kSlots = 4;

struct Bars {
  uint64_t desc_full[kDescs], desc_empty[kDescs];
  uint64_t k_full[2], k_empty[2];
  uint64_t q_full[kSlots], q_empty[kSlots];
  uint64_t rows_full[2], rows_empty[2];
  uint64_t s_full[2], s_free[2];
  uint64_t half_full, half_free, drain;
  Work work[kDescs];
  float half[kTile];  // the second warpgroup's sums, one per key
  uint32_t loads, keys;  // tiles of queries and keys that the producer asked for
  uint32_t tmem_slot;
  int abort;
};

template <int DP>
struct Layout {
  static constexpr uint32_t kHalf = kTile * 128u, kTB = kTile * DP * 2u;
  static constexpr uint32_t k = 0, q = 2 * kTB, rows = q + kSlots * kTB, bars = rows + 2 * kTile * 4u;
  static constexpr uint32_t total = bars + ((sizeof(Bars) + 127) & ~127u);
};

// Tiles of 128 keys of a cache under the tiles of TQ query tokens that see them.
// Work: t0, nt the keys; pos the first new token's position; kv_end the new tokens.
struct CachedKeyBlocks {
  int TQ;
  __device__ __forceinline__ int cost() const { return 2 * TQ; }
  __device__ __forceinline__ int count(const Seq& q) const { return q.n > 0 ? (q.kv + kTile - 1) / kTile : 0; }
  __device__ __forceinline__ int unseen(const Seq& q, int p) const {  // new tokens in front of the keys
    return p * kTile > q.pos0 ? p * kTile - q.pos0 : 0;
  }
  __device__ __forceinline__ long long of(const Seq& q, int p) const { return q.n - unseen(q, p) + cost(); }
  __device__ __forceinline__ long long before(const Seq& q, int p) const {
    const long long whole = q.pos0 >= 0 ? q.pos0 / kTile + 1 : 0;  // blocks that every new token sees
    const long long x = p;
    if (x <= whole) return x * (q.n + cost());
    return x * cost() + whole * q.n + (x - whole) * q.kv - (kTile / 2) * (x * (x - 1) - whole * (whole - 1));
  }
  __device__ __forceinline__ void place(Work& w, const Seq& q, int p) const {
    w.t0 = p * kTile;
    w.nt = q.kv - w.t0 < kTile ? q.kv - w.t0 : kTile;
    w.pos = q.pos0;
    w.kv_end = q.n;
    w.kt = (q.n + TQ - 1) / TQ;
  }
  __device__ __forceinline__ int skipped(const Work& w) const { return w.t0 > w.pos ? w.t0 - w.pos : 0; }
  __device__ __forceinline__ int first(const Work& w) const { return skipped(w) / TQ; }
  __device__ __forceinline__ int tile(const Work& w, long long tokens) const {
    return static_cast<int>((skipped(w) + tokens) / TQ);
  }
};

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

template <int DP>
__device__ __forceinline__ void producer(const SeqWeightsArgs& a, uint8_t* base, Bars* bars, const WaitGuard& g, int lane) {
  using L = Layout<DP>;
  const SeqDesc& s = a.s;
  const int box = s.page < kTile ? s.page : kTile, boxes = kTile / box;
  const uint32_t qbytes = static_cast<uint32_t>(a.TQ * s.group) * 128u * (DP / 64);
  uint32_t n = 0, it = 0, keys = 0;
  bool ok = true;
  Work w;
  for (; ok && take<true>(bars, it, g, w); ++it) {
    __syncwarp();
    if (lane == 0) give_back(bars, it);
    int page = s.num_pages;  // a page past the keys, or a bad one, reads as zeros
    if (lane < boxes && w.t0 + lane * box < w.t0 + w.nt) {
      page = page_of(s, w.b, w.t0 + lane * box);
      if (page < 0) page = s.num_pages;
    }
    const uint32_t ks = it & 1;
    if (!mbar_wait_warp_inl(smem_u32(&bars->k_empty[ks]), ((it >> 1) & 1) ^ 1, g)) break;
    if (lane == 0) mbar_arrive_expect_tx(smem_u32(&bars->k_full[ks]), L::kTB);
    __syncwarp();
    if (lane < boxes)
      for (int h = 0; h < DP / 64; ++h)
        tma_load_4d(smem_u32(base + L::k + ks * L::kTB + h * L::kHalf + lane * box * 128), &a.tk,
                    smem_u32(&bars->k_full[ks]), h * 64, w.kvh, boxes == 1 ? w.t0 % s.page : 0, page);
    ++keys;
    for (int j = w.j0; j < w.j1; ++j, ++n) {
      const uint32_t st = n % kSlots;
      if (!mbar_wait_warp_inl(smem_u32(&bars->q_empty[st]), ((n / kSlots) & 1) ^ 1, g)) { ok = false; break; }
      if (lane == 0) {
        mbar_arrive_expect_tx(smem_u32(&bars->q_full[st]), qbytes);
        for (int h = 0; h < DP / 64; ++h)
          tma_load_4d(smem_u32(base + L::q + st * L::kTB + h * L::kHalf), &a.tq, smem_u32(&bars->q_full[st]), h * 64, 0,
                      w.kvh, w.row0 + j * a.TQ);
      }
    }
  }
  if (lane == 0) bars->loads = n, bars->keys = keys;
}

template <int DP, bool BF16>
__device__ __forceinline__ void mma(const SeqWeightsArgs& a, uint8_t* base, Bars* bars, uint32_t tmem, const WaitGuard& g) {
  using L = Layout<DP>;
  const int steps = (a.s.D + 15) / 16;
  const uint32_t id = idesc_f16(128, 128, BF16, false, false);
  uint32_t n = 0, it = 0;
  bool ok = true;
  Work w;
  for (; ok && take<true>(bars, it, g, w); ++it) {
    __syncwarp();
    if (elect_one()) give_back(bars, it);
    const int j0 = uniform(w.j0), j1 = uniform(w.j1);
    const uint32_t ks = it & 1;
    if (!mbar_wait_warp_inl(smem_u32(&bars->k_full[ks]), (it >> 1) & 1, g)) break;
    const uint64_t kd = smem_desc(smem_u32(base + L::k + ks * L::kTB), 16, 1024, kSwizzle128B);
    for (int j = j0; j < j1; ++j, ++n) {
      const uint32_t st = n % kSlots;
      if (!mbar_wait_warp_inl(smem_u32(&bars->q_full[st]), (n / kSlots) & 1, g)) { ok = false; break; }
      if (!mbar_wait_warp_inl(smem_u32(&bars->s_free[n & 1]), ((n >> 1) & 1) ^ 1, g)) { ok = false; break; }
      tc_fence_after();
      const uint64_t qd = smem_desc(smem_u32(base + L::q + st * L::kTB), 16, 1024, kSwizzle128B);
      if (elect_one()) {
#pragma unroll
        for (int k = 0; k < DP / 16; ++k) {
          const uint64_t o = (k & 3) * 2 + (k >> 2) * (L::kHalf / 16);
          if (k < steps) umma_ss(tmem + (n & 1) * 128, kd + o, qd + o, id, k > 0);
        }
        umma_commit(smem_u32(&bars->s_full[n & 1]));
        umma_commit(smem_u32(&bars->q_empty[st]));
      }
      __syncwarp();
    }
    __syncwarp();
    if (elect_one()) umma_commit(smem_u32(&bars->k_empty[ks]));
  }
  __syncwarp();
  if (elect_one()) umma_commit(smem_u32(&bars->drain));
}

// -log2e·lse of each tile of queries; -inf (P = 0) for a row that saw nothing, or nothing but -inf.
__device__ __forceinline__ void rows(const SeqWeightsArgs& a, float* buf, Bars* bars, const WaitGuard& g, int lane) {
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
      float x[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int t = j * a.TQ + dt[e];
        x[e] = -INFINITY;
        if (dt[e] < a.TQ && t < w.kv_end) {
          const float z = a.lse[static_cast<size_t>(w.kvh * s.group + head[e]) * s.tokens + w.row0 + t];
          if (z != -INFINITY) x[e] = -z * kSeqLog2e;
        }
      }
      const uint32_t st = n & 1;
      if (!mbar_wait_warp_inl(smem_u32(&bars->rows_empty[st]), ((n >> 1) & 1) ^ 1, g)) return;
#pragma unroll
      for (int e = 0; e < 4; ++e) buf[st * kTile + lane + 32 * e] = x[e];
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&bars->rows_full[st]));
    }
  }
}

__device__ __forceinline__ void walk(const SeqWeightsArgs& a, Bars* bars, const WaitGuard& g, int lane) {
  Walk<CachedKeyBlocks> walk;
  walk.init(a.s, CachedKeyBlocks{a.TQ}, blockIdx.x, gridDim.x);
  PieceRecord* rec = a.records + 2 * blockIdx.x;
  if (lane < 2) rec[lane].used = 0;
  __syncwarp();
  for (uint32_t pub = 0;; ++pub) {
    const Work w = walk.next();
    const uint32_t s = pub % kDescs;
    if (!mbar_wait_warp_inl(smem_u32(&bars->desc_empty[s]), ((pub / kDescs) & 1) ^ 1, g)) return;
    if (lane == 0) {
      bars->work[s] = w;
      if (!w.stop && w.slot >= 0) rec[w.slot] = PieceRecord{1, w.j1 == w.kt, w.b, w.kvh, w.row0, w.t0, w.nt, 0};
      mbar_arrive(smem_u32(&bars->desc_full[s]));
    }
    if (w.stop) return;
  }
}

// Σ 2^(S·s + nl) over 64 columns, nl (-lse·log2 e) per column, of those in [from, to).
template <bool MASK>
__device__ __forceinline__ void add_probs(const uint32_t (&y)[64], float2 sl2, const float4* nl, int from, int to,
                                          float2 (&acc)[2]) {
#pragma unroll
  for (int x = 0; x < 64; x += 4) {
    const float4 z = nl[x >> 2];
    const float2 t0 = fma2(make_float2(__uint_as_float(y[x]), __uint_as_float(y[x + 1])), sl2, make_float2(z.x, z.y));
    const float2 t1 = fma2(make_float2(__uint_as_float(y[x + 2]), __uint_as_float(y[x + 3])), sl2, make_float2(z.z, z.w));
    float2 p0 = make_float2(ex2(t0.x), ex2(t0.y)), p1 = make_float2(ex2(t1.x), ex2(t1.y));
    if (MASK) {
      if (x < from || x >= to) p0.x = 0.0f;
      if (x + 1 < from || x + 1 >= to) p0.y = 0.0f;
      if (x + 2 < from || x + 2 >= to) p1.x = 0.0f;
      if (x + 3 < from || x + 3 >= to) p1.y = 0.0f;
    }
    acc[0] = add2(acc[0], p0);
    acc[1] = add2(acc[1], p1);
  }
}

// Thread: key r of the tile, rows 64·grp .. 64·grp + 63 of each tile of queries.
__device__ __forceinline__ void compute(const SeqWeightsArgs& a, const float* rowbuf, Bars* bars, uint32_t tmem,
                                        const WaitGuard& g) {
  const SeqDesc& s = a.s;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int grp = warp >> 2, r = (warp & 3) * 32 + lane;
  const uint32_t trow = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + grp * 64;
  const float2 sl2 = make_float2(a.scale_log2, a.scale_log2);
  uint32_t n = 0, it = 0;
  bool ok = true;
  Work w;
  for (; ok && take<true>(bars, it, g, w); ++it) {
    __syncwarp();
    if (lane == 0) give_back(bars, it);
    const int key = w.t0 + r;
    float sum = 0.0f;
    for (int j = w.j0; j < w.j1; ++j, ++n) {
      const uint32_t st = n & 1;
      const float4* rb = reinterpret_cast<const float4*>(rowbuf + st * kTile + grp * 64);
      // rows [from, to) of this half belong to new tokens that see the key
      const int rows = tile_rows(w.kv_end - j * a.TQ, a.TQ, s.group);
      const int from = first_row(key - w.pos - j * a.TQ, a.TQ, s.group) - grp * 64, to = rows - grp * 64;
      const bool mask = rows < kTile || w.pos + j * a.TQ < w.t0 + kTile - 1;
      if (!mbar_wait_warp_inl(smem_u32(&bars->rows_full[st]), (n >> 1) & 1, g)) { ok = false; break; }
      if (!mbar_wait_warp_inl(smem_u32(&bars->s_full[st]), (n >> 1) & 1, g)) { ok = false; break; }
      tc_fence_after();
      uint32_t y[64];
      tmem_ld64(trow + st * 128, y);
      tmem_wait_ld(y);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&bars->s_free[st]));
      float2 acc[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
      if (mask)
        add_probs<true>(y, sl2, rb, from, to, acc);
      else
        add_probs<false>(y, sl2, rb, 0, 0, acc);
      sum += (acc[0].x + acc[0].y) + (acc[1].x + acc[1].y);
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&bars->rows_empty[st]));
    }
    if (!ok) break;
    if (grp == 1) {  // hand over to the first warpgroup
      if (!mbar_wait_warp_inl(smem_u32(&bars->half_free), (it & 1) ^ 1, g)) break;
      bars->half[r] = sum;
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&bars->half_full));
    } else {
      if (!mbar_wait_warp_inl(smem_u32(&bars->half_full), it & 1, g)) break;
      sum += bars->half[r];
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&bars->half_free));
      if (r < w.nt) {
        if (w.slot >= 0)
          a.part[(static_cast<size_t>(blockIdx.x) * 2 + w.slot) * kTile + r] = sum;
        else
          a.weights[(static_cast<size_t>(w.b) * s.kv_heads + w.kvh) * a.weights_len + key] += sum;
      }
    }
  }
}

template <int DP, bool BF16>
__global__ void __launch_bounds__(kThreads, 1) evo_seq_weights_kernel(const __grid_constant__ SeqWeightsArgs a) {
  using L = Layout<DP>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  Bars* bars = reinterpret_cast<Bars*>(base + L::bars);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    bars->abort = 0;
    for (int i = 0; i < kDescs; ++i) {
      mbar_init(smem_u32(&bars->desc_full[i]), 1);
      mbar_init(smem_u32(&bars->desc_empty[i]), 11);  // producer, MMA, rows, eight compute warps
    }
    for (int i = 0; i < kSlots; ++i) {
      mbar_init(smem_u32(&bars->q_full[i]), 1);
      mbar_init(smem_u32(&bars->q_empty[i]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&bars->k_full[i]), 1);
      mbar_init(smem_u32(&bars->k_empty[i]), 1);
      mbar_init(smem_u32(&bars->rows_full[i]), 1);
      mbar_init(smem_u32(&bars->rows_empty[i]), 8);
      mbar_init(smem_u32(&bars->s_full[i]), 1);
      mbar_init(smem_u32(&bars->s_free[i]), 8);
    }
    mbar_init(smem_u32(&bars->half_full), 4);
    mbar_init(smem_u32(&bars->half_free), 4);
    mbar_init(smem_u32(&bars->drain), 1);
    fence_barrier_init();
  }
  if (warp == kProducerWarp && lane == 0) {
    tma_prefetch_desc(&a.tq);
    tma_prefetch_desc(&a.tk);
  }
  if (warp == kMmaWarp) {
    tmem_alloc(smem_u32(&bars->tmem_slot), 256);
    tmem_relinquish();
  }
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bars->tmem_slot;
  const WaitGuard g{a.wait_ns, a.s.status, &bars->abort};
  float* rowbuf = reinterpret_cast<float*>(base + L::rows);
  if (warp == kProducerWarp) {
    producer<DP>(a, base, bars, g, lane);
  } else if (warp == kMmaWarp) {
    mma<DP, BF16>(a, base, bars, tmem, g);
  } else if (warp == kRowsWarp) {
    rows(a, rowbuf, bars, g, lane);
  } else if (warp > kRowsWarp) {
    walk(a, bars, g, lane);
  } else {
    compute(a, rowbuf, bars, tmem, g);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    const uint32_t all = bars->abort ? 0u : ~0u;  // (a CTA that gave up did not let go of every tile)
    const Owed owed[] = {{bars->q_full, kSlots, bars->loads},        {bars->k_full, 2, bars->keys},
                         {bars->q_empty, kSlots, bars->loads & all}, {bars->k_empty, 2, bars->keys & all},
                         {&bars->drain, 1, 1}};
    drain(owed, g);
    tc_fence_after();
    tmem_dealloc(tmem, 256);
  }
}

// The pieces of a cut item, added in order.
__global__ void __launch_bounds__(kTile) evo_seq_weights_join_kernel(const __grid_constant__ SeqWeightsArgs a, int ctas) {
  const int c0 = blockIdx.x, r = threadIdx.x;
  const PieceRecord first = a.records[2 * c0 + 1];
  const int pieces = count_pieces(a.records, c0, ctas);  // (read beside the first record)
  if (!first.used || r >= first.nt) return;
  float sum = a.part[(static_cast<size_t>(c0) * 2 + 1) * kTile + r];
#pragma unroll 4
  for (int p = 1; p < pieces; ++p) sum += a.part[static_cast<size_t>(c0 + p) * 2 * kTile + r];
  a.weights[(static_cast<size_t>(first.b) * a.s.kv_heads + first.kvh) * a.weights_len + first.t0 + r] += sum;
}

// From the scores that the forward left behind ([tokens][q_heads][ld], times s·log2 e): four keys a
// thread, rows in order.
__global__ void __launch_bounds__(256) evo_scores_sum_kernel(const __grid_constant__ SeqWeightsArgs a, int ctas) {
  const SeqDesc& s = a.s;
  const int crowded = a.records[2 * ctas].used;  // the forward's verdict
  const int hk = blockIdx.y, b = blockIdx.z;
  const Seq q = load_seq(s, b);
  const int key = (blockIdx.x * 256 + threadIdx.x) * 4;
  if (key >= q.kv || q.n == 0 || crowded) return;
  float sum[4] = {};
  // (a token at position p sees the keys up to p)
  for (int i = key > q.pos0 ? key - q.pos0 : 0; i < q.n; ++i) {
    const int seen = q.pos0 + i - key;  // of these keys, those 0 .. seen
    for (int g = 0; g < s.group; ++g) {
      const int h = hk * s.group + g;
      const size_t row = static_cast<size_t>(q.row0) + i;
      const float z = a.lse[static_cast<size_t>(h) * s.tokens + row] * kSeqLog2e;
      const float4 x = *reinterpret_cast<const float4*>(a.scores + (row * s.q_heads + h) * a.scores_ld + key);
      const float xs[4] = {x.x, x.y, x.z, x.w};
      // where every score that the row sees is -inf, it gives no weight (and -inf - z would be no number)
      const int last = z == -INFINITY ? -1 : seen;
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (e <= last) sum[e] += ex2(xs[e] - z);
    }
  }
  float* w = a.weights + (static_cast<size_t>(b) * s.kv_heads + hk) * a.weights_len + key;
#pragma unroll
  for (int e = 0; e < 4; ++e)
    if (key + e < q.kv) w[e] += sum[e];
}

template <int DP, bool BF16>
cudaError_t launch_t(const SeqWeightsArgs& a, int ctas, cudaStream_t st) {
  auto kern = evo_seq_weights_kernel<DP, BF16>;
  static bool limit_set[64] = {};
  cudaError_t e = ensure_smem_limit(kern, 232448, limit_set);
  if (e != cudaSuccess) return e;
  const size_t need = Layout<DP>::total + 1024;
  kern<<<ctas, kThreads, need > 118784 ? need : 118784, st>>>(a);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  evo_seq_weights_join_kernel<<<ctas, kTile, 0, st>>>(a, ctas);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_seq_weights(const SeqWeightsArgs& a, int ctas, bool bf16, cudaStream_t st) {
  if (a.scores) {
    const dim3 grid((a.s.max_kv + 1023) / 1024, a.s.kv_heads, a.s.seqs);
    evo_scores_sum_kernel<<<grid, 256, 0, st>>>(a, ctas);
    return cudaGetLastError();
  }
  if (a.s.D <= 64) return bf16 ? launch_t<64, true>(a, ctas, st) : launch_t<64, false>(a, ctas, st);
  return bf16 ? launch_t<128, true>(a, ctas, st) : launch_t<128, false>(a, ctas, st);
}

}  // namespace evo
