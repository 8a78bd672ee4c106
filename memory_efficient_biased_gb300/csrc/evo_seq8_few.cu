// evo_seq8_few.cu — attention over the 8-bit cache (include/evo_seq.h) for few rows a key: single tokens,
// or a few of them, with their group's heads in 16 rows.
//
// Mathematics, per row (token, head) and block of keys with scales s_k and s_v: S = q·code_k,
// t = s_k s·log2e·S, P' = 2^(t + log2 s_v - M) with M the running maximum of t + log2 s_v, l = Σ P' / s_v and
// O = Σ P' code_v; at the end O / l and lse = ln2·(M + log2 l).  The weight that a value enters with is
// P' = P s_v: held against the largest such product it fits fp16 whatever the scales, and the codes
// themselves, exact in fp16, are the other operand.  q is exact in fp16 too, for bf16 after its row
// is brought to a largest magnitude of 1 to 2 by a power of two (what falls below 2^-24 of that is lost).
//
// Why mma.sync.  A byte of the cache has to be turned into 16 bits before a product of 16 bits
// takes it.  tcgen05 would take it from shared memory: staged, read, written twice as wide and read by the product,
// 6 to 7 bytes through shared memory for each of HBM's (128 a clock and SM, where HBM's share is 23).  Fragments
// in registers are read once from the staged tile and widened on their way into the product: 2 bytes. The
// products need 16 rows · 23 = 370 multiply-adds a clock and SM, a third of what mma.sync has.
//
// Roles (9 warps, one CTA per SM, persistent over its share of the work, evo_seq_sched.cuh):
//   warps 0-7  16 keys of every tile of 128 each, which share their scales; M, l and O of their own,
//              joined at the end of an item
//   warp 8     the walk over the work; K and V tiles by TMA (a page is a box), scales by cp.async
//
// Fragments.  Inside a product the order of the features (scores) and of the keys (P·V) is free, so a lane takes 16
// bytes next to each other: of key g for the scores (lane = 4 g + c: features 16 c .. and 64 + 16 c ..), of keys
// c, c + 4, c + 8, c + 12 for P·V (features 16 G(g) ..), whose bytes are paired by permutes.  Key (g / 2) + 4 (g % 2) stands
// in column g of the scores and G(g) = (g % 2) 4 + g / 2, so that with the tiles' 128-byte swizzle no read meets a bank twice.
#include "evo_seq8_internal.h"
#include "evo_seq_sched.cuh"

namespace evo {
namespace {

constexpr int kRows = 16, kWarps = 8, kThreads = 32 * (kWarps + 1), kDescs = 4;

template <int DP>
struct Layout {
  static constexpr uint32_t kTB = kTile * DP;  // one tile of codes
  static constexpr int kStages = DP == 128 ? 4 : 8;
  static constexpr int kPitch = DP + 4;        // floats between rows of a warp's O
  static constexpr uint32_t ring = 0, merge = kStages * 2 * kTB, bars = merge + kWarps * kRows * kPitch * 4;
};

struct Bars {
  uint64_t desc_full[kDescs], desc_empty[kDescs];
  uint64_t full[8], empty[8];
  uint64_t merge_full, merge_empty;
  Work work[kDescs];
  float scales[8][2][8];          // of a stage: keys and values, 16 tokens each
  float2 ml[kWarps][kRows];
  uint32_t tiles;
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

// ------------------------------------------------------------ walk and loads (one warp)
template <int DP>
__device__ __forceinline__ void produce(const Seq8FwdArgs& a, uint8_t* base, Bars* bars, const WaitGuard& g, int lane) {
  using L = Layout<DP>;
  const SeqDesc& s = a.f.s;
  const Cache8& c = a.c;
  Walk<QueryBlocks> walk;
  walk.init(s, QueryBlocks{a.f.W}, blockIdx.x, gridDim.x);
  PieceRecord* rec = a.f.records + 2 * blockIdx.x;
  if (lane < 2) rec[lane].used = 0;
  __syncwarp();
  const int box = s.page < kTile ? s.page : kTile, boxes = kTile / box;
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
    if (w.stop) break;
    // this lane's page of a tile (a page past the keys, or a bad one, reads as zeros)
    auto page = [&](int j) -> int {
      const int key = j * kTile + lane * box;
      if (lane >= boxes || key >= w.kv_end) return s.num_pages;
      const int p = page_of(s, w.b, key);
      return p < 0 ? s.num_pages : p;
    };
    int mine = page(w.j0);
    bool ok = true;
    for (int j = w.j0; j < w.j1; ++j, ++use) {
      const int cur = mine;
      if (j + 1 < w.j1) mine = page(j + 1);
      const uint32_t st = use % L::kStages;
      if (!mbar_wait_warp_inl(smem_u32(&bars->empty[st]), ((use / L::kStages) & 1) ^ 1, g)) { ok = false; break; }
      const uint32_t full = smem_u32(&bars->full[st]), dst = smem_u32(base + L::ring + st * 2 * L::kTB);
      if (lane == 0) mbar_arrive_expect_tx(full, 2 * L::kTB);
      __syncwarp();
      const int first = boxes == 1 ? (j * kTile) % s.page : 0;
      if (lane < boxes) {
        tma_load_4d(dst + lane * box * DP, &a.f.tk, full, 0, w.kvh, first, cur);
        tma_load_4d(dst + L::kTB + lane * box * DP, &a.f.tv, full, 0, w.kvh, first, cur);
      }
      // the scale of 16 tokens: lanes 0-7 keys, 8-15 values
      const int part = lane & 7, token = part * 16;
      const int p = __shfl_sync(0xffffffffu, cur, token / box);
      if (lane < 16) {
        float* to = &bars->scales[st][lane >> 3][part];
        if (p < s.num_pages && j * kTile + token < w.kv_end) {
          const float* from = (lane >> 3 ? c.v_scales : c.k_scales) + scale_at(c, s, p, w.kvh, first + token);
          asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(to)), "l"(from) : "memory");
          asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(full) : "memory");
        } else {
          *to = 1.0f;
          mbar_arrive(full);
        }
      }
      __syncwarp();
    }
    if (!ok) break;
  }
  if (lane == 0) bars->tiles = use;
}

// ------------------------------------------------------------ compute (warps 0..7)
template <int DP, bool BF16>
__device__ __forceinline__ void compute(const Seq8FwdArgs& a, uint8_t* base, Bars* bars, const WaitGuard& g) {
  using L = Layout<DP>;
  constexpr int kHalves = DP / 64, kCols = DP / 8;  // 16-byte pieces a lane of a key, tiles of eight features
  const SeqDesc& s = a.f.s;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, gr = lane >> 2, c = lane & 3;
  // rows gr and gr + 8: token within the item, head within the group
  const int G = s.group, dt0 = gr / G, dt1 = (gr + 8) / G, h0 = gr % G, h1 = (gr + 8) % G;
  float* mine = reinterpret_cast<float*>(base + L::merge) + warp * kRows * L::kPitch;
  uint32_t use = 0, merges = 0;
  for (uint32_t it = 0;; ++it) {
    const uint32_t ds = it % kDescs;
    if (!mbar_wait_warp_inl(smem_u32(&bars->desc_full[ds]), (it / kDescs) & 1, g)) return;
    const Work w = bars->work[ds];
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_u32(&bars->desc_empty[ds]));
    if (w.stop) return;
    const bool live0 = dt0 < w.nt, live1 = dt1 < w.nt;  // (nt <= 16 / G: rows past the item's are none's)
    // ---- q: features 64 i + 16 c + 4 k + (0, 1 | 2, 3) are elements (2c, 2c + 1 | 2c + 8, 2c + 9) of step 4 i + k
    uint32_t q[4 * kHalves][4];
    float unit[2] = {1.0f, 1.0f};
    {
      uint2 x[2][4 * kHalves];
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const size_t row = static_cast<size_t>(w.row0) + w.t0 + (r ? dt1 : dt0);
        const uint16_t* from = a.q + row * a.q_stride + static_cast<size_t>(w.kvh * G + (r ? h1 : h0)) * s.D + 16 * c;
#pragma unroll
        for (int k = 0; k < 4 * kHalves; ++k) {
          const int at = 64 * (k >> 2) + 4 * (k & 3);
          x[r][k] = make_uint2(0u, 0u);
          if ((r ? live1 : live0) && 16 * c + at < s.D) x[r][k] = *reinterpret_cast<const uint2*>(from + at);
        }
      }
      if constexpr (BF16) {
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          uint32_t most = 0;  // magnitudes, as two 16-bit numbers
#pragma unroll
          for (int k = 0; k < 4 * kHalves; ++k)
            most = __vmaxu2(__vmaxu2(most, x[r][k].x & 0x7fff7fffu), x[r][k].y & 0x7fff7fffu);
          most = max(most & 0xffffu, most >> 16);
          most = max(most, __shfl_xor_sync(0xffffffffu, most, 1));
          most = max(most, __shfl_xor_sync(0xffffffffu, most, 2));
          const uint32_t e = min(max(most >> 7, 1u), 253u);
          const float down = __uint_as_float((254u - e) << 23);
          unit[r] = __uint_as_float(e << 23);
#pragma unroll
          for (int k = 0; k < 4 * kHalves; ++k) {
            const float2 f0 = unpack2<true>(x[r][k].x), f1 = unpack2<true>(x[r][k].y);
            x[r][k] = make_uint2(pack2<false>(f0.x * down, f0.y * down), pack2<false>(f1.x * down, f1.y * down));
          }
        }
      }
#pragma unroll
      for (int k = 0; k < 4 * kHalves; ++k) q[k][0] = x[0][k].x, q[k][1] = x[1][k].x, q[k][2] = x[0][k].y, q[k][3] = x[1][k].y;
    }
    unit[0] *= a.f.scale_log2;
    unit[1] *= a.f.scale_log2;
    const int pos0 = w.pos + dt0, pos1 = w.pos + dt1;
    float o[kCols][4] = {};
    float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.0f, l1 = 0.0f;
    for (int j = w.j0; j < w.j1; ++j, ++use) {
      const uint32_t st = use % L::kStages;
      if (!mbar_wait_warp_inl(smem_u32(&bars->full[st]), (use / L::kStages) & 1, g)) return;
      const int key0 = j * kTile + warp * 16;
      if (key0 >= w.kv_end) {
        if (lane == 0) mbar_arrive(smem_u32(&bars->empty[st]));
        continue;
      }
      const uint32_t kt = smem_u32(base + L::ring + st * 2 * L::kTB) + warp * 16 * DP, vt = kt + L::kTB;
      const float ks = bars->scales[st][0][warp], vs = bars->scales[st][1][warp];
      // ---- scores: column g of tile n is key 8 n + (g / 2) + 4 (g % 2)
      float sc[2][kHalves][4] = {};
#pragma unroll
      for (int n = 0; n < 2; ++n) {
        const int r = 8 * n + (gr >> 1) + 4 * (gr & 1);
        const uint32_t row = kt + r * DP;
#pragma unroll
        for (int i = 0; i < kHalves; ++i) {
          const uint32_t piece = DP == 128 ? static_cast<uint32_t>((c + 4 * i) ^ (r & 7)) : static_cast<uint32_t>(c ^ ((r >> 1) & 3));
          const uint4 x = lds128(row + piece * 16);
          const uint32_t u[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
          for (int k = 0; k < 4; ++k)
            mma16816(sc[n][i], q[4 * i + k], f16x2_of_e4m3x2(u[k]), f16x2_of_e4m3x2(u[k] >> 16));
        }
      }
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
      float t[2][4];  // tile n: (row gr: keys 8n + c, 8n + c + 4), (row gr + 8: the same)
      const float k0 = unit[0] * ks, k1 = unit[1] * ks;
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float x = sc[n][0][e];
          if constexpr (kHalves == 2) x += sc[n][1][e];
          t[n][e] = x * (e < 2 ? k0 : k1);
        }
      const bool edge = key0 + 15 > w.pos;  // some row does not see some key
      if (edge) {
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (key0 + 8 * n + c + 4 * (e & 1) > (e < 2 ? pos0 : pos1)) t[n][e] = -INFINITY;
      }
      float a0 = fmaxf(fmaxf(t[0][0], t[0][1]), fmaxf(t[1][0], t[1][1]));
      float a1 = fmaxf(fmaxf(t[0][2], t[0][3]), fmaxf(t[1][2], t[1][3]));
      a0 = fmaxf(a0, __shfl_xor_sync(0xffffffffu, a0, 1));
      a1 = fmaxf(a1, __shfl_xor_sync(0xffffffffu, a1, 1));
      a0 = fmaxf(a0, __shfl_xor_sync(0xffffffffu, a0, 2));
      a1 = fmaxf(a1, __shfl_xor_sync(0xffffffffu, a1, 2));
      const float lv = lg2(vs), iv = ex2(-lv);
      a0 += lv;
      a1 += lv;
      if (__any_sync(0xffffffffu, a0 > m0 || a1 > m1)) {
        const float n0 = fmaxf(m0, a0), n1 = fmaxf(m1, a1);
        const float f0 = m0 == -INFINITY ? 0.0f : ex2(m0 - n0), f1 = m1 == -INFINITY ? 0.0f : ex2(m1 - n1);
        m0 = n0, m1 = n1;
        l0 *= f0, l1 *= f1;
#pragma unroll
        for (int n = 0; n < kCols; ++n) o[n][0] *= f0, o[n][1] *= f0, o[n][2] *= f1, o[n][3] *= f1;
      }
      const float b0 = lv - (m0 == -INFINITY ? 0.0f : m0), b1 = lv - (m1 == -INFINITY ? 0.0f : m1);
      float p0 = 0.0f, p1 = 0.0f;
#pragma unroll
      for (int n = 0; n < 2; ++n) {
#pragma unroll
        for (int e = 0; e < 4; ++e) t[n][e] = ex2(t[n][e] + (e < 2 ? b0 : b1));
        p0 += t[n][0] + t[n][1];
        p1 += t[n][2] + t[n][3];
      }
      l0 = fmaf(p0, iv, l0);
      l1 = fmaf(p1, iv, l1);
      const uint32_t p[4] = {pack2<false>(t[0][0], t[0][1]), pack2<false>(t[0][2], t[0][3]), pack2<false>(t[1][0], t[1][1]),
                             pack2<false>(t[1][2], t[1][3])};
      uint32_t lost = 0;
      if (edge) {
        // rows behind the last key that anyone sees: nothing; codes that are NaN: taken out, and put back below where they are seen
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int e = 0; e < kCols / 4; ++e) {
            if (key0 + c + 4 * i >= w.kv_end) v[i][e] = 0u;
            lost |= nan_bytes(v[i][e]);
          }
      }
      const bool dirty = edge && __any_sync(0xffffffffu, lost != 0);
      if (dirty) {
        // Which rows see a NaN, and in which feature: the product of ones (a key that a row sees) and ones (a code that is NaN).
        uint32_t seen[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int at = key0 + 8 * (e >> 1) + c, pos = (e & 1) ? pos1 : pos0;
          seen[e] = (at <= pos ? 0x3c00u : 0u) | (at + 4 <= pos ? 0x3c000000u : 0u);
        }
#pragma unroll
        for (int e = 0; e < kCols / 4; ++e) {
          uint32_t bad[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            bad[i] = nan_bytes(v[i][e]);
            v[i][e] &= ~bad[i];
          }
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const uint32_t one = 0x3c00u;
            const uint32_t w0 = ((bad[0] >> (8 * k)) & 1u ? one : 0u) | ((bad[1] >> (8 * k)) & 1u ? one << 16 : 0u);
            const uint32_t w1 = ((bad[2] >> (8 * k)) & 1u ? one : 0u) | ((bad[3] >> (8 * k)) & 1u ? one << 16 : 0u);
            float count[4] = {};
            mma16816(count, seen, w0, w1);
#pragma unroll
            for (int x = 0; x < 4; ++x)
              if (count[x] > 0.0f) o[4 * e + k][x] = NAN;
          }
        }
      }
      // ---- O: bytes of keys (c, c + 4) and (c + 8, c + 12) paired, feature by feature
#pragma unroll
      for (int e = 0; e < kCols / 4; ++e) {
        const uint32_t x0 = __byte_perm(v[0][e], v[1][e], 0x5140), x1 = __byte_perm(v[0][e], v[1][e], 0x7362);
        const uint32_t y0 = __byte_perm(v[2][e], v[3][e], 0x5140), y1 = __byte_perm(v[2][e], v[3][e], 0x7362);
        mma16816(o[4 * e], p, f16x2_of_e4m3x2(x0), f16x2_of_e4m3x2(y0));
        mma16816(o[4 * e + 1], p, f16x2_of_e4m3x2(x0 >> 16), f16x2_of_e4m3x2(y0 >> 16));
        mma16816(o[4 * e + 2], p, f16x2_of_e4m3x2(x1), f16x2_of_e4m3x2(y1));
        mma16816(o[4 * e + 3], p, f16x2_of_e4m3x2(x1 >> 16), f16x2_of_e4m3x2(y1 >> 16));
      }
    }
    // ---- the warps' shares joined
    l0 += __shfl_xor_sync(0xffffffffu, l0, 1);
    l1 += __shfl_xor_sync(0xffffffffu, l1, 1);
    l0 += __shfl_xor_sync(0xffffffffu, l0, 2);
    l1 += __shfl_xor_sync(0xffffffffu, l1, 2);
    if (!mbar_wait_warp_inl(smem_u32(&bars->merge_empty), (merges & 1) ^ 1, g)) return;
    if (c == 0) {
      bars->ml[warp][gr] = make_float2(m0, l0);
      bars->ml[warp][gr + 8] = make_float2(m1, l1);
    }
    // tile n, elements 0 | 1: feature n of piece G(2 c) = c | G(2 c + 1) = 4 + c (D up to 64: 8 (2 c) | 8 (2 c + 1))
#pragma unroll
    for (int half = 0; half < 2; ++half)
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        float* to = mine + (gr + 8 * half) * L::kPitch + (DP == 128 ? 16 * (c + 4 * x) : 8 * (2 * c + x));
#pragma unroll
        for (int n = 0; n < kCols; n += 4)
          *reinterpret_cast<float4*>(to + n) = make_float4(o[n][2 * half + x], o[n + 1][2 * half + x], o[n + 2][2 * half + x],
                                                           o[n + 3][2 * half + x]);
      }
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_u32(&bars->merge_full));
    if (!mbar_wait_warp_inl(smem_u32(&bars->merge_full), merges & 1, g)) return;
    ++merges;
    const int r = threadIdx.x >> 4, d0 = (threadIdx.x & 15) * 8;  // row, eight features
    if (d0 < DP && r / G < w.nt) {
      float2 ml[kWarps];
      float big = -INFINITY, l = 0.0f, f[kWarps];
#pragma unroll
      for (int i = 0; i < kWarps; ++i) {
        ml[i] = bars->ml[i][r];
        if (ml[i].y != 0.0f) big = fmaxf(big, ml[i].x);
      }
#pragma unroll
      for (int i = 0; i < kWarps; ++i) {
        // (a share that saw a NaN may have no maximum: its l is NaN, whatever it is scaled by)
        f[i] = ml[i].y == 0.0f ? 0.0f : (big == -INFINITY ? 1.0f : ex2(ml[i].x - big));
        if (ml[i].y != 0.0f) l += ml[i].y * f[i];
      }
      float x[8] = {};
      const float* from = reinterpret_cast<const float*>(base + L::merge) + r * L::kPitch + d0;
#pragma unroll
      for (int i = 0; i < kWarps; ++i) {
        const float4 y0 = *reinterpret_cast<const float4*>(from + i * kRows * L::kPitch);
        const float4 y1 = *reinterpret_cast<const float4*>(from + i * kRows * L::kPitch + 4);
        if (f[i] == 0.0f && ml[i].y == 0.0f) continue;
        x[0] = fmaf(y0.x, f[i], x[0]), x[1] = fmaf(y0.y, f[i], x[1]), x[2] = fmaf(y0.z, f[i], x[2]), x[3] = fmaf(y0.w, f[i], x[3]);
        x[4] = fmaf(y1.x, f[i], x[4]), x[5] = fmaf(y1.y, f[i], x[5]), x[6] = fmaf(y1.z, f[i], x[6]), x[7] = fmaf(y1.w, f[i], x[7]);
      }
      const size_t row = static_cast<size_t>(w.row0) + w.t0 + r / G;
      const int h = w.kvh * G + r % G;
      if (w.slot < 0) {
        const float inv = l == 0.0f ? 0.0f : 1.0f / l;
        uint32_t y[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) y[e] = l == 0.0f ? 0u : pack2<BF16>(x[2 * e] * inv, x[2 * e + 1] * inv);
        if (d0 < s.D)
          *reinterpret_cast<uint4*>(a.f.out + row * a.f.out_stride + static_cast<size_t>(h) * s.D + d0) =
              make_uint4(y[0], y[1], y[2], y[3]);
        if (d0 == 0) a.f.lse[static_cast<size_t>(h) * s.tokens + row] = l == 0.0f ? -INFINITY : (big + lg2(l)) * kSeqLn2;
      } else {
        const size_t at = (static_cast<size_t>(blockIdx.x) * 2 + w.slot) * 256 + r;
        float4* to = reinterpret_cast<float4*>(a.f.part_o + at * DP + d0);
        to[0] = make_float4(x[0], x[1], x[2], x[3]);
        to[1] = make_float4(x[4], x[5], x[6], x[7]);
        if (d0 == 0) a.f.part_ml[at] = make_float2(big, l);
      }
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_u32(&bars->merge_empty));
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
    bars->tiles = 0;
    for (int i = 0; i < kDescs; ++i) {
      mbar_init(smem_u32(&bars->desc_full[i]), 1);
      mbar_init(smem_u32(&bars->desc_empty[i]), kWarps);
    }
    for (int i = 0; i < L::kStages; ++i) {
      mbar_init(smem_u32(&bars->full[i]), 17);  // the copies' bytes, and a lane for each scale
      mbar_init(smem_u32(&bars->empty[i]), kWarps);
    }
    mbar_init(smem_u32(&bars->merge_full), kWarps);
    mbar_init(smem_u32(&bars->merge_empty), kWarps);
    fence_barrier_init();
  }
  if (warp == kWarps && lane == 0) {
    tma_prefetch_desc(&a.f.tk);
    tma_prefetch_desc(&a.f.tv);
  }
  __syncthreads();
  const WaitGuard g{a.f.wait_ns, a.f.s.status, &bars->abort};
  if (warp == kWarps)
    produce<DP>(a, base, bars, g, lane);
  else
    compute<DP, BF16>(a, base, bars, g);
  __syncthreads();
  if (warp == kWarps) {
    const Owed owed[] = {{bars->full, L::kStages, bars->tiles}};
    drain(owed, g);
  }
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
  if ((e = cudaGetLastError()) != cudaSuccess || a.f.s.max_kv <= kTile) return e;  // one key tile: nothing is cut
  return launch_seq_join(a.f, ctas, BF16, st);
}

}  // namespace

cudaError_t launch_paged8_few(const Seq8FwdArgs& a, int ctas, bool bf16, cudaStream_t st) {
  if (a.f.s.D <= 64) return bf16 ? launch_t<64, true>(a, ctas, st) : launch_t<64, false>(a, ctas, st);
  return bf16 ? launch_t<128, true>(a, ctas, st) : launch_t<128, false>(a, ctas, st);
}

}  // namespace evo
