// evo_seq8_cache.cu — rows into and out of the 8-bit cache of include/evo_seq.h.
#include "evo_seq8_internal.h"

namespace evo {
namespace {

// ------------------------------------------------------------------ append
// One CTA per block of tokens that a sequence's new tokens reach and eight, or fewer, of its
// (keys or values, head) units: a warp per 16 tokens of a unit, the loads of its rows all under way
// together, the largest magnitude joined over the unit's warps.
//
// How many blocks the sequences reach is known on the device only.  n tokens reach at most
// floor(n / B) + 2 blocks of B, so sequence b is given the numbers from floor(cu[b] / B) + 2 b
// on, which the CTAs search; the numbers that are left over have no block.  (The search, not the
// bytes, is what a step of single tokens waits for.)
//
// What it cannot do without: two bytes read and one written an element where the scale does not grow. 10,188 tokens of 8 heads of
// 128, keys and values, take 16 us, where those bytes take 9: a CTA's search, length, table, rows and stores wait for one another, and
// the three CTAs of an SM hold too little of it under way (28 % of DRAM's throughput, 1.7 of 4 instructions a clock).
constexpr int kAppendThreads = 256;

__device__ __forceinline__ long long block_number(const SeqDesc& s, int block, int b) {
  return static_cast<long long>(s.cu[b] / block) + 2 * static_cast<long long>(b);
}

// The last sequence whose numbers begin at or before i, looked for by a whole warp; -1: none.
__device__ __forceinline__ int find_block(const SeqDesc& s, int block, long long i) {
  const int lane = threadIdx.x & 31;
  int lo = 0, n = s.seqs;  // it is in [lo, lo + n), if any
  while (n > 0) {
    const int step = (n + 31) / 32, at = lo + lane * step;
    const bool below = lane * step < n && block_number(s, block, at) <= i;
    const uint32_t m = __ballot_sync(0xffffffffu, below);
    // (offsets out of order: any answer, looked over below)
    const int last = 31 - __clz(m);
    if (last < 0) return -1;
    if (step == 1) return lo + last;
    n = n - last * step < step ? n - last * step : step;
    lo += last * step;
  }
  return -1;
}

// The least power of two s >= 2^-64 with most <= 448 s (448 = 1.75 · 2^8).
__device__ __forceinline__ float scale_for(float most) {
  const uint32_t u = __float_as_uint(most);
  int e = static_cast<int>(u >> 23) - 8 + ((u & 0x7fffffu) > 0x600000u);
  if (e < 127 - 64) e = 127 - 64;
  return __uint_as_float(static_cast<uint32_t>(e) << 23);
}

// The larger of two magnitudes, in pairs of 16 bits (a NaN is larger than every number).
__device__ __forceinline__ uint32_t larger(uint32_t most, uint32_t w) { return __vmaxu2(most, w & 0x7fff7fffu); }

// A pair of bf16 or f16 with what is not finite as `otherwise`.
template <bool BF16>
__device__ __forceinline__ float2 finite2(uint32_t w, float otherwise) {
  float2 f = unpack2<BF16>(w);
  f.x = fabsf(f.x) < INFINITY ? f.x : otherwise;
  f.y = fabsf(f.y) < INFINITY ? f.y : otherwise;
  return f;
}

// A warp's rows lie P lanes each, P the power of two that holds their 16-byte pieces, 32 / P rows at a time; the
// largest magnitude is looked for in pairs of 16 bits, and only where that is no number among numbers
// alone.  (10,188 tokens of 8 heads of 128 in blocks of 64: 16 us, 3.9 TB/s; with a division for every piece's row
// and comparisons in 32 bits 29.  What bounds it now is latency, as above; several units a CTA,
// which saves the lookups, and more CTAs an SM with fewer registers changed nothing.)
template <bool BF16>
__global__ void __launch_bounds__(kAppendThreads) evo_append8_kernel(const __grid_constant__ Cache8Args a) {
  __shared__ uint32_t warp_most[8];
  const SeqDesc& s = a.s;
  const Cache8& c = a.c;
  if (blockIdx.x == 0 && blockIdx.y == 0) check_seqs(s);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int b = find_block(s, c.block, blockIdx.x);
  if (b < 0) return;
  const Seq q = load_seq(s, b);
  if (q.n == 0) return;
  const int p0 = q.pos0 > 0 ? q.pos0 : 0;  // first position that is written
  const long long index = p0 / c.block + (static_cast<long long>(blockIdx.x) - block_number(s, c.block, b));
  if (index * c.block >= q.kv) return;
  const int start = static_cast<int>(index) * c.block;
  const int lo = start > p0 ? start : p0, hi = q.kv - start < c.block ? q.kv : start + c.block;
  if (lo >= hi) return;
  const int p = page_of(s, b, start);
  if (p < 0) return;
  // (up to here every thread of the block went the same way)
  const int team = c.block / 16, units = 8 / team;                               // warps a unit, units at a time
  const int per = s.D / 8, shift = per > 8 ? 4 : per > 4 ? 3 : per > 2 ? 2 : 1;  // pieces a row, log2 P
  const int piece = lane & ((1 << shift) - 1), step = 32 >> shift;               // of the row, and rows at a time
  const int place = (warp % team) * 16 + (lane >> shift), in_page = start % s.page;  // first row in the block
  const int steps = 1 << (shift - 1);
  const int row = s.kv_heads * s.D;
  const bool older = start < lo;
  constexpr uint32_t inf = BF16 ? 0x7f80u : 0x7c00u;
  const int unit = blockIdx.y * units + warp / team;
  const bool work = unit < 2 * s.kv_heads, live = work && piece < per;
  const int kv = unit >= s.kv_heads, h = work ? (kv ? unit - s.kv_heads : unit) : 0;
  const uint16_t* rows = (kv ? a.v : a.k) + static_cast<long long>(h) * s.D + piece * 8;
  const long long stride = kv ? a.v_stride : a.k_stride;
  uint8_t* page = (kv ? c.v_pages + p * c.v_page : c.k_pages + p * c.k_page) + h * s.D + piece * 8;
  float* scale = (kv ? c.v_scales : c.k_scales) + scale_at(c, s, p, h, start);
  const float before = work && older ? *scale : 0.0f;
  uint4 x[8];
#pragma unroll
  for (int r = 0; r < 8; ++r) {
    const int j = start + place + r * step;
    x[r] = make_uint4(0u, 0u, 0u, 0u);
    if (live && r < steps && j >= lo && j < hi)
      x[r] = __ldcs(reinterpret_cast<const uint4*>(rows + (q.row0 + static_cast<long long>(j - q.pos0)) * stride));
  }
  uint32_t bits = 0;
#pragma unroll
  for (int r = 0; r < 8; ++r) bits = larger(larger(larger(larger(bits, x[r].x), x[r].y), x[r].z), x[r].w);
  bits = __reduce_max_sync(0xffffffffu, max(bits & 0xffffu, bits >> 16));
  const bool all_finite = bits < inf;
  if (!all_finite) {
    bits = 0;
#pragma unroll
    for (int r = 0; r < 8; ++r) {
      const uint32_t w[4] = {x[r].x, x[r].y, x[r].z, x[r].w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint32_t l = w[e] & 0x7fffu, u = (w[e] >> 16) & 0x7fffu;
        bits = max(bits, max(l < inf ? l : 0u, u < inf ? u : 0u));
      }
    }
    bits = __reduce_max_sync(0xffffffffu, bits);
  }
  if (team > 1) {
    if (lane == 0) warp_most[warp] = bits;
    __syncthreads();
    for (int i = 0; i < team; ++i) bits = max(bits, warp_most[warp / team * team + i]);
  }
  if (!work) return;
  float now = scale_for(to_f32<BF16>(static_cast<uint16_t>(bits)));
  if (before > now && before < INFINITY) now = before;  // (a block without tokens from before has 0 there)
  if (older && now != before && live) {
    const float shrink = before >= 0.0f && before < INFINITY ? before / now : 1.0f;  // (0: they stand for 0)
    for (int r = 0; r < steps; ++r) {
      const int at = place + r * step;
      if (start + at >= lo) break;
      uint2* to = reinterpret_cast<uint2*>(page + static_cast<long long>(in_page + at) * row);
      float y[8];
      f32_of_codes(*to, y);
#pragma unroll
      for (int e = 0; e < 8; ++e) y[e] *= shrink;
      *to = codes_of_f32(y);
    }
  }
  const float inv = 1.0f / now;  // (exact for a power of two)
#pragma unroll
  for (int r = 0; r < 8; ++r) {
    const int at = place + r * step, j = start + at;
    if (!live || r >= steps || j < lo || j >= hi) continue;
    const uint32_t w[4] = {x[r].x, x[r].y, x[r].z, x[r].w};
    float y[8];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float2 f = all_finite ? unpack2<BF16>(w[e]) : finite2<BF16>(w[e], NAN);
      y[2 * e] = f.x * inv;
      y[2 * e + 1] = f.y * inv;
    }
    *reinterpret_cast<uint2*>(page + static_cast<long long>(in_page + at) * row) = codes_of_f32(y);
  }
  if (lane == 0 && warp % team == 0 && now != before) *scale = now;
}

// ------------------------------------------------------------------ read
// A warp takes eight tokens next to each other: a lane each finds its sequence, page and place, then the warp
// goes over the 16-code pieces of one token after the other, keys and values, which are next to each other in both.
// One byte read and two written an element: 10,460 tokens of 8 heads of 128 take 14 us, where those bytes take 9.5 (loads one
// by one between the stores 18; a thread a piece, each with its own search and divisions, 20).  What bounds it is latency, the searches
// and table entries in front of a warp's loads: 17 % of DRAM's throughput (the writes stay in L2), 1.7 of 4 instructions a clock.
constexpr int kReadTokens = 8;

// x times scale, at most `most` in magnitude, as a pair of the output's type.
template <bool BF16>
__device__ __forceinline__ uint32_t read2(uint32_t codes_f16, float scale) {
  constexpr float most = BF16 ? 3.38953139e38f : 65504.0f;
  float2 f = unpack2<false>(codes_f16);
  f = make_float2(f.x * scale, f.y * scale);
  // (comparisons that a NaN passes unchanged)
  f.x = f.x > most ? most : (f.x < -most ? -most : f.x);
  f.y = f.y > most ? most : (f.y < -most ? -most : f.y);
  return pack2<BF16>(f.x, f.y);
}

// One token's keys and values out of row r of page p (p < 0: zeros), by a warp: pieces of 16 codes, four a lane under way
// together.
struct RowShape {
  int per, chunks, shift;  // pieces a head, and a row; log2 of the tokens a scale
  uint32_t magic;          // ceil(2^32 / per), for exact quotients below 2^29
  __device__ __forceinline__ RowShape(const SeqDesc& s, const Cache8& c) {
    per = s.D / 16;
    chunks = s.kv_heads * per;
    shift = __ffs(c.block) - 1;
    magic = 0xffffffffu / per + 1;
  }
};
template <bool BF16>
__device__ __forceinline__ void read_row(const SeqDesc& s, const Cache8& c, const RowShape& q, int p, int r, uint16_t* ko,
                                         uint16_t* vo, bool wide) {
  const int lane = threadIdx.x & 31;
  const uint8_t* kp = c.k_pages + p * c.k_page + static_cast<long long>(r) * q.chunks * 16;
  const uint8_t* vp = c.v_pages + p * c.v_page + static_cast<long long>(r) * q.chunks * 16;
  const long long scales = static_cast<long long>(p) * s.kv_heads * c.blocks + (r >> q.shift);
  for (int n0 = lane; n0 < 2 * q.chunks; n0 += 128) {
    uint4 x[4];
    float scale[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int n = n0 + 32 * e, kv = n >= q.chunks, at = kv ? n - q.chunks : n;
      x[e] = make_uint4(0u, 0u, 0u, 0u);
      scale[e] = 0.0f;
      if (p >= 0 && n < 2 * q.chunks) {
        const int h = q.per == 1 ? at : static_cast<int>(__umulhi(static_cast<uint32_t>(at), q.magic));  // at / per
        x[e] = __ldcs(reinterpret_cast<const uint4*>((kv ? vp : kp) + at * 16));
        scale[e] = __ldg((kv ? c.v_scales : c.k_scales) + scales + static_cast<long long>(h) * c.blocks);
      }
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int n = n0 + 32 * e, kv = n >= q.chunks, at = kv ? n - q.chunks : n;
      if (n >= 2 * q.chunks) continue;
      const uint2 w[4] = {f16x4_of_codes(x[e].x), f16x4_of_codes(x[e].y), f16x4_of_codes(x[e].z), f16x4_of_codes(x[e].w)};
      uint32_t o[8];
#pragma unroll
      for (int i = 0; i < 4; ++i) o[2 * i] = read2<BF16>(w[i].x, scale[e]), o[2 * i + 1] = read2<BF16>(w[i].y, scale[e]);
      uint16_t* to = (kv ? vo : ko) + at * 16;
      if (wide) {
        st_global_32(to, o);
      } else {
        *reinterpret_cast<uint4*>(to) = make_uint4(o[0], o[1], o[2], o[3]);
        *reinterpret_cast<uint4*>(to + 8) = make_uint4(o[4], o[5], o[6], o[7]);
      }
    }
  }
}

template <bool BF16>
__global__ void __launch_bounds__(256) evo_read8_kernel(const __grid_constant__ Cache8Args a) {
  const SeqDesc& s = a.s;
  if (blockIdx.x == 0) check_seqs(s);
  const int lane = threadIdx.x & 31, tokens = a.tokens_a_warp;
  const long long first = (static_cast<long long>(blockIdx.x) * 8 + (threadIdx.x >> 5)) * tokens;
  if (first >= s.tokens) return;
  // this lane's token: -2 in no sequence, -1 not there, otherwise its page, and the row in it
  int page = -2, row = 0;
  if (lane < tokens && first + lane < s.tokens) {
    const int t = static_cast<int>(first) + lane, b = find_seq(s, t);
    if (b >= 0) {
      const Seq q = load_seq(s, b);
      if (t >= q.row0 && t < q.row0 + q.n) {
        const int j = q.pos0 + (t - q.row0);
        page = j < 0 ? -1 : page_of(s, b, j);
        row = j < 0 ? 0 : j % s.page;
      }
    }
  }
  const RowShape shape(s, a.c);
  for (int i = 0; i < tokens; ++i) {
    const int p = __shfl_sync(0xffffffffu, page, i), r = __shfl_sync(0xffffffffu, row, i);
    if (p != -2) read_row<BF16>(s, a.c, shape, p, r, a.k + (first + i) * a.k_stride, a.v + (first + i) * a.v_stride,
                                a.wide);
  }
}

// ------------------------------------------------------------------ a copy in 16 bits
// Every sequence's pages as pages of 16 bits, one behind the other, with a table for them, for the attention of many
// rows a key: page i of sequence b becomes page b · pages_per_seq + i.  The CTAs take the pages there are by turns,
// a warp a token.  Rows behind a sequence's end stay as they are.  (23,348 tokens of 8 heads of 128: 27 us, 5.3 TB/s.)
template <bool BF16>
__global__ void __launch_bounds__(256) evo_copy8_kernel(const __grid_constant__ Cache8Args a, int* table) {
  const SeqDesc& s = a.s;
  if (blockIdx.x == 0) check_seqs(s);
  const int warp = threadIdx.x >> 5;
  const RowShape shape(s, a.c);
  const long long row = static_cast<long long>(s.kv_heads) * s.D;
  unsigned turn = blockIdx.x;  // the first page of the sequence that is this CTA's
  for (int b = 0; b < s.seqs; ++b) {
    const Seq q = load_seq(s, b);
    const unsigned n = q.n > 0 ? static_cast<unsigned>((q.kv + s.page - 1) / s.page) : 0u;
    unsigned i = turn;
    for (; i < n; i += gridDim.x) {
      const int to = b * s.pages_per_seq + static_cast<int>(i), p = page_of(s, b, static_cast<int>(i) * s.page);
      const int tokens = min(s.page, q.kv - static_cast<int>(i) * s.page);
      if (threadIdx.x == 0) table[to] = to;
      for (int r = warp; r < tokens; r += 8) {
        const long long at = (static_cast<long long>(to) * s.page + r) * row;
        read_row<BF16>(s, a.c, shape, p, r, a.k + at, a.v + at, true);
      }
    }
    turn = i - n;  // (one behind the last page that was there: the turns go on in the next sequence)
  }
}

}  // namespace

cudaError_t launch_cache8_append(const Cache8Args& a, bool bf16, cudaStream_t st) {
  const long long blocks = static_cast<long long>(a.s.tokens) / a.c.block + 2ll * a.s.seqs;
  const int units = 8 / (a.c.block / 16), groups = (2 * a.s.kv_heads + units - 1) / units;  // a CTA, CTAs a block
  const dim3 grid(static_cast<unsigned>(blocks), static_cast<unsigned>(groups));
  if (bf16)
    evo_append8_kernel<true><<<grid, kAppendThreads, 0, st>>>(a);
  else
    evo_append8_kernel<false><<<grid, kAppendThreads, 0, st>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_cache8_read(const Cache8Args& args, int sms, bool bf16, cudaStream_t st) {
  Cache8Args a = args;
  // fewer tokens a warp where there would be fewer than six blocks an SM
  a.tokens_a_warp = kReadTokens;
  while (a.tokens_a_warp > 1 && a.s.tokens / (8 * a.tokens_a_warp) < 6 * sms) a.tokens_a_warp /= 2;
  const long long tokens = 8ll * a.tokens_a_warp;
  const unsigned grid = static_cast<unsigned>((a.s.tokens + tokens - 1) / tokens);
  if (bf16)
    evo_read8_kernel<true><<<grid, 256, 0, st>>>(a);
  else
    evo_read8_kernel<false><<<grid, 256, 0, st>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_cache8_copy(const Cache8Args& a, int* table, int sms, bool bf16, cudaStream_t st) {
  const long long pages = static_cast<long long>(a.s.seqs) * a.s.pages_per_seq;
  const unsigned grid = static_cast<unsigned>(pages < 6ll * sms ? pages : 6ll * sms);
  if (bf16)
    evo_copy8_kernel<true><<<grid, 256, 0, st>>>(a, table);
  else
    evo_copy8_kernel<false><<<grid, 256, 0, st>>>(a, table);
  return cudaGetLastError();
}

}  // namespace evo
