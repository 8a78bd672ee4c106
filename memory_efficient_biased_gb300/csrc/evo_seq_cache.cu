// evo_seq_cache.cu — the paged cache of include/evo_seq.h: new rows written into
// its pages, and eviction by accumulated attention weight.
#include "evo_seq_internal.h"

namespace evo {
namespace {

// ------------------------------------------------------------------ append
// One thread per 16 bytes of a token's key row and the same of its value row.  Bound by
// the bytes (2 reads and 2 writes of tokens x kv_heads x head_dim), in practice by the
// launch for the few tokens of a step.
__global__ void __launch_bounds__(256) evo_append_kernel(const AppendArgs a) {
  const SeqDesc& s = a.s;
  if (blockIdx.x == 0) check_seqs(s);
  const int chunks = s.kv_heads * s.D / 8;
  const long long i = static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x;
  if (i >= static_cast<long long>(s.tokens) * chunks) return;
  const int t = static_cast<int>(i / chunks), c = static_cast<int>(i % chunks);
  const int b = find_seq(s, t);
  if (b < 0) return;
  const Seq q = load_seq(s, b);
  if (t < q.row0 || t >= q.row0 + q.n) return;
  const int j = q.pos0 + (t - q.row0);
  if (j < 0) return;
  const int p = page_of(s, b, j);
  if (p < 0) return;
  const long long in = static_cast<long long>(j % s.page) * s.kv_heads * s.D + c * 8;
  *reinterpret_cast<uint4*>(a.k_pages + p * a.k_page + in) =
      *reinterpret_cast<const uint4*>(a.k + t * a.k_stride + c * 8);
  *reinterpret_cast<uint4*>(a.v_pages + p * a.v_page + in) =
      *reinterpret_cast<const uint4*>(a.v + t * a.v_stride + c * 8);
}

// ------------------------------------------------------------------ eviction: choice
// A weight as an unsigned number in the same order: NaN below everything, -0 equal to 0.
__device__ __forceinline__ uint32_t ordered(float w) {
  if (w != w) return 0u;
  const uint32_t u = w == 0.0f ? 0u : __float_as_uint(w);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

constexpr int kSelThreads = 1024, kSelPer = 4, kSelDeep = 8, kBins = 2048;

// One CTA per (kv head, sequence).  The smallest weight that stays is found by radix
// selection over the ordered weights (11 + 11 + 10 bits: three histograms in shared
// memory, whose counts do not depend on the order of the atomics); then one pass in order
// of place gives every kept row its new place (a running count of what is kept: those
// above the threshold, the first `ties` equal to it, the newest `recent`) and moves the
// weights down in place.  The weights (4 bytes a place) are read four times, the repeats
// from L2; the rows they stand for are 512 bytes a place at head_dim 128, so the moves
// below are what an eviction costs.
__global__ void __launch_bounds__(kSelThreads) evo_evict_select_kernel(const EvictArgs a) {
  __shared__ uint32_t hist[kBins];
  __shared__ uint32_t warp_sums[32];
  __shared__ uint32_t pick[2];
  const SeqDesc& s = a.s;
  const int h = blockIdx.x, b = blockIdx.y, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const long long bh = static_cast<long long>(b) * s.kv_heads + h;
  int* kept = a.kept + bh * a.budget;
  int len = a.seq_lens[b];
  if (len < 0 || len > s.max_kv) {
    if (tid == 0) report_bad_index(s.status);
    len = 0;
  }
  if (len <= a.budget) {
    for (int i = tid; i < a.budget; i += kSelThreads) kept[i] = i < len ? i : -1;
    return;
  }
  float* w = a.weights + bh * a.weights_len;
  // Places are unsigned: the last pass over them may look up to 8192 past 2^31 (and see that nothing is there).
  const uint32_t size = len, n = len - a.recent;
  const int k = a.budget - a.recent;  // of the n oldest that stay
  uint32_t prefix = 0, mask = 0, want = k;                // of those matching prefix, `want` stay
  if (k > 0) {
#pragma unroll 1
    for (int round = 0; round < 3; ++round) {
      const int shift = round == 0 ? 21 : (round == 1 ? 10 : 0), bits = round == 2 ? 10 : 11;
      const uint32_t low = (1u << bits) - 1u;
      for (int i = tid; i < kBins; i += kSelThreads) hist[i] = 0;
      __syncthreads();
      for (uint32_t base = tid; base < n; base += kSelThreads * kSelDeep) {
        float x[kSelDeep];  // loads in front of the counting, so that they are under way together
#pragma unroll
        for (int e = 0; e < kSelDeep; ++e) x[e] = base + e * kSelThreads < n ? w[base + e * kSelThreads] : 0.0f;
#pragma unroll
        for (int e = 0; e < kSelDeep; ++e) {
          const uint32_t u = ordered(x[e]);
          if (base + e * kSelThreads < n && (u & mask) == prefix) atomicAdd(&hist[(u >> shift) & low], 1u);
        }
      }
      __syncthreads();
      // bins from the largest down: thread t holds bins 2047 - 2t and 2046 - 2t
      const uint32_t c0 = hist[kBins - 1 - 2 * tid], c1 = hist[kBins - 2 - 2 * tid];
      uint32_t run = c0 + c1;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t x = __shfl_up_sync(0xffffffffu, run, o);
        if (lane >= o) run += x;
      }
      if (lane == 31) warp_sums[warp] = run;
      __syncthreads();
      uint32_t before = run - c0 - c1;
      for (int x = 0; x < warp; ++x) before += warp_sums[x];
      if (before < want && before + c0 >= want) {
        pick[0] = kBins - 1 - 2 * tid;
        pick[1] = want - before;
      } else if (before + c0 < want && before + c0 + c1 >= want) {
        pick[0] = kBins - 2 - 2 * tid;
        pick[1] = want - before - c0;
      }
      __syncthreads();
      prefix |= pick[0] << shift;
      mask |= low << shift;
      want = pick[1];
    }
  }
  // `want` of the weights equal to `prefix` stay (k == 0: none does)
  uint32_t above = 0, equal = 0;  // kept so far: above the threshold (or recent), equal to it
  for (uint32_t base = 0; base < size; base += kSelThreads * kSelPer) {
    const uint32_t j0 = base + tid * kSelPer;
    float x[kSelPer];
    uint32_t up = 0, eq = 0;  // bits
#pragma unroll
    for (int e = 0; e < kSelPer; ++e) {
      x[e] = 0.0f;
      if (j0 + e < size) {
        x[e] = w[j0 + e];
        const uint32_t u = ordered(x[e]);
        if (j0 + e >= n || (k > 0 && u > prefix))
          up |= 1u << e;
        else if (k > 0 && u == prefix)
          eq |= 1u << e;
      }
    }
    // counts of this pass before this thread (both below 2^13: one word)
    const uint32_t mine = static_cast<uint32_t>(__popc(up)) << 16 | static_cast<uint32_t>(__popc(eq));
    uint32_t run = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t y = __shfl_up_sync(0xffffffffu, run, o);
      if (lane >= o) run += y;
    }
    if (lane == 31) warp_sums[warp] = run;
    __syncthreads();
    uint32_t before = run - mine, total = 0;
    for (int y = 0; y < 32; ++y) {
      const uint32_t v = warp_sums[y];
      if (y < warp) before += v;
      total += v;
    }
    uint32_t u0 = above + (before >> 16), e0 = equal + (before & 0xffffu);
#pragma unroll
    for (int e = 0; e < kSelPer; ++e) {
      const bool is_up = (up >> e) & 1u, is_eq = (eq >> e) & 1u;
      if (is_up || (is_eq && e0 < want)) {
        const uint32_t to = u0 + (e0 < want ? e0 : want);
        kept[to] = static_cast<int>(j0 + e);
        w[to] = x[e];  // to <= j0 + e: places of this pass, already read, or of an earlier one
      }
      u0 += is_up;
      e0 += is_eq;
    }
    above += total >> 16;
    equal += total & 0xffffu;
    __syncthreads();  // warp_sums is rewritten by the next pass, and w below it is final
  }
  for (uint32_t j = a.budget + tid; j < size; j += kSelThreads) w[j] = 0.0f;
}

// ------------------------------------------------------------------ eviction: moves
constexpr int kMoveThreads = 512, kMoveDeep = 4, kMoveTable = 4096;

// One CTA per 64-byte slice of the rows of one (sequence, kv head) of keys or values.
// Row i moves from place kept[i] >= i: no row that is still to be read lies at or below a
// place already written, so batches in order need only all of a batch's reads to be done
// before its writes (one barrier), and the next batch's reads may be under way meanwhile.
// Bound by the bytes: a row read and written once.  64-byte slices rather than whole rows
// give four times the CTAs at head_dim 128 and keep whole sectors.  The places of a batch are
// read two batches ahead and the sequence's pages are looked up in shared memory, so that
// only the rows themselves are waited for.  (16 sequences, 8 heads of 128, 4096 rows kept: 512 threads
// with four rows each in flight 88 us, 6.1 TB/s; 256 threads 6 us more, eight rows each 38, 128-byte
// slices 16.)
__global__ void __launch_bounds__(kMoveThreads) evo_evict_move_kernel(const EvictArgs a, int slices) {
  __shared__ int table[kMoveTable];
  const SeqDesc& s = a.s;
  const int slice = blockIdx.x % slices, kv = blockIdx.x / slices, h = blockIdx.y, b = blockIdx.z;
  const int* kept = a.kept + (static_cast<long long>(b) * s.kv_heads + h) * a.budget;
  const int len = kept[a.budget - 1] + 1;  // places read are below it (0: the sequence is not cut)
  const int entries = len / s.page + 1;
  for (int i = threadIdx.x; i < entries && i < s.pages_per_seq && i < kMoveTable; i += kMoveThreads)
    table[i] = s.table[static_cast<size_t>(b) * s.pages_per_seq + i];
  __syncthreads();
  uint16_t* pages = kv ? a.v_pages : a.k_pages;
  const long long page_stride = kv ? a.v_page : a.k_page;
  const int chunk = slice * 4 + (threadIdx.x & 3);  // 16 bytes
  const bool live = chunk * 8 < s.D;
  constexpr int kRows = kMoveThreads / 4 * kMoveDeep;
  const int r0 = threadIdx.x >> 2;
  const int row = s.kv_heads * s.D;
  const int shift = (s.page & (s.page - 1)) ? -1 : __ffs(s.page) - 1;  // (a division each way was half of the instructions)
  pages += static_cast<long long>(h) * s.D + chunk * 8;
  auto place = [&](int j) -> uint16_t* {
    const int e = shift >= 0 ? j >> shift : j / s.page;
    int p;
    if (e < kMoveTable) {
      p = table[e];
      if (p < 0 || p >= s.num_pages) {
        report_bad_index(s.status);
        return nullptr;
      }
    } else {
      p = page_of(s, b, j);
      if (p < 0) return nullptr;
    }
    return pages + p * page_stride + static_cast<long long>(j - e * s.page) * row;
  };
  auto places = [&](int base, int (&from)[kMoveDeep]) {
#pragma unroll
    for (int e = 0; e < kMoveDeep; ++e) {
      const int i = base + e * (kMoveThreads / 4) + r0;
      from[e] = i < a.budget && live ? kept[i] : -1;
    }
  };
  auto load = [&](int base, const int (&from)[kMoveDeep], uint4 (&x)[kMoveDeep]) -> uint32_t {
    uint32_t has = 0;
#pragma unroll
    for (int e = 0; e < kMoveDeep; ++e) {
      // (a row that stays where it is is left alone)
      if (from[e] < 0 || from[e] == base + e * (kMoveThreads / 4) + r0) continue;
      const uint16_t* p = place(from[e]);
      if (!p) continue;
      x[e] = __ldcg(reinterpret_cast<const uint4*>(p));
      has |= 1u << e;
    }
    return has;
  };
  uint4 now[kMoveDeep], ahead[kMoveDeep];
  int from[kMoveDeep], next[kMoveDeep];
  places(0, from);
  places(kRows, next);
  uint32_t has_now = load(0, from, now), has_ahead = 0;
  for (int base = 0; base < a.budget; base += kRows) {
#pragma unroll
    for (int e = 0; e < kMoveDeep; ++e) from[e] = next[e];
    places(base + 2 * kRows, next);
    has_ahead = load(base + kRows, from, ahead);
    __syncthreads();
#pragma unroll
    for (int e = 0; e < kMoveDeep; ++e) {
      if (!((has_now >> e) & 1u)) continue;
      uint16_t* p = place(base + e * (kMoveThreads / 4) + r0);
      if (p) *reinterpret_cast<uint4*>(p) = now[e];
    }
#pragma unroll
    for (int e = 0; e < kMoveDeep; ++e) now[e] = ahead[e];
    has_now = has_ahead;
  }
  // the only reader and writer of this length in this launch
  if (blockIdx.x == 0 && h == 0 && threadIdx.x == 0) {
    const int n = a.seq_lens[b];
    if (n > a.budget && n <= s.max_kv) a.seq_lens[b] = a.budget;
  }
}

}  // namespace

cudaError_t launch_cache_append(const AppendArgs& a, cudaStream_t st) {
  const long long n = static_cast<long long>(a.s.tokens) * (a.s.kv_heads * a.s.D / 8);
  evo_append_kernel<<<static_cast<unsigned>((n + 255) / 256), 256, 0, st>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_cache_evict(const EvictArgs& a, cudaStream_t st) {
  evo_evict_select_kernel<<<dim3(a.s.kv_heads, a.s.seqs), kSelThreads, 0, st>>>(a);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const int slices = (a.s.D + 31) / 32;
  evo_evict_move_kernel<<<dim3(2 * slices, a.s.kv_heads, a.s.seqs), kMoveThreads, 0, st>>>(a, slices);
  return cudaGetLastError();
}

}  // namespace evo
