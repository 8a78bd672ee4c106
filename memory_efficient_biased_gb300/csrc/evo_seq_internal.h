// evo_seq_internal.h — what the kernels of the causal-sequence operators
// (include/evo_seq.h) share: their arguments, and how a sequence is read from
// the offsets, lengths and block table in device memory, which are checked here.
#pragma once

#include "evo_internal.h"
#include "evo_ptx.cuh"
#include "evo_seq_index.h"

namespace evo {

constexpr float kSeqLog2e = 1.4426950408889634f;
constexpr float kSeqLn2 = 0.6931471805599453f;

// One call's sequences.  A prompt has no seq_lens and no table: its keys are its own rows.
struct SeqDesc {
  const int* cu;
  const int* seq_lens;
  const int* table;
  int tokens, seqs;
  int q_heads, kv_heads, group, D;
  int page, pages_per_seq, num_pages;
  int max_kv;  // longest length the table (and weights) can hold
  int* status;
};

// Sequence b: first row, new tokens, length, position of its first new token.
struct Seq {
  int row0, n, kv, pos0;
};

__device__ __forceinline__ void report_bad_index(int* status) { atomicExch(status, kStatusBadIndex); }

__device__ __forceinline__ Seq load_seq(const SeqDesc& d, int b) {
  const int c0 = d.cu[b], c1 = d.cu[b + 1];
  const int kv = d.seq_lens ? d.seq_lens[b] : c1 - c0;
  if (c0 < 0 || c1 < c0 || c1 > d.tokens || kv < 0 || kv > d.max_kv) {
    report_bad_index(d.status);
    return Seq{0, 0, 0, 0};
  }
  return Seq{c0, c1 - c0, kv, kv - (c1 - c0)};
}

// Looks every sequence over (one block's threads): a row's search below may never meet a bad one.
__device__ __forceinline__ void check_seqs(const SeqDesc& d) {
  for (int b = threadIdx.x; b < d.seqs; b += blockDim.x) load_seq(d, b);
}

// The sequence that holds row t, or -1 (a row in front of the first or behind the last).
__device__ __forceinline__ int find_seq(const SeqDesc& d, int t) {
  int lo = 0, hi = d.seqs;  // the last b with cu[b] <= t
  if (t < d.cu[0]) return -1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (d.cu[mid] <= t)
      lo = mid;
    else
      hi = mid - 1;
  }
  return lo < d.seqs ? lo : -1;
}

// The page that holds place j of sequence b, or -1 (recorded) when the table's entry is bad.
__device__ __forceinline__ int page_of(const SeqDesc& d, int b, int j) {
  const int p = d.table[static_cast<size_t>(b) * d.pages_per_seq + j / d.page];
  if (p < 0 || p >= d.num_pages) {
    report_bad_index(d.status);
    return -1;
  }
  return p;
}

// What may still be under way when every role of a CTA has ended, and has to be over before its shared
// memory is anybody else's or its barriers begin anew: copies, MMAs, and the arrivals of the MMAs' last commits
// at barriers that no one else waits on (a commit's arrival may come later than that of a commit behind it).
// Each is a ring of barriers that has gone through `uses` phases.
struct Owed {
  uint64_t* bars;
  uint32_t slots, uses;
};
// Waits for the newest phase of every barrier, one a lane (at most 32).  The limit is not the caller's alone: that
// may be a microsecond, and has just run out where a CTA gives up.
constexpr uint64_t kDrainNs = 2000000000ull;
template <int N>
__device__ __forceinline__ void drain(const Owed (&owed)[N], const WaitGuard& g) {
  const int lane = threadIdx.x & 31;
  uint32_t bar = 0, phase = 0, base = 0;
#pragma unroll
  for (int r = 0; r < N; ++r) {
    const uint32_t i = lane - base;  // (wraps below the ring's first lane)
    if (i < owed[r].slots && i < owed[r].uses) {
      bar = smem_u32(owed[r].bars + i);
      phase = newest_phase(owed[r].uses, owed[r].slots, i);
    }
    base += owed[r].slots;
  }
  if (bar) {
    volatile int never = 0;
    const WaitGuard own{g.limit_ns > kDrainNs ? g.limit_ns : kDrainNs, g.status, &never};
    if (!mbar_wait_inl(bar, phase & 1, own)) *g.abort = 1;
  }
  __syncwarp();
}

struct AppendArgs {
  SeqDesc s;
  const uint16_t *k, *v;
  uint16_t *k_pages, *v_pages;
  long long k_stride, v_stride, k_page, v_page;
};

struct EvictArgs {
  SeqDesc s;  // cu unused
  uint16_t *k_pages, *v_pages;
  long long k_page, v_page;
  int* seq_lens;
  float* weights;
  long long weights_len;
  int* kept;
  int budget, recent;
};

struct PieceRecord;

// The forward on the tensor cores.
struct SeqFwdArgs {
  CUtensorMap tq;       // q as (D, group, kv_heads, tokens), box (64, group, 1, TQ)
  CUtensorMap tk, tv;   // prompt: (D, kv_heads, tokens), box (64, 1, 128); cache: (D, kv_heads, page, num_pages),
                        // box (64, 1, min(page, 128), 1); 128-byte swizzle, zeros outside
  SeqDesc s;
  int TQ, W;            // tokens of a query tile (floor(128 / group)) and of an item (two tiles)
  int out32;            // rows of out start at multiples of 32 bytes
  float scale_log2;     // scale · log2 e
  const uint16_t* v;    // plain pointer and strides of V, for what add_back reads
  long long v_stride, v_page;
  uint16_t* out;
  long long out_stride;
  float* lse;
  PieceRecord* records;  // workspace: two per CTA, and one for the sums of the scores
  float2* part_ml;       // ... [ctas][2][256] (m, l); of few rows a key 16 instead of 256
  float* part_o;         // ... [ctas][2][256][DP], not yet divided by l
  float* scores;         // nullable: s·log2e·S left behind for the weights, [tokens][q_heads][scores_ld]
  long long scores_ld;   // max_kv rounded up to whole tiles
  uint64_t wait_ns;
};
// The sums of the attention weights: from the forward's scores where it left them (scores), else
// formed again (tq, tk as the forward's).
struct SeqWeightsArgs {
  CUtensorMap tq, tk;
  SeqDesc s;
  int TQ;
  float scale_log2;
  const float* lse;
  float* weights;
  long long weights_len;
  const float* scores;
  long long scores_ld;
  PieceRecord* records;  // workspace of the forward, which is done with it
  float* part;           // ... [ctas][2][128]
  uint64_t wait_ns;
};
// Bytes of the workspace for `ctas` CTAs and pieces of `rows` rows; with a and ws, a's pointers into it.
size_t seq_fwd_workspace(int ctas, int D, SeqFwdArgs* a, uint8_t* ws, int rows = 256);

// The prompt's backward on the tensor cores (tk, tv as the prompt forward's).
struct SeqBwdArgs {
  CUtensorMap tq, tdo, tk, tv;
  SeqDesc s;
  int TQ;
  int dq32, dk32, dv32;  // rows of the gradients start at multiples of 32 bytes
  float scale, scale_log2;
  const uint16_t *out, *dout;
  const float* lse;
  uint16_t *dq, *dk, *dv;
  long long out_stride, dout_stride, dq_stride, dk_stride, dv_stride;
  PieceRecord* records;  // workspace: two per CTA for dK and dV, then two for dQ
  float2* rows;          // ... [tokens][q_heads] (-lse·log2 e, -delta)
  float* part;           // ... [ctas][2][dV, dK][128][DP]
  float* part_q;         // ... [ctas][2][128][DP]
  uint64_t wait_ns;
};
size_t prompt_bwd_workspace(int ctas, const SeqDesc& s, SeqBwdArgs* a, uint8_t* ws);

cudaError_t launch_cache_append(const AppendArgs& a, cudaStream_t st);
cudaError_t launch_cache_evict(const EvictArgs& a, cudaStream_t st);
cudaError_t launch_seq_fwd(const SeqFwdArgs& a, int ctas, bool bf16, cudaStream_t st);
// Joins the pieces that cut items left in a forward's workspace (a: s, TQ, out, lse, and the workspace's).
cudaError_t launch_seq_join(const SeqFwdArgs& a, int ctas, bool bf16, cudaStream_t st);
cudaError_t launch_seq_weights(const SeqWeightsArgs& a, int ctas, bool bf16, cudaStream_t st);
cudaError_t launch_prompt_bwd(const SeqBwdArgs& a, int ctas, int rows, bool bf16, cudaStream_t st);

}  // namespace evo
