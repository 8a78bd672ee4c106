/*
 * evo_seq.h — C ABI of the causal-sequence attention operators of
 * libevo_attn.so (GB300, sm_103a), beside the Evoformer attention of
 * evo_attn.h, whose status codes, data types and conventions they share.
 *
 * The operators serve and train models that read their tokens in order:
 *
 *   evo_prompt_fwd / evo_prompt_bwd  attention over whole prompts, packed one
 *                      behind the other, with its gradients;
 *   evo_cache_append   new keys and values into a paged cache;
 *   evo_paged_fwd      attention of a chunk of new tokens (a single one
 *                      included) over that cache, and, where asked for, the sum
 *                      of the attention weight every cached key received;
 *   evo_cache_evict    the cache cut down, in place, to the keys that received
 *                      the most weight and the newest ones;
 *   evo_rotary         queries and keys turned by their positions, in front of
 *                      either attention, and gradients turned back;
 *   evo_cache8_append / evo_cache8_read / evo_paged8_fwd  a cache in 8 bits with a
 *                      scale for each block of tokens and head: rows into it,
 *                      rows out of it, and attention over it.
 *
 * What they compute.  Sequence b has n_b new tokens, the last of its L_b
 * tokens (for a prompt n_b = L_b).  Its new token i sits at position
 * p = L_b - n_b + i and sees the keys j <= p (none when p < 0).  Query head h
 * reads key/value head h / (q_heads / kv_heads).  With s the scale:
 *
 *     S_ij = s q_i·k_j     P_ij = softmax_j S_ij     O_i = Σ_j P_ij v_j
 *     lse_i = ln Σ_j exp S_ij
 *
 * and, for a gradient dO: delta_i = dO_i·O_i, dP_ij = dO_i·v_j,
 * dS_ij = P_ij (dP_ij - delta_i), dQ_i = s Σ_j dS_ij k_j,
 * dK_j = s Σ_h Σ_i dS_ij q_i and dV_j = Σ_h Σ_i P_ij dO_i over the heads h of a
 * group.  A row that sees no key, or none with a score above -inf, gives O = 0 and
 * lse = -inf, and no key a weight.
 *
 * Layouts.  All device memory.
 *     q, out, dout, dq        [tokens, q_heads, head_dim]   dtype
 *     k, v, dk, dv            [tokens, kv_heads, head_dim]  dtype
 *     lse                     [q_heads, tokens]             float32
 *     cu_seqlens              [seqs + 1]                    int32: sequence b's
 *         tokens are the rows cu_seqlens[b] .. cu_seqlens[b+1] - 1.  Sequences
 *         may be empty.  Rows in no sequence (before the first or behind the
 *         last) are not touched in any output.
 *     seq_lens                [seqs]                        int32: L_b, the new
 *         tokens included
 *     k_pages, v_pages        [num_pages, page_size, kv_heads, head_dim] dtype
 *     block_table             [seqs, pages_per_seq]         int32: token j of
 *         sequence b is row j % page_size of page block_table[b][j / page_size]
 *     weights                 [seqs, kv_heads, weights_len] float32
 * The token rows of q, k, v, out and the gradients may be strided
 * (evo_seq_strides_t) and the pages of a cache too (evo_cache_shape_t).
 *
 * Supported: head_dim a multiple of 8 from 8 to 128; q_heads a multiple of
 * kv_heads, at most 128 times it; page_size 16, 32, 64 or a multiple of 128 up
 * to 1024; fp16 or bf16 with fp32 accumulation; tokens and seqs of zero
 * (nothing is then done), up to 2^31 - 1024 tokens and 65535 sequences;
 * q_heads up to 65535, kv_heads up to 16384.
 *
 * What the device arrays hold is checked on the device: an offset outside
 * [0, tokens] or below its predecessor, a length that is negative or beyond the
 * table (or weights_len), a page index outside [0, num_pages).  A sequence with
 * a bad offset or length counts as empty; a bad page reads as zeros and is not
 * written.  Either records EVO_ERR_BAD_INDEX in the call's status word (the
 * outputs of that sequence are then undefined, everything else is as usual).
 * Offsets out of order may give a row to two sequences, and the outputs of both
 * are undefined then; attention counts every sequence as empty where all of them
 * together have more rows than tokens.
 *
 * A value that a row does not see does not reach it: what lies behind a
 * sequence's last token, in its last page or in the next sequence, may be
 * anything, NaN and infinities included.
 *
 * Products take their operands in dtype and sum in fp32: P and dS are rounded to
 * dtype in between, and delta is formed from the rounded O.  With fp16 a dS beyond
 * 65504 becomes infinite (and so do the gradients that it enters) and steps
 * below 2^-24 are lost: dO should be scaled to stay within them.
 *
 * Every sum is formed in a fixed order: a call repeated on the same device
 * gives the same bytes.  Calls are asynchronous on `stream`, take no memory of
 * their own and keep nothing; a workspace's contents need not be initialised,
 * and two calls that may run at the same time (streams, captured graphs) need
 * two workspaces.
 */
#ifndef EVO_SEQ_H
#define EVO_SEQ_H

#include "evo_attn.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct {
  int64_t tokens;   /* rows of q, k, v                       */
  int64_t seqs;     /* sequences                             */
  int64_t q_heads, kv_heads, head_dim;
} evo_seq_shape_t;

/* Element strides between token rows (heads and head_dim packed inside a row):
 * multiples of 8, at least heads * head_dim, below 2^36 elements.  0 = packed. */
typedef struct {
  int64_t q, k, v, out, dout, dq, dk, dv;
} evo_seq_strides_t;

/* A paged cache.  The page strides are in elements: multiples of 8, at least
 * page_size * kv_heads * head_dim, below 2^36; 0 = packed.  (Keys and values interleaved in one
 * buffer [num_pages, 2, page_size, kv_heads, head_dim] have twice the packed
 * stride.) */
typedef struct {
  int64_t num_pages, page_size, pages_per_seq;
  int64_t k_page_stride, v_page_stride;
} evo_cache_shape_t;

/* Per-call options; NULL or all zero (but size) = the defaults.
 *   scale          s above; 0 = head_dim^-1/2, otherwise positive, and s·log2 e finite
 *                  (s below 2.358e38)
 *   wait_limit_ns  bound on every device-side wait (0 = 2e9, below 1000 = 1000).  A kernel that gave
 *                  up still waits for its own copies and products, up to 2 s whatever the limit.
 *   status         device int set to EVO_ERR_DEVICE_TIMEOUT or EVO_ERR_BAD_INDEX
 *                  (the caller clears it); NULL = the fallback word, read with
 *                  evo_attn_device_status */
typedef struct {
  uint32_t size;
  uint32_t flags; /* must be 0 */
  float scale;
  uint32_t reserved;
  uint64_t wait_limit_ns;
  int* status;
} evo_seq_options_t;

/* Bytes of device workspace (256-byte aligned) that the calls need; 0 on a bad
 * shape.  They depend on the shape and on the current device's number of SMs.
 * With weights and few rows a key (tokens * group up to 16 * seqs) there is room in it
 * for the scores, 4 bytes for every token, query head and place that the table (or
 * weights_len, if that is less) can hold, as long as that is at most a quarter of the
 * cache's bytes; beyond, the keys are read a second time instead. */
EVO_API size_t evo_prompt_fwd_workspace_bytes(evo_seq_shape_t shape);
EVO_API size_t evo_prompt_bwd_workspace_bytes(evo_seq_shape_t shape);
EVO_API size_t evo_paged_fwd_workspace_bytes(evo_seq_shape_t shape, evo_cache_shape_t cache,
                                             int64_t weights_len /* 0: a call without weights */);

/* Attention over whole prompts: out and lse of every row of a sequence. */
EVO_API evo_status_t evo_prompt_fwd(const void* q, const void* k, const void* v, const int32_t* cu_seqlens,
                                    void* out, float* lse, void* workspace, size_t workspace_bytes,
                                    evo_seq_shape_t shape, evo_dtype_t dtype, const evo_seq_strides_t* strides,
                                    const evo_seq_options_t* opts, void* stream);

/* Its gradients, from the forward's inputs and outputs and dout.  A NaN or an
 * infinity in a sequence may reach every gradient of that sequence, and none of
 * another. */
EVO_API evo_status_t evo_prompt_bwd(const void* q, const void* k, const void* v, const int32_t* cu_seqlens,
                                    const void* out, const float* lse, const void* dout, void* dq, void* dk,
                                    void* dv, void* workspace, size_t workspace_bytes, evo_seq_shape_t shape,
                                    evo_dtype_t dtype, const evo_seq_strides_t* strides,
                                    const evo_seq_options_t* opts, void* stream);

/* Writes the rows of k and v (sequence b's new tokens, the last of its
 * seq_lens[b]) into the cache.  A new token at a negative position (more new
 * tokens than seq_lens) is not written.  No two tokens may share a cache row. */
EVO_API evo_status_t evo_cache_append(const void* k, const void* v, const int32_t* cu_seqlens,
                                      const int32_t* seq_lens, const int32_t* block_table, void* k_pages,
                                      void* v_pages, evo_seq_shape_t shape, evo_cache_shape_t cache,
                                      evo_dtype_t dtype, const evo_seq_strides_t* strides,
                                      const evo_seq_options_t* opts, void* stream);

/* Attention of new tokens over the cache, which already holds their own keys
 * and values (evo_cache_append).  With weights (nullable; weights_len columns),
 * weights[b][h][j] += Σ P_ij over the new tokens i of sequence b and the query
 * heads of group h, for every j < seq_lens[b]; other entries are not touched. */
EVO_API evo_status_t evo_paged_fwd(const void* q, const void* k_pages, const void* v_pages,
                                   const int32_t* cu_seqlens, const int32_t* seq_lens, const int32_t* block_table,
                                   void* out, float* lse, float* weights, int64_t weights_len, void* workspace,
                                   size_t workspace_bytes, evo_seq_shape_t shape, evo_cache_shape_t cache,
                                   evo_dtype_t dtype, const evo_seq_strides_t* strides,
                                   const evo_seq_options_t* opts, void* stream);

/* Cuts every sequence with seq_lens[b] > budget down to budget tokens, for each
 * key/value head on its own: the `recent` newest tokens and, of the others, the
 * budget - recent with the largest weights (of equal ones the oldest; a NaN
 * counts as less than every number).  The rows that stay keep their order and
 * move to places 0 .. budget - 1 of the same pages, their weights with them; the
 * weights of the places given up become 0, and seq_lens[b] becomes budget.
 *   kept  [seqs, kv_heads, budget] int32 output: the place each row came from,
 *         -1 behind the last row of a shorter sequence.
 * Sequences with seq_lens[b] <= budget stay as they are.  1 <= budget,
 * 0 <= recent <= budget.  No page may appear twice among the sequences' tables
 * (up to their lengths): rows are moved in place.  (shape.tokens and
 * shape.q_heads are not used.) */
EVO_API evo_status_t evo_cache_evict(void* k_pages, void* v_pages, const int32_t* block_table, int32_t* seq_lens,
                                     float* weights, int64_t weights_len, int32_t* kept, int64_t budget,
                                     int64_t recent, evo_seq_shape_t shape, evo_cache_shape_t cache,
                                     evo_dtype_t dtype, const evo_seq_options_t* opts, void* stream);

/* ---------------------------------------------------------------- rotary positions
 *
 * Feature pair i < rotary_dim / 2 of every head of token t is turned by the angle
 * a = positions[t] * inv_freq[i] and multiplied by `factor`:
 *
 *     y1 = factor (x1 cos a - x2 sin a)      y2 = factor (x2 cos a + x1 sin a)
 *
 * Pair i is the features (i, i + rotary_dim / 2), with EVO_ROTARY_INTERLEAVED
 * (2i, 2i + 1); features from rotary_dim on pass unchanged.  EVO_ROTARY_INVERSE turns
 * by -a: with it the call takes the gradients of its outputs to those of its inputs.
 * Contexts longer than trained on are a matter of inv_freq and factor.  Angles are
 * formed modulo a turn in 64-bit integers: position and frequency lose nothing up
 * to positions of 2^31 (an error of 2^-52 turns a position).  fp32 arithmetic, rounded once. */
#define EVO_ROTARY_INTERLEAVED 1u
#define EVO_ROTARY_INVERSE 2u
typedef struct {
  int64_t rotary_dim;   /* even, 2 .. head_dim                                */
  uint32_t flags;
  float factor;         /* finite; 0 = 1                                      */
  int64_t q_out, k_out; /* token strides of the outputs, as evo_seq_strides_t */
} evo_rotary_t;

/* q [tokens, q_heads, head_dim] and k [tokens, kv_heads, head_dim] (k and k_out may
 * be NULL: q alone) into q_out and k_out.  An output may be its own input, with the same
 * stride, and overlaps no other tensor of the call.  positions [tokens] int32, of either sign;
 * inv_freq [rotary_dim / 2] float64, finite.  q_heads 1 to 65535, kv_heads up to 16384, neither a
 * multiple of the other; shape.seqs is not used, of the strides q and k are. */
EVO_API evo_status_t evo_rotary(const void* q, const void* k, const int32_t* positions, const double* inv_freq,
                                void* q_out, void* k_out, evo_seq_shape_t shape, const evo_rotary_t* rotary,
                                evo_dtype_t dtype, const evo_seq_strides_t* strides, void* stream);

/* ---------------------------------------------------------------- a cache in 8 bits
 *
 *     k_pages, v_pages    [num_pages, page_size, kv_heads, head_dim]  e4m3 (1 + 4 + 3 bits,
 *         bias 7, no infinities, 0x7f and 0xff are NaN)
 *     k_scales, v_scales  [num_pages, kv_heads, page_size / scale_block] float32: a code
 *         stands for code * scale of its block of scale_block tokens and head
 *
 * head_dim is a multiple of 16, scale_block 16, 32, 64 or 128 and divides page_size;
 * everything else (tables, lengths, offsets, what is checked on the device) is as for
 * the 16-bit cache.
 *
 * Appending: a block's scale is the least power of two s, 2^-64 at the least, with |x| <= 448 s
 * for the block's new values x, and not below the scale that tokens from before left the
 * block with.  Where it grows, their codes are rescaled: exactly, but for what falls
 * below the smallest code, 2^-9 of the new scale.  A code is x (1 / s) rounded to nearest even.  A value
 * that is not finite is stored as NaN and does not enter the scale.  Where a block's first
 * token is new, what its scale held before does not matter.
 *
 * Scales that others wrote may be 0 and any numbers from 2^-64 to 2^120.  Reading rounds code * scale to
 * dtype (for scales that are powers of two exact within its range) and saturates at its largest
 * finite number.  Attention takes code * scale as it is (a value with a scale of 0 with 2^-64), or, over a copy (see
 * evo_paged8_fwd), as reading gives it: for scales as an append writes them and values within dtype's normal numbers the
 * same.  P is rounded to dtype, with few rows a key to fp16 whatever dtype is; bf16 queries then
 * lose what is below 2^-39 of their row's largest.  The scales of the values that a row sees lie within 2^90 of one
 * another: a key whose scale is farther below another's may lose its weight.  With many rows a key sums of q times codes have to
 * be float32 numbers (bf16: |q| below 2^111, as head_dim is at most 128); with fp16 values are taken in steps of 2^-24
 * then, and some beyond 65504 may cost those beside them their precision. */
typedef struct {
  int64_t num_pages, page_size, pages_per_seq;
  int64_t scale_block;
  int64_t k_page_stride, v_page_stride; /* in elements: multiples of 16, at least a page, below 2^36; 0 = packed */
} evo_cache8_shape_t;

/* As evo_cache_append; k and v are in dtype.  No two sequences of a call may write
 * into the same block. */
EVO_API evo_status_t evo_cache8_append(const void* k, const void* v, const int32_t* cu_seqlens,
                                       const int32_t* seq_lens, const int32_t* block_table, void* k_pages,
                                       void* v_pages, float* k_scales, float* v_scales, evo_seq_shape_t shape,
                                       evo_cache8_shape_t cache, evo_dtype_t dtype, const evo_seq_strides_t* strides,
                                       const evo_seq_options_t* opts, void* stream);

/* The last tokens of every sequence out of the cache: the rows cu_seqlens[b] ..
 * cu_seqlens[b+1] - 1 of k and v become the last of sequence b's seq_lens[b] tokens, as the
 * rows of an append would be.  A row at a negative position or on a bad page becomes zeros. */
EVO_API evo_status_t evo_cache8_read(const void* k_pages, const void* v_pages, const float* k_scales,
                                     const float* v_scales, const int32_t* cu_seqlens, const int32_t* seq_lens,
                                     const int32_t* block_table, void* k, void* v, evo_seq_shape_t shape,
                                     evo_cache8_shape_t cache, evo_dtype_t dtype, const evo_seq_strides_t* strides,
                                     const evo_seq_options_t* opts, void* stream);

/* As evo_paged_fwd without weights; q and out are in dtype.  With many rows a key (tokens * group above 512 * seqs)
 * the workspace has room for a copy in 16 bits of all that the table can hold, as long as that is at most
 * 512 MB; otherwise codes are widened where they are used.  With few rows (tokens * group up to 32 * seqs, group up to
 * 16) short contexts need no workspace: 0, and NULL will do.  Those are tables of at most 128 places, and of at most 1024 where
 * the call has no more than a kv head's 16 rows for every SM: kv_heads * (tokens / floor(16 / group) + seqs) up to their
 * number.  (A bad shape gives 0 too, and the call says so.) */
EVO_API size_t evo_paged8_fwd_workspace_bytes(evo_seq_shape_t shape, evo_cache8_shape_t cache);
EVO_API evo_status_t evo_paged8_fwd(const void* q, const void* k_pages, const void* v_pages, const float* k_scales,
                                    const float* v_scales, const int32_t* cu_seqlens, const int32_t* seq_lens,
                                    const int32_t* block_table, void* out, float* lse, void* workspace,
                                    size_t workspace_bytes, evo_seq_shape_t shape, evo_cache8_shape_t cache,
                                    evo_dtype_t dtype, const evo_seq_strides_t* strides,
                                    const evo_seq_options_t* opts, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* EVO_SEQ_H */
