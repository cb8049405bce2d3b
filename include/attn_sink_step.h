/*
 * attn_sink_step.h -- C ABI of libattn_sink.so, continued: what a model step
 * does around the attention of attn_sink.h.
 *
 *   attn_sink_page_plan      block tables, slot map and positions of a serving
 *                            step over the paged cache, from request lengths
 *   attn_sink_qkv_rope       RMS norm of every query and key head and rotary
 *                            positions in one pass over the packed projection;
 *                            in serving k and v go straight into their pages
 *   attn_sink_qkv_rope_bwd   its gradient
 *   attn_sink_extend         attention with a sink of several new tokens per
 *                            sequence over the paged cache (chunks of prompts,
 *                            drafted tokens)
 *
 * A serving step is plan -> qkv_rope (slots given) -> extend, or
 * attn_sink_decode when every sequence has one new token.  A training step is
 * qkv_rope -> attn_sink_fwd / attn_sink_bwd -> qkv_rope_bwd.
 *
 * Conventions (ownership, streams, errors, the device error word) are those of
 * attn_sink.h: every pointer but params is device memory of the caller on the
 * current device, calls are asynchronous on `stream`, allocate nothing, never
 * synchronise, can be captured into a graph, and validate their arguments on
 * the host before any launch.  Two calls that may overlap need a workspace
 * each; two graphs that are never replayed at the same time may share one.
 */
#ifndef ATTN_SINK_STEP_H
#define ATTN_SINK_STEP_H

#include <stddef.h>

#ifdef __cplusplus
extern "C" {
#endif

/*
 * Device error code of attn_sink_page_plan (see attn_sink_device_error): a
 * length was negative or did not fit its block-table row, the tokens did not
 * fit max_tokens, the free pages ran out, or a page index was outside the
 * cache.  attn_sink_qkv_rope records 0x800 for a slot outside the cache, and
 * attn_sink_extend for a bad length, block-table entry or cu_seqlens entry.
 */
#define ATTN_SINK_DEVERR_PLAN 0x1000

typedef struct attn_sink_plan_params {
  int batch;      /* 0 <= B <= 2^24 sequences */
  int page_size;  /* keys per page, >= 1 */
  int num_pages;  /* pages of the cache: valid page indices are [0, num_pages) */
  int max_pages;  /* columns of block_table; max_pages * page_size <= 2^30 */
  int num_free;   /* entries of free_pages */
  int max_tokens; /* entries of slots and positions: tokens of the step at most */
} attn_sink_plan_params;

/*
 * Plan of a serving step in which sequence b, with cached_lens[b] keys in the
 * cache, gets new_lens[b] new tokens (either may be 0).  The pages of its
 * cached keys are in block_table[b, 0 .. ceil(cached / page_size)); a partly
 * filled last page is filled up first, and further pages come from free_pages
 * in order, sequence by sequence.  In place and out:
 *   block_table [B, max_pages] int32: the new pages are written behind the
 *     cached ones; every other entry keeps its value
 *   slots [max_tokens] int64: the cache row page * page_size + offset of each
 *     new token, packed sequence by sequence; -1 behind the last token and for
 *     a token that got no page
 *   positions [max_tokens] int32: the token's position in its sequence (its
 *     key index); 0 behind the last token
 *   cu_seqlens [B + 1] int32: the packed new tokens' offsets
 *   seq_lens [B] int32: cached + new
 *   pages_needed [1] int32: entries of free_pages this plan takes (more than
 *     num_free when they ran out)
 * The next step's free list is this one without its first pages_needed entries; to
 * shift it on the device, fill its end with -1 (no page: outside the cache).
 * A second call with the same inputs gives the same plan.  Lengths are clamped
 * to [0, max_pages * page_size] and cu_seqlens to max_tokens; when free_pages
 * runs out the entries are -1.  Each of these records ATTN_SINK_DEVERR_PLAN.
 * Sequences may share pages that are full (a common prefix), not one that is
 * partly filled and gets new tokens.  Outputs must not overlap inputs: seq_lens
 * in the place of cached_lens or new_lens is refused.  No workspace; one launch, two
 * from 65536 sequences on.
 */
int attn_sink_page_plan(const attn_sink_plan_params* params, const int* cached_lens,
                        const int* new_lens, const int* free_pages, int* block_table,
                        long long* slots, int* positions, int* cu_seqlens, int* seq_lens,
                        int* pages_needed, void* stream);

#define ATTN_SINK_ROPE_MAX_AXES 4

typedef struct attn_sink_rope_params {
  long long q_stride;  /* elements from one token to the next in q, k and v: */
  long long k_stride;  /*   multiples of 8, at least heads * 64 */
  long long v_stride;
  int tokens;          /* T >= 0 */
  int heads_q;         /* >= 1 */
  int heads_kv;        /* >= 1 */
  int head_dim;        /* must be 64 */
  int rotary_dim;      /* leading dimensions that are rotated: 0, 16, 32, 48 or 64 */
  int interleaved;     /* pair i is (i, i + rotary_dim / 2), or (2i, 2i + 1) if 1 */
  int num_axes;        /* rows of positions, 1 .. 4 */
  unsigned char pair_axis[32]; /* the axis whose position turns pair i */
  int norm;            /* 1: RMS norm of each q and k head before the rotation */
  int weight_bf16;     /* norm weights: 0 = fp32 [64], 1 = bf16 [64] */
  float eps;           /* added to the mean square; finite and >= 0 */
  float amplitude;     /* factor of the rotated dimensions; finite */
  int page_size;       /* serving: cache of num_pages * page_size rows; else 0 */
  int num_pages;
  int grad_dtype;      /* backward: dq, dk, dv come as 0 = bf16, 1 = fp32 */
} attn_sink_rope_params;

/*
 * For every token t and head, with x the head's 64 numbers:
 *   u = x / sqrt(mean(x^2) + eps) * weight    (norm = 1; q and k have a weight
 *                                              each, shared by their heads)
 *   (y_a, y_b) = amplitude * (u_a cos - u_b sin, u_b cos + u_a sin) for every
 *   pair, angle = positions[pair_axis[i], t] * inv_freq[i],
 * and the dimensions from rotary_dim on pass unrotated.  v passes unchanged.
 * q [T, heads_q, 64], k and v [T, heads_kv, 64] bf16 with the token strides of
 * params (heads contiguous): views of one packed projection, or tensors of
 * their own; positions [num_axes, T] int32; inv_freq [rotary_dim / 2] fp32
 * (with whatever frequency scaling the model uses).
 * Writes q_out [T, heads_q, 64] and, where they are not NULL, k_out and v_out
 * [T, heads_kv, 64] (contiguous bf16).  With slots [T] int64 (NULL: no cache),
 * k and v also go to row slots[t] of k_cache and v_cache [num_pages *
 * page_size, heads_kv, 64]; a slot of -1 writes no row, any other slot outside
 * the cache is skipped and recorded as 0x800.  Slots of one call have to be
 * distinct (as attn_sink_page_plan makes them).  Outputs must not overlap
 * inputs.  The angle is reduced to one turn in 64 bits (inv_freq / 2 pi to 2^-64
 * turns, times the position) and rounded to fp32 then, so far positions lose nothing
 * and small angles keep 24 bits; the rest is fp32, rounded once.  q_weight and
 * k_weight may be NULL with norm = 0, inv_freq and positions with rotary_dim = 0.
 * No workspace; one launch.
 */
int attn_sink_qkv_rope(const attn_sink_rope_params* params, const void* q, const void* k,
                       const void* v, const int* positions, const float* inv_freq,
                       const void* q_weight, const void* k_weight, const long long* slots,
                       void* q_out, void* k_out, void* v_out, void* k_cache, void* v_cache,
                       void* stream);

/* Bytes of device workspace attn_sink_qkv_rope_bwd needs: the weight
 * gradients' partial sums (0 with norm = 0, tokens = 0 or invalid params).
 * Query it on the device the call will run on. */
size_t attn_sink_qkv_rope_bwd_workspace_size(const attn_sink_rope_params* params);

/*
 * Gradient of attn_sink_qkv_rope (slots play no part).  q and k are the
 * forward's inputs (only read with norm = 1, NULL allowed otherwise) with
 * their strides; dq [T, heads_q, 64], dk and dv [T, heads_kv, 64] contiguous,
 * bf16 or fp32 (grad_dtype, as attn_sink_bwd writes them).  Writes dq_in, dk_in
 * and dv_in (bf16, rounded once from fp32; token strides dq_in_stride,
 * dk_in_stride, dv_in_stride: views of one packed gradient, or tensors of
 * their own) and, with norm = 1, the weights' gradients dq_weight and
 * dk_weight [64] fp32, summed in a fixed order (bitwise reproducible).  dv and
 * dv_in may both be NULL.  positions and inv_freq as in the forward.  Outputs
 * must not overlap inputs.
 */
int attn_sink_qkv_rope_bwd(const attn_sink_rope_params* params, const void* q, const void* k,
                           const int* positions, const float* inv_freq, const void* q_weight,
                           const void* k_weight, const void* dq, const void* dk, const void* dv,
                           void* dq_in, void* dk_in, void* dv_in, long long dq_in_stride,
                           long long dk_in_stride, long long dv_in_stride, float* dq_weight,
                           float* dk_weight, void* workspace, size_t workspace_bytes,
                           void* stream);

typedef struct attn_sink_extend_params {
  int batch;          /* 0 <= B <= 2^24 sequences */
  int total_q;        /* T <= 2^30: rows of q and out; cu_seqlens_q[B] <= T */
  int heads_q;        /* G * heads_kv with 1 <= G <= 128 */
  int heads_kv;       /* >= 1 */
  int head_dim;       /* must be 64 */
  int page_size;      /* keys per page, >= 1 */
  int num_pages;      /* pages of the cache; num_pages * page_size * heads_kv < 2^32 */
  int max_pages;      /* columns of block_table; max_pages * page_size <= 2^30 */
  int window;         /* <= 0: none; W > 0: the W most recent keys */
  float softmax_scale;/* multiplies q.k only; finite and > 0 */
} attn_sink_extend_params;

/* Bytes of device workspace attn_sink_extend needs, on the current device (0 if
 * the params are invalid or there is nothing to do): the list of work items and
 * either the partial results of key ranges that are split over several CTAs or,
 * for windows on the band kernel, the keys and values gathered from their pages. */
size_t attn_sink_extend_workspace_size(const attn_sink_extend_params* params);

/*
 * Attention with the sink of attn_sink_fwd, causal, of the n_b =
 * cu_seqlens_q[b + 1] - cu_seqlens_q[b] last tokens of each sequence over its
 * seq_lens[b] = L_b cached keys (the new tokens' own included, written before
 * the call): token i of sequence b sits at key position L_b - n_b + i and sees
 * the keys up to it, or the last W of them.  n_b = 0 and L_b = 0 are allowed,
 * and n_b > L_b too: a token before the first key sees none and gets out = 0,
 * lse = sink.  A sink of -inf is none, one of +inf gives out = 0, lse = inf.
 * Layouts as attn_sink_decode, with q, out [T, heads_q, 64] bf16
 * and lse [heads_q, T] fp32; rows of out and lse behind cu_seqlens_q[B] are
 * left as they were.  Cache rows past a sequence's keys and pages behind every
 * token's window are not used, whatever they hold (block-table entries of such
 * pages are not read); a value of +-inf or NaN in a key or value row that some
 * token of a tile sees reaches that tile's outputs.
 * S = q k^T multiplies the bf16 inputs exactly with fp32 sums, and lse comes
 * from fp32 probabilities.  For O = P v they are rounded to bf16 next to the bf16
 * values.  With a window that the band kernel of attn_sink_fwd covers (128 / G +
 * W - 1 <= 176 keys, G > 1 a power of two), 8 new tokens a sequence on average
 * (128 where G = 2) and more than 128 sequences or more tiles than the GPU holds at
 * once, they are rounded to fp16 next to fp16 copies of the values, which have
 * to lie within the fp16 range there (|v| <= 65504, else 0x400 is recorded, as by
 * attn_sink_fwd; below 2^-14 they are rounded to multiples of 2^-24).
 * A length outside [0, max_pages * page_size] is clamped, the keys of a
 * block-table entry outside [0, num_pages) are skipped, and cu_seqlens_q is
 * clamped to [0, T]; each is recorded as 0x800.  The workspace is 256-byte
 * aligned.  out and lse must not overlap the inputs.  The result does not depend
 * on timing: the same inputs give the same bits.
 */
int attn_sink_extend(const attn_sink_extend_params* params, const void* q, const void* k_cache,
                     const void* v_cache, const int* block_table, const int* seq_lens,
                     const int* cu_seqlens_q, const float* sink, void* out, float* lse,
                     void* workspace, size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* ATTN_SINK_STEP_H */
