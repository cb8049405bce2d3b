/*
 * attn_sink_cache.h -- C ABI of libattn_sink.so, continued: decode steps that read
 * less of a long paged key/value cache, and caches that keep less of it.
 *
 *   attn_sink_decode_shared  a decode step in which groups of sequences share a
 *                            prefix, whose keys are read once a group
 *   attn_sink_page_bounds    the elementwise bounds of the keys of every page
 *   attn_sink_select_pages   the pages whose bounds promise the largest scores
 *   attn_sink_decode_pages   a decode step over selected pages
 *   attn_sink_key_mass       the weight every cached key gets from new tokens
 *   attn_sink_evict          keys of little weight leave the cache
 *
 * They stand between attn_sink_page_plan / attn_sink_qkv_rope and the next step:
 *   sparse decode:  plan -> qkv_rope -> page_bounds -> select_pages -> decode_pages
 *   eviction:       plan -> qkv_rope -> decode or extend -> key_mass, and now and
 *                   then evict, whose freed pages go to the next plan
 *
 * Conventions (ownership, streams, errors, the device error word) are those of
 * attn_sink.h and attn_sink_step.h: every pointer but params is device memory of the
 * caller on the current device, calls are asynchronous on `stream`, allocate
 * nothing, never synchronise, can be captured into a graph, and validate their
 * arguments on the host before any launch.  Two calls that may overlap need a
 * workspace each; two graphs that are never replayed at the same time may share
 * one.  Outputs must not overlap inputs where nothing else is said.  The results do
 * not depend on timing: the same inputs give the same bits.  Caches are [num_pages,
 * page_size, heads_kv, 64] bf16, block_table [B, max_pages] int32 and seq_lens [B]
 * int32, as for attn_sink_decode.  Lengths outside [0, max_pages * page_size] are
 * clamped and block-table entries outside [0, num_pages) skipped, where a key that
 * the call uses has one; each is recorded as 0x800 in the device error word.
 */
#ifndef ATTN_SINK_CACHE_H
#define ATTN_SINK_CACHE_H

#include <stddef.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef struct attn_sink_shared_params {
  int batch;          /* 0 <= B <= 65535 sequences; B * heads_q < 2^31 */
  int num_groups;     /* 0 <= P <= B (0 only with B = 0) */
  int heads_q;        /* G * heads_kv with G in {1, 2, 4, 8} */
  int heads_kv;       /* 1 .. 65535 */
  int head_dim;       /* must be 64 */
  int page_size;      /* keys per page, >= 1 */
  int num_pages;      /* num_pages * page_size * heads_kv < 2^32 */
  int max_pages;      /* columns of block_table; max_pages * page_size <= 2^30 */
  float softmax_scale;/* multiplies q.k only; finite and > 0 */
} attn_sink_shared_params;

/* Bytes of device workspace attn_sink_decode_shared needs, on the current device (0
 * if the params are invalid or there is nothing to do). */
size_t attn_sink_decode_shared_workspace_size(const attn_sink_shared_params* params);

/*
 * attn_sink_decode (without window and residual) for sequences in groups: group p
 * is the sequences cu_groups[p] .. cu_groups[p + 1] - 1 (cu_groups [P + 1] int32,
 * from 0 to B, ascending), whose first prefix_lens[p] keys are the same (as where
 * attn_sink_page_plan's block tables share full pages).  Those keys are read through
 * the block-table row of the group's first sequence, once for the group, and meet
 * all its query rows in one product; the keys behind them are each sequence's own.
 * A group's prefix is clamped to its shortest sequence (the rest is read through
 * each sequence's own row), so that the result is attn_sink_decode's whatever
 * prefix_lens holds, as long as the rows' keys there are the same.  A sequence's own
 * keys are shared out over several CTAs only where batch * heads_kv of them leave
 * half of the GPU empty: a larger batch in which some sequences have much longer keys
 * of their own than the others is faster with attn_sink_decode (40 sequences behind
 * 1024 shared keys and 24 of 1000 to 100000 own ones: 771 us, decode 316 us).  A sequence
 * outside every group has no prefix; a cu_groups that does not ascend or leaves
 * [0, B], and a negative prefix_lens, are clamped and recorded as 0x800.
 * q, out [B, heads_q, 64] bf16, lse [heads_q, B] fp32, sink [heads_q] fp32.
 * Scores multiply the bf16 inputs exactly with fp32 sums and the softmax is fp32; in
 * O = P v the values enter as they are, probabilities as the sum of two bf16, off by
 * 2^-16 of their size at most, in the prefix by 2^-14.
 */
int attn_sink_decode_shared(const attn_sink_shared_params* params, const void* q,
                            const void* k_cache, const void* v_cache, const int* block_table,
                            const int* seq_lens, const int* cu_groups, const int* prefix_lens,
                            const float* sink, void* out, float* lse, void* workspace,
                            size_t workspace_bytes, void* stream);

typedef struct attn_sink_bounds_params {
  int batch;          /* 0 <= B <= 2^24 sequences */
  int heads_kv;       /* >= 1 */
  int head_dim;       /* must be 64 */
  int page_size;      /* keys per page, >= 1 */
  int num_pages;      /* num_pages * page_size * heads_kv < 2^32 */
  int max_pages;      /* columns of block_table; max_pages * page_size <= 2^30 */
} attn_sink_bounds_params;

/*
 * For every page that holds keys [cached_lens[b], seq_lens[b]) of a sequence b:
 *   bounds[page, h, 0, d] = min of k[d] over the page's keys of b, all that have been
 *   bounds[page, h, 1, d] = max     written, those before cached_lens[b] too
 * bounds [num_pages, heads_kv, 2, 64] bf16; those of other pages stay as they are.
 * With the cached_lens of attn_sink_page_plan's call and its seq_lens it keeps the
 * bounds of a cache up to date step by step; with cached_lens = 0 it makes them anew
 * (after attn_sink_evict).  A NaN in a key makes its bounds NaN.  Rows of the cache
 * behind seq_lens[b] are not read.  A page that several sequences write has to hold
 * the same keys for each.  A cached_lens outside [0, seq_lens[b]] is clamped; a
 * negative one is recorded.  No workspace; one launch.
 */
int attn_sink_page_bounds(const attn_sink_bounds_params* params, const void* k_cache,
                          const int* block_table, const int* cached_lens, const int* seq_lens,
                          void* bounds, void* stream);

typedef struct attn_sink_select_params {
  int batch;          /* 0 <= B <= 65535 sequences; B * heads_q < 2^31 */
  int heads_q;        /* G * heads_kv with G in {1, 2, 4, 8} */
  int heads_kv;       /* >= 1; B * heads_kv < 2^31 */
  int head_dim;       /* must be 64 */
  int page_size;      /* keys per page, >= 1 */
  int num_pages;      /* num_pages * page_size * heads_kv < 2^32 */
  int max_pages;      /* columns of block_table; max_pages * page_size <= 2^30 */
  int count;          /* entries of a list: pages to select, >= 1 */
  int keep_first;     /* first and last pages of a sequence that are always selected: */
  int keep_last;      /*   >= 0, keep_first + keep_last <= count */
} attn_sink_select_params;

/* Bytes of device workspace attn_sink_select_pages needs, on the current device (0 if
 * the params are invalid or there is nothing to do): the pages' scores. */
size_t attn_sink_select_pages_workspace_size(const attn_sink_select_params* params);

/*
 * For each sequence b and kv head h, with q [B, heads_q, 64] bf16 the new token's
 * queries, the score of page c (a column of the block table, c < N = ceil(seq_lens[b]
 * / page_size)) is
 *   max over the heads of h's group of  sum_d max(q_d, 0) bounds[page, h, 1, d]
 *                                           + min(q_d, 0) bounds[page, h, 0, d],
 * which no q.k of a key of the page exceeds.  Writes selected [B, heads_kv, count]
 * int32: columns in ascending order, -1 behind the last one: all N pages where N <=
 * count, else the keep_first first, the keep_last last and those of the largest
 * scores between them, of equal scores the lower columns.  Scores are compared as in
 * 64 bits: they are computed in 32, and those within the error of the last selected
 * one again in 64.  A NaN score counts as the largest, a page whose block-table
 * entry is outside the cache as the smallest.
 */
int attn_sink_select_pages(const attn_sink_select_params* params, const void* q,
                           const void* bounds, const int* block_table, const int* seq_lens,
                           int* selected, void* workspace, size_t workspace_bytes, void* stream);

typedef struct attn_sink_pages_params {
  int batch;          /* 0 <= B <= 65535 sequences; B * heads_q < 2^31 */
  int heads_q;        /* G * heads_kv with G in {1, 2, 4, 8} */
  int heads_kv;       /* 1 .. 65535 */
  int head_dim;       /* must be 64 */
  int page_size;      /* keys per page, >= 1 */
  int num_pages;      /* num_pages * page_size * heads_kv < 2^32 */
  int max_pages;      /* columns of block_table; max_pages * page_size <= 2^30 */
  int count;          /* entries of a list, >= 0; count * page_size <= 2^30 */
  float softmax_scale;/* multiplies q.k only; finite and > 0 */
} attn_sink_pages_params;

/* Bytes of device workspace attn_sink_decode_pages needs, on the current device (0 if
 * the params are invalid or there is nothing to do). */
size_t attn_sink_decode_pages_workspace_size(const attn_sink_pages_params* params);

/*
 * attn_sink_decode (without window and residual) over selected pages: the heads of kv
 * head h of sequence b see the keys j < seq_lens[b] of the pages selected[b, h, :]
 * (columns of the block table, as attn_sink_select_pages writes them).  Entries are
 * distinct, in any order; at most the first N = ceil(seq_lens[b] / page_size) of a
 * list are read.  A negative entry is no page, one of N or more is skipped and
 * recorded as 0x800.  A head that sees no key gets out = 0, lse = sink.  Layouts as
 * attn_sink_decode, arithmetic as the own keys of attn_sink_decode_shared.
 */
int attn_sink_decode_pages(const attn_sink_pages_params* params, const void* q,
                           const void* k_cache, const void* v_cache, const int* block_table,
                           const int* seq_lens, const int* selected, const float* sink, void* out,
                           float* lse, void* workspace, size_t workspace_bytes, void* stream);

typedef struct attn_sink_mass_params {
  int batch;          /* 0 <= B <= 65535 sequences */
  int total_q;        /* T <= 2^30: rows of q; cu_seqlens_q[B] <= T */
  int heads_q;        /* G * heads_kv with 1 <= G <= 128 */
  int heads_kv;       /* 1 .. 65535 */
  int head_dim;       /* must be 64 */
  int page_size;      /* keys per page, >= 1 */
  int num_pages;      /* num_pages * page_size * heads_kv < 2^32 */
  int max_pages;      /* columns of block_table; max_pages * page_size <= 2^30 */
  int max_keys;       /* 0 <= C <= 2^30: keys a row of mass has room for */
  int accumulate;     /* 1: added to mass; 0: mass is overwritten */
  float softmax_scale;/* finite and > 0 */
} attn_sink_mass_params;

/*
 * The weight each cached key got from the new tokens, summed over them and over the
 * query heads of its kv head:
 *   mass[b, h, j] (+)= sum over heads of h's group and tokens i of b that see key j
 *                      of exp(S_ij - lse_i)
 * with the causal S of attn_sink_extend (q [T, heads_q, 64] packed by cu_seqlens_q
 * [B + 1], the n_b last tokens of seq_lens[b] keys) and the lse [heads_q, T] that
 * attn_sink_extend, attn_sink_decode or any call above gave for these rows (an lse of
 * +-inf: no weight).  mass [B, heads_kv, C] fp32, one row of C keys for each kv head
 * of a row of the block table.  accumulate = 1 changes entries j < seq_lens[b] only;
 * 0 overwrites them and sets those behind to zero.  One of two kernels takes the whole
 * call: where the sequences have 32 rows of q (tokens times heads of a group) or fewer
 * on average, one that walks through a sequence's keys once for every 32 of its rows,
 * else one for prompts.  Single tokens and chunks of prompts belong in calls of their
 * own: 255 tokens on 1024 keys each take 53 us, one chunk of 512 on 16384 keys 111 us,
 * both in one call 36 ms.  The first kernel also takes prompts of groups of more than
 * 96 heads and of scales outside 2^-10 .. 2^10.  A sequence without new tokens
 * adds nothing.  Keys without a page get no weight.  seq_lens above C are clamped to C
 * for mass and recorded as 0x800: keys behind have no entry.  Scores multiply the bf16
 * inputs exactly; all sums are fp32 in a fixed order (of many tokens, the score's takes
 * the lse in as well).  No workspace; one launch.
 */
int attn_sink_key_mass(const attn_sink_mass_params* params, const void* q, const void* k_cache,
                       const int* block_table, const int* seq_lens, const int* cu_seqlens_q,
                       const float* lse, float* mass, void* stream);

typedef struct attn_sink_evict_params {
  int batch;          /* 0 <= B <= 65535 sequences */
  int heads_kv;       /* >= 1; B * heads_kv < 2^31 - 1 */
  int head_dim;       /* must be 64 */
  int page_size;      /* keys per page, >= 1 */
  int num_pages;      /* num_pages * page_size * heads_kv < 2^32 */
  int max_pages;      /* columns of block_table; max_pages * page_size <= 2^30, B * max_pages < 2^31 */
  int max_keys;       /* 0 <= C <= 2^30: keys a row of mass has room for */
  int budget;         /* keys that a sequence keeps at most, >= 0 */
  int keep_first;     /* first and last keys of a sequence that always stay: */
  int keep_last;      /*   >= 0, keep_first + keep_last <= budget */
  int max_freed;      /* entries of freed_pages, >= 0 */
} attn_sink_evict_params;

/* Bytes of device workspace attn_sink_evict needs (0 if the params are invalid or
 * there is nothing to do): which rows move where. */
size_t attn_sink_evict_workspace_size(const attn_sink_evict_params* params);

/*
 * Cuts every sequence down to budget keys, each kv head choosing its own: with L =
 * seq_lens[b] > budget, those of positions < keep_first, those of positions >= L -
 * keep_last, and of the rest the ones with the largest mass[b, h, :] (of equal ones
 * the lower positions; NaN counts as the largest).  The kept keys and values at
 * positions >= budget move, in order, into the places below that became free, in
 * order, in k_cache and v_cache; the others stay where they are.  A head's keys are
 * then no longer in the order of their tokens, which attention without a window does
 * not depend on; keep_last means the newest tokens as long as a sequence gets at least
 * keep_last new ones between two evictions.  Positions that were rotated into the keys
 * stay theirs; new tokens go on counting from the sequence's own length.
 * Writes mass_out [B, heads_kv, C] fp32, the kept keys' mass at their new places and
 * zero behind; new_lens [B] = min(L, budget); freed_pages [max_freed], the
 * block-table entries of pages that hold no key any more, sequence by sequence, in
 * the order of their columns, -1 behind the last (the free pages of
 * attn_sink_page_plan; block_table itself stays as it is; entries outside the cache
 * are left out and recorded); num_freed [1], how many there are (more than max_freed
 * when they do not fit).  Sequences of at most budget
 * keys, and the rows behind a sequence's new length, keep what they hold.  Pages that
 * hold any of a changed sequence's keys must be in no other sequence's row.
 * seq_lens above C are clamped and recorded as 0x800; where the block table has no
 * page for a key that moves, or for its new place, that move is left out and recorded.
 * mass and mass_out, and seq_lens and new_lens, must not overlap (the same pointer is
 * refused).
 */
int attn_sink_evict(const attn_sink_evict_params* params, void* k_cache, void* v_cache,
                    const int* block_table, const int* seq_lens, const float* mass,
                    float* mass_out, int* new_lens, int* freed_pages, int* num_freed,
                    void* workspace, size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* ATTN_SINK_CACHE_H */
