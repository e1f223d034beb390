/*
 * fp8rl_attn.h -- attention between the q/k/v linear and the output linear of a decoder block, in
 * the same library as fp8rl.h and fp8rl_block.h and under their conventions (device pointers, row
 * pitches in elements, all validation on the host before any HIP call, no allocation, no
 * synchronization, re-entrant, status codes, bf16 as uint16_t bit patterns, E4M3 codes as uint8_t,
 * workspaces that are overwritten and keep nothing from one call for the next):
 *
 *   serving     one new token of every sequence against the paged cache that fp8rl_rope_kv_append
 *               fills (fp8rl_attn_decode), and cached rows back as contiguous bf16 rows
 *               (fp8rl_kv_read), the prefix in front of a chunk of prompt;
 *   documents   packed queries against packed keys (fp8rl_attn_fwd), prompts as well as training,
 *               and the gradients (fp8rl_attn_bwd).
 *
 * Heads. Rows hold their heads side by side, head_dim columns each; kv_heads divides q_heads, and
 * q head h reads key head h / (q_heads / kv_heads).
 *
 * Which keys a query sees. A query at position p of its sequence sees key j of that sequence if
 *   (not causal or j <= p) and (window == 0 or p - j < window),   or if   j < prefix.
 * Its score for such a key is, with s = sm_scale <q, k>,
 *   a = c - slopes[h] |p - j|,     c = cap tanh(s / cap)   (s itself with cap == 0),
 * without the slopes' term where slopes is NULL, and out = sum_j softmax(a)_j v_j. A query that
 * sees no key gives zeros.
 *
 * Outputs and workspaces overlap no input and not one another; outputs may be columns of one row.
 */
#ifndef FP8RL_ATTN_H
#define FP8RL_ATTN_H

#include "fp8rl.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Arguments of fp8rl_attn_decode (a HOST struct, read during the call only). */
typedef struct {
  const void* q; /* [B][ld_q]: q_heads * head_dim columns, bf16, or E4M3 codes with q_scale */
  int64_t ld_q;
  const float* q_scale; /* one float32 (device), or NULL */
  int64_t B;            /* sequences, one query each */
  int32_t q_heads, kv_heads, head_dim;
  const void* k_cache; /* bf16, or E4M3 codes where k_scale and v_scale are given */
  const void* v_cache;
  const float* k_scale; /* one float32 each (device), both or neither */
  const float* v_scale;
  int64_t num_pages;
  int32_t page_size;
  int64_t page_stride, slot_stride, head_stride; /* elements, of both caches */
  const int32_t* page_table; /* [B][ld_table]: the page of keys i * page_size .. of a sequence */
  int64_t ld_table;
  int32_t table_width;    /* entries of a row of the table */
  const int32_t* lengths; /* [B]: a sequence's cached keys, its query's own among them */
  float sm_scale;
  int32_t window; /* 0: none */
  float cap;      /* 0: none */
  const float* slopes; /* [q_heads] float32, or NULL */
  uint16_t* out;       /* bf16 [B][ld_out] */
  int64_t ld_out;
} fp8rl_attn_decode_args;

/*
 * Attention of one query per sequence over the paged cache: causal, the query at position
 * p = lengths[b] - 1. Key j of sequence b is row
 *   cache + page * page_stride + place * slot_stride + head * head_stride,
 *   page = page_table[b][j / page_size], place = j % page_size
 * of either cache, as fp8rl_rope_kv_append stores it. Stored E4M3 codes count as code * scale.
 * A length counts as at most table_width * page_size, and as 0 where it is negative. A key whose
 * page lies outside [0, num_pages) is not seen. What the cache holds in places that are not seen
 * (behind a sequence's end, before its window) is of no consequence, NaN and infinities included.
 * Sums and statistics are float32. For their products with the values the weights are split in two
 * bf16 terms (16 bits, however small a weight is beside the largest). out is rounded once. Deterministic; where sequences are split over waves, the cuts follow from all the lengths
 * of the call, so that a sequence's last bits can change with its neighbours.
 *   workspace : at least fp8rl_attn_decode_workspace_bytes(...) bytes, 16-byte aligned,
 *               overwritten; may be NULL when that is 0
 * Requires head_dim % 16 == 0, 16 <= head_dim <= 256, 1 <= kv_heads, q_heads a multiple of
 * kv_heads, q_heads <= 4096, B <= 65536, B * kv_heads * ceil(q_heads / kv_heads / 16) < 2^22,
 * page_size >= 1, table_width * page_size <= 2^30, B * table_width * page_size < 2^35,
 * num_pages * page_size < 2^62, |sm_scale| <= 2^60, window >= 0, cap 0 or within 2^-60 .. 2^60;
 * bf16 pointers 16-byte and codes 8-byte aligned, pitches and strides multiples of 8 elements,
 * ld_q, ld_out >= the columns, ld_table >= table_width, page_stride (with more than one page),
 * slot_stride and head_stride >= head_dim. B == 0 returns FP8RL_OK.
 */
fp8rl_status fp8rl_attn_decode(const fp8rl_attn_decode_args* args, void* workspace,
                               size_t workspace_bytes, void* stream);

/* Bytes of workspace fp8rl_attn_decode needs for up to max_keys = table_width * page_size keys of a
 * sequence (0 where no sequence is split). Host-only. */
size_t fp8rl_attn_decode_workspace_bytes(int64_t B, int32_t q_heads, int32_t kv_heads,
                                         int32_t head_dim, int64_t max_keys, int32_t window);

/* Arguments of fp8rl_kv_read (a HOST struct, read during the call only). */
typedef struct {
  const void* k_cache; /* the caches as in fp8rl_attn_decode_args */
  const void* v_cache;
  const float* k_scale;
  const float* v_scale;
  int64_t num_pages;
  int32_t page_size;
  int64_t page_stride, slot_stride, head_stride;
  int32_t kv_heads, head_dim;
  const int32_t* page_table;
  int64_t ld_table;
  int32_t table_width;
  int64_t B;
  const int32_t* offsets; /* [B + 1], not decreasing: sequence b's rows of the outputs */
  const int32_t* starts;  /* [B]: the key that a sequence's first row holds; NULL: key 0 */
  int64_t R;              /* rows of the outputs */
  uint16_t* k_out;        /* bf16 [R][ld_k]: kv_heads * head_dim columns */
  uint16_t* v_out;
  int64_t ld_k, ld_v;
} fp8rl_kv_read_args;

/*
 * Cached rows back in order: row offsets[b] + i of k_out and v_out is key starts[b] + i of sequence
 * b (as fp8rl_attn_decode finds it), a bf16 cache's as it is, E4M3 codes as code * scale, formed in
 * float32 and rounded once. Rows that belong to no sequence, and those of keys that the table or
 * the cache does not have, are left as they were.
 * Requires head_dim % 8 == 0, 8 <= head_dim <= 512, 1 <= kv_heads <= 65536, R < 2^24, B < 2^20 and
 * for the caches, the table and the alignment what fp8rl_attn_decode does; ld_k, ld_v multiples of
 * 8 and >= the columns. R == 0 or B == 0 returns FP8RL_OK.
 */
fp8rl_status fp8rl_kv_read(const fp8rl_kv_read_args* args, void* stream);

/* Arguments of fp8rl_attn_fwd and fp8rl_attn_bwd (a HOST struct, read during the call only). */
typedef struct {
  const uint16_t* q; /* bf16 [Tq][ld_q]: q_heads * head_dim columns */
  const uint16_t* k; /* bf16 [Tk][ld_k]: kv_heads * head_dim columns */
  const uint16_t* v; /* bf16 [Tk][ld_v] */
  int64_t ld_q, ld_k, ld_v;
  int64_t Tq, Tk;
  int32_t q_heads, kv_heads, head_dim;
  int64_t docs;
  const int32_t* q_offsets; /* [docs + 1], not decreasing: document d's queries are rows
                               q_offsets[d] .. q_offsets[d + 1] - 1 of q */
  const int32_t* k_offsets; /* [docs + 1]: its keys' rows of k and v */
  int32_t causal;
  int32_t window;         /* 0: none */
  const int32_t* prefix;  /* [docs], or NULL (none) */
  float sm_scale;
  float cap;              /* 0: none */
  const float* slopes;    /* [q_heads] float32, or NULL */
  uint16_t* out;          /* bf16 [Tq][ld_out]; written by fwd, read by bwd */
  int64_t ld_out;
  float* lse;             /* float32 [q_heads][Tq]: log sum_j exp(a_j), -inf where no key is seen;
                             written by fwd (NULL: not), read by bwd */
  const uint16_t* dout;   /* bf16 [Tq][ld_dout]: the gradient at out (bwd) */
  int64_t ld_dout;
  uint16_t* dq;           /* bf16 [Tq][ld_dq] (bwd) */
  uint16_t* dk;           /* bf16 [Tk][ld_dk] */
  uint16_t* dv;           /* bf16 [Tk][ld_dv] */
  int64_t ld_dq, ld_dk, ld_dv;
} fp8rl_attn_args;

/*
 * Attention of packed documents. With Lq queries and Lk keys, query i of a document is at position
 * p = i + Lk - Lq: the keys of a chunk of prompt may begin with those of the prefix that is cached
 * already. Rows that belong to no document are neither read nor written. Offsets outside [0, Tq] or
 * [0, Tk] count as the nearest bound.
 * Scores, statistics and sums are float32; the weights are rounded to bf16 for their product with
 * v; out is rounded once. Deterministic.
 * Values of v that are NaN or infinite reach rows of their document that do not see them (as
 * 0 * NaN does); they reach no other document.
 * Requires head_dim % 16 == 0, 16 <= head_dim <= 256, 1 <= kv_heads, q_heads a multiple of
 * kv_heads, q_heads <= 4096, Tq, Tk < 2^24, docs < 2^20,
 * (max(Tq, Tk) / 128 + docs) * q_heads < 2^24, past 128 columns (Tq / 128 + docs) * q_heads < 2^23,
 * 0 < sm_scale <= 2^60, window >= 0, cap 0 or within 2^-60 .. 2^60; 16-byte aligned rows, pitches
 * multiples of 8, >= the columns and < 2^24; offsets, prefix, lse and slopes 4-byte aligned.
 * Tq == 0 or docs == 0 returns FP8RL_OK.
 */
fp8rl_status fp8rl_attn_fwd(const fp8rl_attn_args* args, void* stream);

/*
 * Gradients of fp8rl_attn_fwd. With P = exp(a - lse), dP = <dout, v> and D = <dout, out>:
 *   dv_j = sum P dout,   dS = P (dP - D) (1 - (c / cap)^2),   dq_i = sm_scale sum_j dS k_j,
 *   dk_j = sm_scale sum dS q,
 * the sums for keys taken over the queries of all heads that share them. sm_scale, cap and slopes
 * are constants. Rows of dq, dk and dv that belong to no document are not written; keys that no
 * query sees get zeros. P and dS are rounded to bf16 for their products; sums are float32; each
 * result is rounded once. Deterministic: no atomics. Values of q, k, v and dout that are NaN or
 * infinite reach any row of their document, and no other document.
 *   workspace : at least fp8rl_attn_bwd_workspace_bytes(...) bytes, 16-byte aligned, overwritten
 * Requires what fp8rl_attn_fwd does, head_dim <= 128 and (Tk / 128 + docs) * kv_heads < 2^23. Tq == Tk
 * == 0 or docs == 0 returns FP8RL_OK.
 */
fp8rl_status fp8rl_attn_bwd(const fp8rl_attn_args* args, void* workspace, size_t workspace_bytes,
                            void* stream);

/* Bytes of workspace fp8rl_attn_bwd needs. Host-only. */
size_t fp8rl_attn_bwd_workspace_bytes(int64_t Tq, int64_t Tk, int64_t docs, int32_t q_heads,
                                      int32_t kv_heads, int32_t head_dim);

#ifdef __cplusplus
}
#endif

#endif /* FP8RL_ATTN_H */
