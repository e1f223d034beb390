/*
 * fp8rl_attn.h -- attention between the q/k/v linear and the output linear of a decoder block, in the
 * same library as fp8rl.h and fp8rl_block.h and under their conventions (device pointers, row pitches
 * in elements, all validation on the host before any HIP call, no allocation, no synchronization,
 * re-entrant, status codes, bf16 as uint16_t bit patterns, E4M3 codes as uint8_t, workspaces that
 * are overwritten and keep nothing from one call for the next):
 *
 *   serving     one new token of every sequence against the paged cache that fp8rl_rope_kv_append
 *               fills (fp8rl_attn_decode), and cached rows back as contiguous bf16 rows
 *               (fp8rl_kv_read), the prefix in front of a chunk of prompt.
 *
 * Heads. Rows hold their heads side by side, head_dim columns each; kv_heads divides q_heads, and
 * q head h reads key head h / (q_heads / kv_heads).
 *
 * Which keys a query sees. A query at position p of its sequence sees key j of that sequence if
 *   j <= p and (window == 0 or p - j < window).
 * Its score for such a key is, with s = sm_scale <q, k>,
 *   a = c - slopes[h] |p - j|,     c = cap tanh(s / cap)   (s itself with cap == 0),
 * without the slopes' term where slopes is NULL, and out = sum_j softmax(a)_j v_j. A query that sees
 * no key gives zeros.
 */
#ifndef FP8RL_ATTN_H
#define FP8RL_ATTN_H

#include "fp8rl.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Arguments of fp8rl_attn_decode (a HOST struct, read during the call only). */
typedef struct {
  const void* q; /* [B][ld_q]: q_heads * head_dim columns, bf16, or E4M3 codes where q_scale is given */
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
  const int32_t* lengths; /* [B]: a sequence's cached keys, that of the query's own token included */
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
 * A length counts as at most table_width * page_size, and as 0 where it is negative. A key whose page
 * lies outside [0, num_pages) is not seen. What the cache holds in places that are not seen (behind
 * a sequence's end, before its window) is of no consequence, NaN and infinities included.
 * Sums and statistics are float32. The weights are rounded to fp16 for the products with an E4M3
 * cache's values; for a bf16 cache's they are split in two bf16 terms (16 bits). out is
 * rounded once. Deterministic; the split of a sequence's keys over workgroups follows from all the
 * lengths of the call, so a sequence's last bits can change with its neighbours.
 *   workspace : at least fp8rl_attn_decode_workspace_bytes(...) bytes, 16-byte aligned, overwritten;
 *               may be NULL when that is 0
 * Requires head_dim % 16 == 0, 16 <= head_dim <= 256, 1 <= kv_heads, q_heads a multiple of kv_heads,
 * q_heads <= 4096, B <= 65536, B * kv_heads * ceil(q_heads / kv_heads / 16) < 2^22, page_size >= 1,
 * table_width * page_size <= 2^30, num_pages * page_size < 2^62, sm_scale finite, window >= 0, cap
 * finite and >= 0; bf16 pointers 16-byte and codes 8-byte aligned, pitches and strides multiples of 8
 * elements, ld_q, ld_out >= the columns, ld_table >= table_width, page_stride (with more than one
 * page), slot_stride and head_stride >= head_dim. B == 0 returns FP8RL_OK.
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
 * float32 and rounded once. Rows that belong to no sequence, and those of keys that the table or the
 * cache does not have, are left as they were.
 * Requires head_dim % 8 == 0, 8 <= head_dim <= 512, 1 <= kv_heads <= 65536, R < 2^24, B < 2^20 and
 * for the caches, the table and the alignment what fp8rl_attn_decode does; ld_k, ld_v multiples of 8
 * and >= the columns. R == 0 or B == 0 returns FP8RL_OK.
 */
fp8rl_status fp8rl_kv_read(const fp8rl_kv_read_args* args, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* FP8RL_ATTN_H */
