/*
 * fp8rl_block.h -- the operators between the FP8 linears of a decoder block, in the same library
 * as fp8rl.h and under its conventions (device pointers, row pitches in elements, all validation
 * on the host before any HIP call, no allocation, no synchronization, re-entrant, status codes,
 * bf16 as uint16_t bit patterns, E4M3 codes as uint8_t). They make what the linears read and take
 * what the linears write:
 *
 *   norm        the root-mean-square norm of the residual stream, with the addition that produces
 *               the stream and an E4M3 output with 1x128 scales, ready for
 *               fp8rl_gemm_w8a8_blockscaled (fp8rl_add_rmsnorm_quant), and its backward pass
 *               (fp8rl_add_rmsnorm_bwd);
 *   experts     the router's choices as the expert offsets and row ids that the grouped GEMMs read
 *               (fp8rl_moe_sort), the rows moved into that order (fp8rl_moe_dispatch), the
 *               experts' rows weighted and summed per token (fp8rl_moe_combine) and the gradients
 *               of that sum (fp8rl_moe_combine_bwd);
 *   KV cache    q and k normalised per head where the model does that, rotated by their positions,
 *               k and v stored into a paged cache (fp8rl_rope_kv_append).
 *
 * A workspace is overwritten and keeps nothing from one call for the next (no header to clear): any
 * memory of the size will do, and calls may share it that do not run at the same time.
 *
 * Where a result is said to be written "in place", the output may be the very memory (same pointer,
 * same pitch) of the named input; any other overlap of outputs with inputs is not allowed.
 */
#ifndef FP8RL_BLOCK_H
#define FP8RL_BLOCK_H

#include "fp8rl.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * Residual addition, root-mean-square norm and 1x128 quantization of M rows of K values:
 *   h[m][k]  = bf16(x[m][k] + residual[m][k])           (x itself without a residual)
 *   y[m][k]  = h[m][k] * weight[k] / sqrt(mean_k h[m][k]^2 + eps)
 *   sa[m][g] = scale of max |y[m][group g]| as fp8rl_quant_act_tok128_ex forms it (scale_fmt),
 *   xq[m][k] = E4M3 code nearest to y[m][k] / sa[m][k/128].
 * The stream h is rounded once, to bf16, and the norm is taken of that stored value, so that
 * fp8rl_add_rmsnorm_bwd, which reads h, differentiates this very function. y is never rounded on
 * its way to the codes: the result is closer to y than quantizing the bf16 rows would be. With
 * FP8RL_SCALE_FP32 the row's statistic cancels out of y / sa and the codes are those of the exact
 * quotients; the scales carry float32 rounding (a few units in the last place). With
 * FP8RL_SCALE_POW2 a scale may be the neighbouring power of two where the float32 value of
 * max |y| lies on the other side of 448 2^e than the exact one.
 *   x         : bf16, M rows of pitch ld_x (>= K)
 *   residual  : bf16, M rows of pitch ld_res, or NULL
 *   weight    : bf16, K values (dense)
 *   eps       : finite, a normal positive float32 (at least 2^-126)
 *   h         : bf16 [M][ld_h], or NULL (not written). Needs a residual. May be written in place of
 *               x or of residual.
 *   y         : bf16 [M][ld_y], the normalised rows rounded once, or NULL. (The router of a
 *               mixture-of-experts layer and a training step's weight gradients read these.)
 *   xq, sa    : codes [M][ld_xq] and scales, dense [M][K/128], or both NULL (then y is required)
 * Requires K % 128 == 0, K <= 32768, M < 2^22; bf16 pointers 16-byte aligned and their
 * pitches multiples of 8, xq 16-byte aligned and ld_xq a multiple of 16. A row whose sum of squares
 * is not finite in float32 (an infinity, a NaN, magnitudes past about 2^63) comes out with NaN
 * scales and NaN y. h * weight is formed in float32: weights below 2^60 (a product below 2^-126
 * loses bits). Deterministic.
 */
fp8rl_status fp8rl_add_rmsnorm_quant(const uint16_t* x, int64_t ld_x, const uint16_t* residual,
                                     int64_t ld_res, const uint16_t* weight, float eps, int64_t M,
                                     int64_t K, uint16_t* h, int64_t ld_h, uint16_t* y,
                                     int64_t ld_y, uint8_t* xq, int64_t ld_xq, float* sa,
                                     int scale_fmt, void* stream);

/*
 * Backward pass of the norm and its addition. With r[m] = 1 / sqrt(mean_k h[m][k]^2 + eps):
 *   dx[m][k] = r[m] (dy[m][k] weight[k] - h[m][k] r[m]^2 mean_j(dy[m][j] weight[j] h[m][j]))
 *              + dh[m][k]
 *   dw[k]    = sum_m dy[m][k] h[m][k] r[m]
 * dx is the gradient of the stream, hence of x and of residual alike. dy is the gradient at the
 * norm's output (the quantization passes it through unchanged); dh the gradient that reaches the
 * stream from the blocks behind (NULL: none). The statistic is recomputed from h. Sums are held in
 * float32, dx is rounded once.
 *   dy, h, dh, dx : bf16, M rows of pitch ld_*; dx may be written in place of dy or of dh
 *   weight        : bf16, K values
 *   dw            : float32, K values, overwritten (zeros when M == 0), or NULL (not computed)
 *   workspace     : at least fp8rl_add_rmsnorm_bwd_workspace_bytes(M, K) bytes, 16-byte aligned,
 *                   overwritten; may be NULL when dw is
 * Requires K % 128 == 0, K <= 32768, M < 2^22; alignment as for fp8rl_add_rmsnorm_quant (dw
 * 4-byte).
 * Deterministic: the sum over rows has a fixed order.
 */
fp8rl_status fp8rl_add_rmsnorm_bwd(const uint16_t* dy, int64_t ld_dy, const uint16_t* h,
                                   int64_t ld_h, const uint16_t* weight, const uint16_t* dh,
                                   int64_t ld_dh, float eps, int64_t M, int64_t K, uint16_t* dx,
                                   int64_t ld_dx, float* dw, void* workspace,
                                   size_t workspace_bytes, void* stream);

/* Bytes of workspace fp8rl_add_rmsnorm_bwd needs to compute dw. Host-only. */
size_t fp8rl_add_rmsnorm_bwd_workspace_bytes(int64_t M, int64_t K);

/* Type of the router's choices. */
typedef enum { FP8RL_IDS_I32 = 0, FP8RL_IDS_I64 = 1 } fp8rl_ids_dtype;

/*
 * The router's choices in expert order. Choice (t, j) is the j-th expert of token t. Choices of
 * expert 0 come first, then those of expert 1, ...; those of one expert by increasing (t, j).
 *   topk_ids       : dense [T][top_k] expert ids of type ids_dtype. An id outside [0, E) -- by
 *                    convention -1, an expert that lives on another rank -- gets no grouped row. A
 *                    token may name the same expert twice (two grouped rows).
 *   expert_offsets : E+1 int32: expert e owns grouped rows expert_offsets[e] ..
 *                    expert_offsets[e+1]-1 (the array fp8rl_grouped_gemm_w8a8 reads)
 *   row_ids        : T * top_k int32: the token of each grouped row (the array
 *                    fp8rl_grouped_gemm_w8a8_fused_act_quant reads); -1 from row
 *                    expert_offsets[E] on
 *   pos            : [T][top_k] int32: the grouped row of each choice, -1 where it has none
 *   workspace      : at least fp8rl_moe_sort_workspace_bytes(T, top_k, E) bytes, 16-byte aligned,
 *                    overwritten; may be NULL when that is 0
 * Requires 1 <= E <= 1024, 1 <= top_k <= 64, T < 2^24. T == 0 writes expert_offsets
 * (zeros). Deterministic.
 */
fp8rl_status fp8rl_moe_sort(const void* topk_ids, int ids_dtype, int64_t T, int32_t top_k,
                            int32_t E, int32_t* expert_offsets, int32_t* row_ids, int32_t* pos,
                            void* workspace, size_t workspace_bytes, void* stream);

/* Bytes of workspace fp8rl_moe_sort needs (0 where one workgroup does it). Host-only. */
size_t fp8rl_moe_sort_workspace_bytes(int64_t T, int32_t top_k, int32_t E);

/*
 * Token rows moved into expert order: out[pos[t][j]] = x[t] for every choice with
 * 0 <= pos[t][j] < R; other choices move nothing, and rows of out that no choice names are left as
 * they were. The gradient of x is fp8rl_moe_combine of the gradient of out, without weights.
 * (The grouped GEMM on bf16 activations reads token rows through row_ids and needs no moved copy;
 * this is for what does, e.g. an expert's weight gradient.)
 *   x   : bf16 [T][ld_x]          pos : [T][top_k] int32, its rows distinct (fp8rl_moe_sort's)
 *   out : bf16 [R][ld_out], not overlapping x
 * Requires N % 8 == 0, pitches multiples of 8 and >= N, 16-byte aligned rows, 1 <= top_k <= 64,
 * T < 2^24, T * ceil(N / 2048) <= 2^26 - 4.
 */
fp8rl_status fp8rl_moe_dispatch(const uint16_t* x, int64_t ld_x, const int32_t* pos, int64_t T,
                                int32_t top_k, int64_t N, uint16_t* out, int64_t R, int64_t ld_out,
                                void* stream);

/*
 * The experts' rows back in token order, weighted and summed:
 *   out[t][n] = sum_j weights[t][j] * y[pos[t][j]][n]   over the j with 0 <= pos[t][j] < R,
 * added in float32 by increasing j and rounded once; a token without such a j gets zeros.
 *   y        : [R][ld_y] of y_dtype (fp8rl_out_dtype), the down projection's output
 *   pos      : [T][top_k] int32
 *   weights  : [T][top_k] float32, or NULL (every weight 1)
 *   out      : [T][ld_out] of out_dtype (fp8rl_out_dtype), not overlapping y
 * Requires N % 8 == 0, pitches >= N and multiples of 8, 16-byte aligned rows, 1 <= top_k <= 64,
 * T < 2^24.
 */
fp8rl_status fp8rl_moe_combine(const void* y, int y_dtype, int64_t R, int64_t ld_y,
                               const int32_t* pos, const float* weights, int64_t T, int32_t top_k,
                               int64_t N, void* out, int out_dtype, int64_t ld_out, void* stream);

/*
 * Gradients of fp8rl_moe_combine, for the choices with 0 <= pos[t][j] < R:
 *   dy[pos[t][j]][n] = weights[t][j] * dout[t][n]             (rounded once)
 *   dweights[t][j]   = sum_n dout[t][n] * y[pos[t][j]][n]     (float32; 0 for the other choices)
 * Rows of dy that no choice names are left as they were.
 *   dout     : bf16 [T][ld_dout]
 *   y, dy    : [R][ld_y] and [R][ld_dy] of y_dtype; y and dweights both given or both NULL; dy may
 *              be written in place of y
 *   weights  : [T][top_k] float32, or NULL (every weight 1)
 *   dweights : [T][top_k] float32, dense
 * The rows named by pos must be distinct (fp8rl_moe_sort's are). Requires what fp8rl_moe_combine
 * does. Deterministic.
 */
fp8rl_status fp8rl_moe_combine_bwd(const uint16_t* dout, int64_t ld_dout, const void* y,
                                   int64_t ld_y, int y_dtype, int64_t R, const int32_t* pos,
                                   const float* weights, int64_t T, int32_t top_k, int64_t N,
                                   void* dy, int64_t ld_dy, float* dweights, void* stream);

/* Arguments of fp8rl_rope_kv_append (a HOST struct, read during the call only). */
typedef struct {
  const uint16_t* q; /* bf16 [T][ld_q]: q_heads * head_dim columns; NULL when q_heads == 0 */
  const uint16_t* k; /* bf16 [T][ld_k]: kv_heads * head_dim columns */
  const uint16_t* v; /* bf16 [T][ld_v]: kv_heads * head_dim columns */
  int64_t ld_q, ld_k, ld_v;
  int64_t T;
  int32_t q_heads, kv_heads, head_dim;
  int32_t rot_dim;     /* columns of a head that are rotated: 0 <= rot_dim <= head_dim */
  int32_t interleaved; /* 0: column i turns with column i + rot_dim/2; 1: column 2i with 2i + 1 */
  float eps;           /* of the head norms; not read without them */
  const int64_t* positions; /* [T] */
  const float* cos_sin; /* [max_pos][rot_dim]: the cosines of a position's rot_dim/2 angles, then
                           their sines; NULL when rot_dim == 0 */
  int64_t max_pos;
  const uint16_t* q_weight; /* bf16 [head_dim]: per-head norm weights; both or neither */
  const uint16_t* k_weight;
  void* q_out;          /* [T][ld_qo]: bf16, or E4M3 codes where q_scale is given */
  int64_t ld_qo;
  const float* q_scale; /* one float32 (device; positive, finite), or NULL */
  const int64_t* slot_mapping; /* [T]: page * page_size + place in the page; negative: no store */
  void* k_cache;        /* bf16, or E4M3 codes where k_scale and v_scale are given */
  void* v_cache;
  const float* k_scale; /* one float32 each (device), both or neither */
  const float* v_scale;
  int64_t num_pages;
  int32_t page_size;
  int64_t page_stride, slot_stride, head_stride; /* elements, of both caches */
} fp8rl_rope_kv_args;

/*
 * New tokens' q, k and v on their way from the q/k/v linear into attention: with x one head of one
 * token,
 *   u = x * weight / sqrt(mean(x^2) + eps)     (q and k, where q_weight and k_weight are given)
 *   w[a] = u[a] cos - u[b] sin,  w[b] = u[b] cos + u[a] sin     for every rotated pair (a, b)
 * rounded once: to bf16 (formed in float32), or to the E4M3 code nearest to w / scale, ties to the
 * even one (formed in float64: a quotient that lies within 2^-48 of its size from a tie may round
 * as the tie; columns that are not rotated, and v, as fp8rl_quant_bf16_per_tensor rounds them)
 * (saturating). q goes to q_out, k (and v, neither normalised nor rotated) to row
 *   cache + page * page_stride + place * slot_stride + head * head_stride,
 *   page = slot / page_size, place = slot % page_size,
 * so pages may be laid out token by token, head by head, or with keys and values interleaved. A
 * token whose slot is negative or past the last page stores nothing; one whose position lies
 * outside [0, max_pos) (with rot_dim > 0) is skipped altogether, q included. Every byte that no
 * token names is left as it was. Slots must be distinct (of two tokens with one slot, either may be
 * kept, piece by piece).
 * bf16 q_out may be written in place of q.
 * Requires head_dim % 8 == 0, 8 <= head_dim <= 512, rot_dim % 16 == 0, kv_heads >= 1,
 * page_size >= 1, num_pages * page_size < 2^62, T * (q_heads + 2 kv_heads) < 2^25, eps as for
 * fp8rl_add_rmsnorm_quant where norms are given; bf16 pointers 16-byte and codes 8-byte aligned,
 * the table 16-byte, pitches and strides multiples of 8 elements, ld_* >= the columns, page_stride
 * (with more than one page), slot_stride and head_stride >= head_dim. A NaN stores a NaN code. The
 * head norms take any finite bf16 x (weights below 2^60; x * weight is formed in float32, where a
 * product below 2^-126 loses bits); a normalised head that holds an infinity or a NaN comes out as
 * NaN in every column.
 * T == 0 returns FP8RL_OK.
 */
fp8rl_status fp8rl_rope_kv_append(const fp8rl_rope_kv_args* args, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* FP8RL_BLOCK_H */
