// C ABI entry points of attention: argument validation (host only, before any HIP call) and
// dispatch.
#include <math.h>
#include <stdint.h>

#include "attn_ops.hpp"
#include "fp8rl_attn.h"

namespace {

constexpr int64_t kMaxDim = (int64_t{1} << 31) - 1;

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
fp8rl_status hip_status(hipError_t e) { return e == hipSuccess ? FP8RL_OK : FP8RL_ERR_HIP; }
hipStream_t as_stream(void* s) { return reinterpret_cast<hipStream_t>(s); }

// A matrix of rows of n values: FP8RL_OK when laid out as required.
fp8rl_status check_rows(const void* p, int64_t ld, int64_t n, uintptr_t align = 16) {
  if (ld < n || ld > kMaxDim) return FP8RL_ERR_SHAPE;
  if (!aligned(p, align) || ld % 8) return FP8RL_ERR_ALIGN;
  return FP8RL_OK;
}

// What both readers of a paged cache ask of it and of the page table (a cache of no pages is not
// looked at).
struct Cache {
  const void *k, *v;
  const float *k_scale, *v_scale;
  int64_t num_pages;
  int32_t page_size;
  int64_t page_stride, slot_stride, head_stride;
  int32_t kv_heads, head_dim;
  const int32_t* table;
  int64_t ld_table;
  int32_t table_width;
};

template <typename Args>
Cache cache_of(const Args& a) {
  return {a.k_cache,     a.v_cache,     a.k_scale,     a.v_scale,  a.num_pages,
          a.page_size,   a.page_stride, a.slot_stride, a.head_stride, a.kv_heads,
          a.head_dim,    a.page_table,  a.ld_table,    a.table_width};
}

fp8rl_status check_cache_shape(const Cache& c) {
  if (c.num_pages < 0 || c.page_size < 1 || c.num_pages >= (int64_t{1} << 62) / c.page_size)
    return FP8RL_ERR_SHAPE;
  if (c.table_width < 0 || (int64_t)c.table_width * c.page_size > (int64_t{1} << 30))
    return FP8RL_ERR_SHAPE;
  if (c.kv_heads < 1 || c.kv_heads > 65536) return FP8RL_ERR_SHAPE;
  if ((!c.k_scale) != (!c.v_scale)) return FP8RL_ERR_NULL;
  return FP8RL_OK;
}

fp8rl_status check_cache(const Cache& c) {
  if (c.table_width > 0) {
    if (!c.table) return FP8RL_ERR_NULL;
    if (c.ld_table < c.table_width || c.ld_table > kMaxDim) return FP8RL_ERR_SHAPE;
    if (!aligned(c.table, 4)) return FP8RL_ERR_ALIGN;
  }
  if (!aligned(c.k_scale, 4) || !aligned(c.v_scale, 4)) return FP8RL_ERR_ALIGN;
  if (c.num_pages == 0) return FP8RL_OK;
  if (!c.k || !c.v) return FP8RL_ERR_NULL;
  if (c.slot_stride < c.head_dim || c.head_stride < c.head_dim ||
      c.page_stride < (c.num_pages > 1 ? c.head_dim : 0))
    return FP8RL_ERR_SHAPE;
  // offsets of any row of the cache, in bytes, stay inside 63 bits
  constexpr int64_t kFar = int64_t{1} << 60;
  if (c.slot_stride > kFar / c.page_size || c.page_stride > kFar / c.num_pages ||
      c.head_stride > kFar / c.kv_heads)
    return FP8RL_ERR_SHAPE;
  const uintptr_t align = c.k_scale ? 8 : 16;
  if (!aligned(c.k, align) || !aligned(c.v, align) || c.page_stride % 8 || c.slot_stride % 8 ||
      c.head_stride % 8)
    return FP8RL_ERR_ALIGN;
  return FP8RL_OK;
}

fp8rl_status check_heads(int32_t q_heads, int32_t kv_heads, int32_t head_dim, int32_t widest) {
  if (kv_heads < 1 || q_heads < kv_heads || q_heads > 4096 || q_heads % kv_heads)
    return FP8RL_ERR_SHAPE;
  if (head_dim < 16 || head_dim > widest || head_dim % 16) return FP8RL_ERR_SHAPE;
  return FP8RL_OK;
}

fp8rl_status check_scores(float sm_scale, int32_t window, float cap) {
  constexpr float kFar = 0x1p60f;  // their products with log2(e) and with one another stay finite
  if (!(fabsf(sm_scale) <= kFar) || window < 0) return FP8RL_ERR_ARG;
  if (cap != 0.f && !(cap >= 1.f / kFar && cap <= kFar)) return FP8RL_ERR_ARG;
  return FP8RL_OK;
}

// Workgroups that one piece of every sequence takes.
int64_t decode_items(int64_t B, int32_t q_heads, int32_t kv_heads) {
  return B * kv_heads * ((q_heads / kv_heads + 15) / 16);
}

fp8rl_status check_decode_shape(int64_t B, int32_t q_heads, int32_t kv_heads, int32_t head_dim) {
  if (B < 0 || B > 65536) return FP8RL_ERR_SHAPE;
  if (fp8rl_status s = check_heads(q_heads, kv_heads, head_dim, 256)) return s;
  if (decode_items(B, q_heads, kv_heads) >= (int64_t{1} << 22)) return FP8RL_ERR_SHAPE;
  return FP8RL_OK;
}

}  // namespace

extern "C" {

size_t fp8rl_attn_decode_workspace_bytes(int64_t B, int32_t q_heads, int32_t kv_heads,
                                         int32_t head_dim, int64_t max_keys, int32_t window) {
  if (check_decode_shape(B, q_heads, kv_heads, head_dim) != FP8RL_OK || max_keys < 0 ||
      max_keys > (int64_t{1} << 30) || window < 0)
    return 0;
  return fp8rl::attn_decode_workspace(B, q_heads, kv_heads, head_dim, max_keys, window);
}

fp8rl_status fp8rl_attn_decode(const fp8rl_attn_decode_args* args, void* workspace,
                               size_t workspace_bytes, void* stream) {
  if (!args) return FP8RL_ERR_NULL;
  const fp8rl_attn_decode_args& a = *args;
  const Cache c = cache_of(a);
  if (fp8rl_status s = check_decode_shape(a.B, a.q_heads, a.kv_heads, a.head_dim)) return s;
  if (fp8rl_status s = check_cache_shape(c)) return s;
  if (fp8rl_status s = check_scores(a.sm_scale, a.window, a.cap)) return s;
  // (the units of all sequences are counted in 32 bits)
  if (a.B * ((int64_t)a.table_width * a.page_size) >= int64_t{1} << 35) return FP8RL_ERR_SHAPE;
  if (a.B == 0) return FP8RL_OK;
  if (!a.q || !a.lengths || !a.out) return FP8RL_ERR_NULL;
  if (fp8rl_status s = check_cache(c)) return s;
  const int64_t cols = (int64_t)a.q_heads * a.head_dim;
  if (fp8rl_status s = check_rows(a.q, a.ld_q, cols, a.q_scale ? 8 : 16)) return s;
  if (fp8rl_status s = check_rows(a.out, a.ld_out, cols)) return s;
  if (!aligned(a.lengths, 4) || !aligned(a.q_scale, 4) || !aligned(a.slopes, 4))
    return FP8RL_ERR_ALIGN;
  const size_t need = fp8rl::attn_decode_workspace(
      a.B, a.q_heads, a.kv_heads, a.head_dim, (int64_t)a.table_width * a.page_size, a.window);
  if (need > 0) {
    if (!workspace || workspace_bytes < need) return FP8RL_ERR_WORKSPACE;
    if (!aligned(workspace, 16)) return FP8RL_ERR_ALIGN;
  }
  return hip_status(fp8rl::launch_attn_decode(a, workspace, as_stream(stream)));
}

fp8rl_status fp8rl_kv_read(const fp8rl_kv_read_args* args, void* stream) {
  if (!args) return FP8RL_ERR_NULL;
  const fp8rl_kv_read_args& a = *args;
  const Cache c = cache_of(a);
  if (a.R < 0 || a.R >= (int64_t{1} << 24) || a.B < 0 || a.B >= (int64_t{1} << 20))
    return FP8RL_ERR_SHAPE;
  if (a.head_dim < 8 || a.head_dim > 512 || a.head_dim % 8) return FP8RL_ERR_SHAPE;
  if (fp8rl_status s = check_cache_shape(c)) return s;
  if (a.R == 0 || a.B == 0) return FP8RL_OK;
  if (!a.offsets || !a.k_out || !a.v_out) return FP8RL_ERR_NULL;
  if (fp8rl_status s = check_cache(c)) return s;
  const int64_t cols = (int64_t)a.kv_heads * a.head_dim;
  if (fp8rl_status s = check_rows(a.k_out, a.ld_k, cols)) return s;
  if (fp8rl_status s = check_rows(a.v_out, a.ld_v, cols)) return s;
  if (!aligned(a.offsets, 4) || !aligned(a.starts, 4)) return FP8RL_ERR_ALIGN;
  if (a.num_pages == 0 || a.table_width == 0) return FP8RL_OK;  // no row is there
  return hip_status(fp8rl::launch_kv_read(a, as_stream(stream)));
}

namespace {

constexpr int64_t kMaxPitch = int64_t{1} << 24;  // 128 rows are less than 2^32 bytes apart
// A dispatch has fewer than 2^32 threads: so many workgroups of 256, and of 512, are past it.
constexpr int64_t kMax256 = int64_t{1} << 24, kMax512 = int64_t{1} << 23;

fp8rl_status check_attn_sizes(int64_t Tq, int64_t Tk, int64_t docs, int32_t q_heads,
                              int32_t kv_heads, int32_t head_dim, int32_t widest) {
  constexpr int64_t kRows = int64_t{1} << 24;
  if (Tq < 0 || Tk < 0 || Tq >= kRows || Tk >= kRows) return FP8RL_ERR_SHAPE;
  if (docs < 0 || docs >= (int64_t{1} << 20)) return FP8RL_ERR_SHAPE;
  if (fp8rl_status s = check_heads(q_heads, kv_heads, head_dim, widest)) return s;
  if (((Tq > Tk ? Tq : Tk) / 128 + docs) * q_heads >= kMax256) return FP8RL_ERR_SHAPE;
  return FP8RL_OK;
}

fp8rl_status check_bwd_sizes(int64_t Tq, int64_t Tk, int64_t docs, int32_t q_heads,
                             int32_t kv_heads, int32_t head_dim) {
  if (fp8rl_status s = check_attn_sizes(Tq, Tk, docs, q_heads, kv_heads, head_dim, 128)) return s;
  // (dk's and dv's workgroups have 512 threads)
  return (Tk / 128 + docs) * kv_heads < kMax512 ? FP8RL_OK : FP8RL_ERR_SHAPE;
}

fp8rl_status check_attn_scores(const fp8rl_attn_args& a) {
  if (a.causal != 0 && a.causal != 1) return FP8RL_ERR_ARG;
  if (fp8rl_status s = check_scores(a.sm_scale, a.window, a.cap)) return s;
  return a.sm_scale > 0.f ? FP8RL_OK : FP8RL_ERR_ARG;
}

fp8rl_status check_attn_rows(const void* p, int64_t ld, int64_t n) {
  if (!p) return FP8RL_ERR_NULL;
  return ld >= kMaxPitch ? FP8RL_ERR_SHAPE : check_rows(p, ld, n);
}

// What both passes read (and fwd writes).
fp8rl_status check_attn_inputs(const fp8rl_attn_args& a) {
  const int64_t qc = (int64_t)a.q_heads * a.head_dim, kc = (int64_t)a.kv_heads * a.head_dim;
  if (!a.q_offsets || !a.k_offsets) return FP8RL_ERR_NULL;
  if (fp8rl_status s = check_attn_rows(a.q, a.ld_q, qc)) return s;
  if (fp8rl_status s = check_attn_rows(a.out, a.ld_out, qc)) return s;
  if (a.Tk > 0) {
    if (fp8rl_status s = check_attn_rows(a.k, a.ld_k, kc)) return s;
    if (fp8rl_status s = check_attn_rows(a.v, a.ld_v, kc)) return s;
  }
  if (!aligned(a.q_offsets, 4) || !aligned(a.k_offsets, 4) || !aligned(a.prefix, 4) ||
      !aligned(a.slopes, 4) || !aligned(a.lse, 4))
    return FP8RL_ERR_ALIGN;
  return FP8RL_OK;
}

}  // namespace

fp8rl_status fp8rl_attn_fwd(const fp8rl_attn_args* args, void* stream) {
  if (!args) return FP8RL_ERR_NULL;
  const fp8rl_attn_args& a = *args;
  if (fp8rl_status s =
          check_attn_sizes(a.Tq, a.Tk, a.docs, a.q_heads, a.kv_heads, a.head_dim, 256))
    return s;
  // (heads past 128 columns: workgroups of 512 threads)
  if (a.head_dim > 128 && (a.Tq / 128 + a.docs) * a.q_heads >= kMax512) return FP8RL_ERR_SHAPE;
  if (fp8rl_status s = check_attn_scores(a)) return s;
  if (a.Tq == 0 || a.docs == 0) return FP8RL_OK;
  if (fp8rl_status s = check_attn_inputs(a)) return s;
  return hip_status(fp8rl::launch_attn_fwd(a, as_stream(stream)));
}

size_t fp8rl_attn_bwd_workspace_bytes(int64_t Tq, int64_t Tk, int64_t docs, int32_t q_heads,
                                      int32_t kv_heads, int32_t head_dim) {
  if (check_bwd_sizes(Tq, Tk, docs, q_heads, kv_heads, head_dim) != FP8RL_OK) return 0;
  return fp8rl::attn_bwd_workspace(Tq, Tk, docs, q_heads, kv_heads, head_dim);
}

fp8rl_status fp8rl_attn_bwd(const fp8rl_attn_args* args, void* workspace, size_t workspace_bytes,
                            void* stream) {
  if (!args) return FP8RL_ERR_NULL;
  const fp8rl_attn_args& a = *args;
  if (fp8rl_status s = check_bwd_sizes(a.Tq, a.Tk, a.docs, a.q_heads, a.kv_heads, a.head_dim))
    return s;
  if (fp8rl_status s = check_attn_scores(a)) return s;
  if ((a.Tq == 0 && a.Tk == 0) || a.docs == 0) return FP8RL_OK;
  const int64_t qc = (int64_t)a.q_heads * a.head_dim, kc = (int64_t)a.kv_heads * a.head_dim;
  if (!a.q_offsets || !a.k_offsets) return FP8RL_ERR_NULL;
  if (a.Tq > 0) {
    if (fp8rl_status s = check_attn_inputs(a)) return s;
    if (!a.lse) return FP8RL_ERR_NULL;
    if (fp8rl_status s = check_attn_rows(a.dout, a.ld_dout, qc)) return s;
    if (fp8rl_status s = check_attn_rows(a.dq, a.ld_dq, qc)) return s;
  }
  if (a.Tk > 0) {
    if (fp8rl_status s = check_attn_rows(a.k, a.ld_k, kc)) return s;
    if (fp8rl_status s = check_attn_rows(a.v, a.ld_v, kc)) return s;
    if (fp8rl_status s = check_attn_rows(a.dk, a.ld_dk, kc)) return s;
    if (fp8rl_status s = check_attn_rows(a.dv, a.ld_dv, kc)) return s;
  }
  if (!aligned(a.q_offsets, 4) || !aligned(a.k_offsets, 4)) return FP8RL_ERR_ALIGN;
  const size_t need =
      fp8rl::attn_bwd_workspace(a.Tq, a.Tk, a.docs, a.q_heads, a.kv_heads, a.head_dim);
  if (need > 0) {
    if (!workspace || workspace_bytes < need) return FP8RL_ERR_WORKSPACE;
    if (!aligned(workspace, 16)) return FP8RL_ERR_ALIGN;
  }
  return hip_status(fp8rl::launch_attn_bwd(a, (float*)workspace, as_stream(stream)));
}

}  // extern "C"
