// C ABI entry points of the operators between the linears: argument validation (host only, before
// any HIP call) and dispatch.
#include <float.h>
#include <math.h>
#include <stdint.h>

#include "block_ops.hpp"
#include "fp8rl_block.h"

namespace {

constexpr int64_t kMaxDim = (int64_t{1} << 31) - 1;
constexpr int64_t kMaxGrid = int64_t{1} << 22;  // workgroups: up to 1024 threads each, below 2^32

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
bool in_range(int64_t v) { return v >= 0 && v <= kMaxDim; }
fp8rl_status hip_status(hipError_t e) { return e == hipSuccess ? FP8RL_OK : FP8RL_ERR_HIP; }
hipStream_t as_stream(void* s) { return reinterpret_cast<hipStream_t>(s); }

// A matrix of rows of n values, `bytes` each: FP8RL_OK when absent (null) or laid out as required.
fp8rl_status check_rows(const void* p, int64_t ld, int64_t n, int64_t align = 16,
                        int64_t pitch = 8) {
  if (!p) return FP8RL_OK;
  if (ld < n || ld > kMaxDim) return FP8RL_ERR_SHAPE;
  if (!aligned(p, (uintptr_t)align) || ld % pitch) return FP8RL_ERR_ALIGN;
  return FP8RL_OK;
}

fp8rl_status check_norm_shape(int64_t M, int64_t K) {
  if (!in_range(M) || !in_range(K)) return FP8RL_ERR_SHAPE;
  if (K % 128 || K > 32768 || M >= kMaxGrid) return FP8RL_ERR_SHAPE;
  return FP8RL_OK;
}

// (a smaller eps beside a row of zeros has no finite reciprocal root in float32)
bool bad_eps(float eps) { return !(eps >= FLT_MIN) || isinf(eps); }

}  // namespace

extern "C" {

fp8rl_status fp8rl_add_rmsnorm_quant(const uint16_t* x, int64_t ld_x, const uint16_t* residual,
                                     int64_t ld_res, const uint16_t* weight, float eps, int64_t M,
                                     int64_t K, uint16_t* h, int64_t ld_h, uint16_t* y,
                                     int64_t ld_y, uint8_t* xq, int64_t ld_xq, float* sa,
                                     int scale_fmt, void* stream) {
  if (scale_fmt != FP8RL_SCALE_FP32 && scale_fmt != FP8RL_SCALE_POW2) return FP8RL_ERR_ARG;
  if (bad_eps(eps)) return FP8RL_ERR_ARG;
  if (fp8rl_status s = check_norm_shape(M, K)) return s;
  if (M == 0 || K == 0) return FP8RL_OK;
  if (!x || !weight || (!xq) != (!sa) || (!xq && !y)) return FP8RL_ERR_NULL;
  if (h && !residual) return FP8RL_ERR_ARG;
  if (fp8rl_status s = check_rows(x, ld_x, K)) return s;
  if (fp8rl_status s = check_rows(residual, ld_res, K)) return s;
  if (fp8rl_status s = check_rows(h, ld_h, K)) return s;
  if (fp8rl_status s = check_rows(y, ld_y, K)) return s;
  if (fp8rl_status s = check_rows(xq, ld_xq, K, 16, 16)) return s;
  if (!aligned(weight, 16) || !aligned(sa, 4)) return FP8RL_ERR_ALIGN;
  const fp8rl::NormArgs a{x,    residual, weight, h,     y, xq,           sa,  ld_x,
                          ld_res, ld_h,   ld_y,   ld_xq, M, (int)(K / 8), eps,
                          scale_fmt == FP8RL_SCALE_POW2};
  return hip_status(fp8rl::launch_add_rmsnorm_quant(a, as_stream(stream)));
}

size_t fp8rl_add_rmsnorm_bwd_workspace_bytes(int64_t M, int64_t K) {
  if (check_norm_shape(M, K) != FP8RL_OK) return 0;
  return (size_t)fp8rl::norm_bwd_groups(M, K) * (size_t)K * sizeof(float);
}

fp8rl_status fp8rl_add_rmsnorm_bwd(const uint16_t* dy, int64_t ld_dy, const uint16_t* h,
                                   int64_t ld_h, const uint16_t* weight, const uint16_t* dh,
                                   int64_t ld_dh, float eps, int64_t M, int64_t K, uint16_t* dx,
                                   int64_t ld_dx, float* dw, void* workspace,
                                   size_t workspace_bytes, void* stream) {
  if (bad_eps(eps)) return FP8RL_ERR_ARG;
  if (fp8rl_status s = check_norm_shape(M, K)) return s;
  if (K == 0 || (M == 0 && !dw)) return FP8RL_OK;
  if (M > 0) {
    if (!dy || !h || !weight || !dx) return FP8RL_ERR_NULL;
    if (fp8rl_status s = check_rows(dy, ld_dy, K)) return s;
    if (fp8rl_status s = check_rows(h, ld_h, K)) return s;
    if (fp8rl_status s = check_rows(dh, ld_dh, K)) return s;
    if (fp8rl_status s = check_rows(dx, ld_dx, K)) return s;
    if (!aligned(weight, 16)) return FP8RL_ERR_ALIGN;
  }
  if (!aligned(dw, 4)) return FP8RL_ERR_ALIGN;
  const size_t need = dw ? fp8rl_add_rmsnorm_bwd_workspace_bytes(M, K) : 0;
  if (need > 0) {
    if (!workspace || workspace_bytes < need) return FP8RL_ERR_WORKSPACE;
    if (!aligned(workspace, 16)) return FP8RL_ERR_ALIGN;
  }
  const fp8rl::NormBwdArgs a{dy,   h,     weight, dh,    dx, need ? (float*)workspace : nullptr,
                             ld_dy, ld_h, ld_dh,  ld_dx, M,  (int)(K / 8), eps};
  return hip_status(fp8rl::launch_add_rmsnorm_bwd(a, dw, as_stream(stream)));
}

namespace {

fp8rl_status check_choices(int64_t T, int32_t top_k) {
  if (!in_range(T) || T >= (int64_t{1} << 24)) return FP8RL_ERR_SHAPE;  // T * top_k < 2^30
  if (top_k < 1 || top_k > 64) return FP8RL_ERR_ARG;
  return FP8RL_OK;
}

fp8rl_status check_moe_rows(int64_t T, int32_t top_k, int64_t N, int64_t R) {
  if (fp8rl_status s = check_choices(T, top_k)) return s;
  if (!in_range(N) || !in_range(R) || N % 8) return FP8RL_ERR_SHAPE;
  return FP8RL_OK;
}

bool bad_dtype(int d) { return d != FP8RL_OUT_BF16 && d != FP8RL_OUT_F32; }

}  // namespace

size_t fp8rl_moe_sort_workspace_bytes(int64_t T, int32_t top_k, int32_t E) {
  if (check_choices(T, top_k) != FP8RL_OK || E < 1 || E > 1024) return 0;
  const int64_t blocks = fp8rl::sort_blocks(T * top_k);
  return blocks > 1 ? (size_t)blocks * E * sizeof(int32_t) : 0;
}

fp8rl_status fp8rl_moe_sort(const void* topk_ids, int ids_dtype, int64_t T, int32_t top_k,
                            int32_t E, int32_t* expert_offsets, int32_t* row_ids, int32_t* pos,
                            void* workspace, size_t workspace_bytes, void* stream) {
  if (ids_dtype != FP8RL_IDS_I32 && ids_dtype != FP8RL_IDS_I64) return FP8RL_ERR_DTYPE;
  if (E < 1 || E > 1024) return FP8RL_ERR_ARG;
  if (fp8rl_status s = check_choices(T, top_k)) return s;
  if (!expert_offsets || (T > 0 && (!topk_ids || !row_ids || !pos))) return FP8RL_ERR_NULL;
  if (!aligned(expert_offsets, 4) || !aligned(row_ids, 4) || !aligned(pos, 4) ||
      !aligned(topk_ids, ids_dtype == FP8RL_IDS_I64 ? 8 : 4))
    return FP8RL_ERR_ALIGN;
  const size_t need = fp8rl_moe_sort_workspace_bytes(T, top_k, E);
  if (need > 0) {
    if (!workspace || workspace_bytes < need) return FP8RL_ERR_WORKSPACE;
    if (!aligned(workspace, 16)) return FP8RL_ERR_ALIGN;
  }
  return hip_status(fp8rl::launch_moe_sort(topk_ids, ids_dtype == FP8RL_IDS_I64, T * top_k, top_k,
                                           E, expert_offsets, row_ids, pos, (int32_t*)workspace,
                                           as_stream(stream)));
}

fp8rl_status fp8rl_moe_dispatch(const uint16_t* x, int64_t ld_x, const int32_t* pos, int64_t T,
                                int32_t top_k, int64_t N, uint16_t* out, int64_t R, int64_t ld_out,
                                void* stream) {
  if (fp8rl_status s = check_moe_rows(T, top_k, N, R)) return s;
  if (T == 0 || N == 0 || R == 0) return FP8RL_OK;
  if (!x || !pos || !out) return FP8RL_ERR_NULL;
  if (fp8rl_status s = check_rows(x, ld_x, N)) return s;
  if (fp8rl_status s = check_rows(out, ld_out, N)) return s;
  if (!aligned(pos, 4)) return FP8RL_ERR_ALIGN;
  // a wave per 2048 values of a row, four to a workgroup: below 2^32 threads in a grid
  if (T * ((N + 2047) / 2048) > (int64_t{1} << 26) - 4) return FP8RL_ERR_SHAPE;
  fp8rl::MoeArgs a{};
  a.x = x, a.out = out, a.pos = pos;
  a.ld_x = ld_x, a.ld_out = ld_out;
  a.T = T, a.R = R, a.top_k = top_k, a.nc = (int)(N / 8);
  return hip_status(fp8rl::launch_moe_dispatch(a, as_stream(stream)));
}

fp8rl_status fp8rl_moe_combine(const void* y, int y_dtype, int64_t R, int64_t ld_y,
                               const int32_t* pos, const float* weights, int64_t T, int32_t top_k,
                               int64_t N, void* out, int out_dtype, int64_t ld_out, void* stream) {
  if (bad_dtype(y_dtype) || bad_dtype(out_dtype)) return FP8RL_ERR_DTYPE;
  if (fp8rl_status s = check_moe_rows(T, top_k, N, R)) return s;
  if (T == 0 || N == 0) return FP8RL_OK;
  if ((!y && R > 0) || !pos || !out) return FP8RL_ERR_NULL;
  if (fp8rl_status s = check_rows(R > 0 ? y : nullptr, ld_y, N)) return s;
  if (fp8rl_status s = check_rows(out, ld_out, N)) return s;
  if (!aligned(pos, 4) || !aligned(weights, 4)) return FP8RL_ERR_ALIGN;
  fp8rl::MoeArgs a{};
  a.x = y, a.out = out, a.pos = pos, a.weights = weights;
  a.ld_x = ld_y, a.ld_out = ld_out;
  a.T = T, a.R = R, a.top_k = top_k, a.nc = (int)(N / 8);
  return hip_status(fp8rl::launch_moe_combine(a, y_dtype == FP8RL_OUT_F32,
                                              out_dtype == FP8RL_OUT_F32, as_stream(stream)));
}

fp8rl_status fp8rl_moe_combine_bwd(const uint16_t* dout, int64_t ld_dout, const void* y,
                                   int64_t ld_y, int y_dtype, int64_t R, const int32_t* pos,
                                   const float* weights, int64_t T, int32_t top_k, int64_t N,
                                   void* dy, int64_t ld_dy, float* dweights, void* stream) {
  if (bad_dtype(y_dtype)) return FP8RL_ERR_DTYPE;
  if (fp8rl_status s = check_moe_rows(T, top_k, N, R)) return s;
  if (T == 0) return FP8RL_OK;
  if (N > 0 && (!dout || (R > 0 && (!dy || (!y) != (!dweights))))) return FP8RL_ERR_NULL;
  if (!pos) return FP8RL_ERR_NULL;
  if (N > 0) {
    if (fp8rl_status s = check_rows(dout, ld_dout, N)) return s;
    if (R > 0) {
      if (fp8rl_status s = check_rows(y, ld_y, N)) return s;
      if (fp8rl_status s = check_rows(dy, ld_dy, N)) return s;
    }
  }
  if (!aligned(pos, 4) || !aligned(weights, 4) || !aligned(dweights, 4)) return FP8RL_ERR_ALIGN;
  fp8rl::MoeArgs a{};
  a.x = dout, a.y = y, a.out = dy, a.pos = pos, a.weights = weights, a.dweights = dweights;
  a.ld_x = ld_dout, a.ld_y = ld_y, a.ld_out = ld_dy;
  a.T = T, a.R = R, a.top_k = top_k, a.nc = (int)(N / 8);
  return hip_status(fp8rl::launch_moe_combine_bwd(a, y_dtype == FP8RL_OUT_F32, as_stream(stream)));
}

fp8rl_status fp8rl_rope_kv_append(const fp8rl_rope_kv_args* args, void* stream) {
  if (!args) return FP8RL_ERR_NULL;
  const fp8rl_rope_kv_args& a = *args;
  if (!in_range(a.T) || a.num_pages < 0) return FP8RL_ERR_SHAPE;
  if (a.q_heads < 0 || a.kv_heads < 1 || a.q_heads > 65536 || a.kv_heads > 65536)
    return FP8RL_ERR_SHAPE;
  if (a.head_dim < 8 || a.head_dim > 512 || a.head_dim % 8) return FP8RL_ERR_SHAPE;
  if (a.rot_dim < 0 || a.rot_dim > a.head_dim || a.rot_dim % 16) return FP8RL_ERR_SHAPE;
  // up to 32 threads per head of a token in whole waves, below 2^32 in a grid
  if (a.T * (a.q_heads + 2 * (int64_t)a.kv_heads) >= (int64_t{1} << 25)) return FP8RL_ERR_SHAPE;
  if (a.interleaved != 0 && a.interleaved != 1) return FP8RL_ERR_ARG;
  if (a.page_size < 1 || a.num_pages >= (int64_t{1} << 62) / a.page_size) return FP8RL_ERR_SHAPE;
  if ((!a.q_weight) != (!a.k_weight) || (!a.k_scale) != (!a.v_scale)) return FP8RL_ERR_NULL;
  if (a.q_weight && bad_eps(a.eps)) return FP8RL_ERR_ARG;
  if (a.T == 0) return FP8RL_OK;
  if (!a.k || !a.v || !a.slot_mapping) return FP8RL_ERR_NULL;
  if (a.num_pages > 0 && (!a.k_cache || !a.v_cache)) return FP8RL_ERR_NULL;
  if (a.q_heads > 0 && (!a.q || !a.q_out)) return FP8RL_ERR_NULL;
  if (a.rot_dim > 0 && (!a.cos_sin || !a.positions)) return FP8RL_ERR_NULL;
  if (a.max_pos < 0 || a.max_pos > kMaxDim) return FP8RL_ERR_SHAPE;
  const int64_t qc = (int64_t)a.q_heads * a.head_dim, kc = (int64_t)a.kv_heads * a.head_dim;
  if (a.q_heads > 0) {
    if (fp8rl_status s = check_rows(a.q, a.ld_q, qc)) return s;
    if (fp8rl_status s = check_rows(a.q_out, a.ld_qo, qc, a.q_scale ? 8 : 16)) return s;
  }
  if (fp8rl_status s = check_rows(a.k, a.ld_k, kc)) return s;
  if (fp8rl_status s = check_rows(a.v, a.ld_v, kc)) return s;
  if (a.num_pages > 0) {
    if (a.slot_stride < a.head_dim || a.head_stride < a.head_dim ||
        a.page_stride < (a.num_pages > 1 ? a.head_dim : 0))
      return FP8RL_ERR_SHAPE;
    // offsets of any row of the cache stay inside 63 bits
    constexpr int64_t kFar = int64_t{1} << 60;
    if (a.slot_stride > kFar / a.page_size || a.page_stride > kFar / a.num_pages ||
        a.head_stride > kFar / a.kv_heads)
      return FP8RL_ERR_SHAPE;
    const uintptr_t cache_align = a.k_scale ? 8 : 16;
    if (!aligned(a.k_cache, cache_align) || !aligned(a.v_cache, cache_align) ||
        a.page_stride % 8 || a.slot_stride % 8 || a.head_stride % 8)
      return FP8RL_ERR_ALIGN;
  }
  if (!aligned(a.cos_sin, 16) || !aligned(a.positions, 8) || !aligned(a.slot_mapping, 8) ||
      !aligned(a.q_weight, 16) || !aligned(a.k_weight, 16) || !aligned(a.q_scale, 4) ||
      !aligned(a.k_scale, 4) || !aligned(a.v_scale, 4))
    return FP8RL_ERR_ALIGN;
  return hip_status(fp8rl::launch_rope_kv_append(a, as_stream(stream)));
}

}  // extern "C"
