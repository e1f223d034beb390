// Host-side launchers and shared device helpers of attention (arguments are validated in
// attn_abi.hip before these are called).
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "block_ops.hpp"
#include "fp8rl_attn.h"

namespace fp8rl {

// ---- attn_decode.hip
size_t attn_decode_workspace(int64_t B, int q_heads, int kv_heads, int head_dim, int64_t max_keys,
                             int window);
hipError_t launch_attn_decode(const fp8rl_attn_decode_args& a, void* workspace, hipStream_t stream);

// ---- attn_fwd.hip
hipError_t launch_attn_fwd(const fp8rl_attn_args& a, hipStream_t stream);

// ---- attn_bwd.hip
size_t attn_bwd_workspace(int64_t Tq, int64_t Tk, int64_t docs, int q_heads, int kv_heads,
                          int head_dim);
hipError_t launch_attn_bwd(const fp8rl_attn_args& a, float* workspace, hipStream_t stream);

// ---- kv_read.hip
hipError_t launch_kv_read(const fp8rl_kv_read_args& a, hipStream_t stream);

// ---------------------------------------------------------------------------------------------
// Device helpers
// ---------------------------------------------------------------------------------------------

constexpr float kLog2e = 1.4426950408889634f;

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }

// tanh of N values x = s * scale, in the places of s. Scores are small beside a cap as a rule: up
// to 1/2 an odd polynomial, fitted to tanh at Chebyshev nodes, is off by 2 units in the last place
// and takes no longer than 1 - 2 / (exp(2x) + 1), which is off by a few 2^-24 of 1, and so of the
// cap, however small x is. The latter, exact at both ends, takes over beyond; which it is is
// decided for the wave.
template <int N, typename V>
__device__ __forceinline__ void tanh_places(V& s, float scale) {
  float top = 0.f;
#pragma unroll
  for (int e = 0; e < N; ++e) {
    s[e] *= scale;
    top = fmaxf(top, fabsf(s[e]));
  }
  auto small = [](float x) {
    const float u = x * x;
    float f = __builtin_fmaf(u, 0.0179992182f, -0.0533910541f);
    f = __builtin_fmaf(u, f, 0.133305137f);
    f = __builtin_fmaf(u, f, -0.333333116f);
    return __builtin_fmaf(x * u, f, x);
  };
  if (!__any(top > 0.5f)) {  // (a NaN stays one on either way)
#pragma unroll
    for (int e = 0; e < N; ++e) s[e] = small(s[e]);
  } else {
#pragma unroll
    for (int e = 0; e < N; ++e) {
      const float x = s[e];
      const float far = __builtin_fmaf(
          2.f, __builtin_amdgcn_rcpf(-1.f - exp2_fast(2.f * kLog2e * x)), 1.f);
      s[e] = fabsf(x) <= 0.5f ? small(x) : far;
    }
  }
}

// Sums over the lanes up to each.
__device__ __forceinline__ int sum_upto(int v) {
  v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xF, 0xF, false);  // row_shr:1, 2, 4, 8
  v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xF, 0xF, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xF, 0xF, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xF, 0xF, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xA, 0xF, false);  // row_bcast:15 into rows 1 and 3
  v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xC, 0xF, false);  // row_bcast:31 into rows 2 and 3
  return v;
}

// Max (sum) over the lanes that differ in bit 4 or 5 of their number, in each of them.
__device__ __forceinline__ float max_rows(float v) {
  auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  v = fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1]));
  auto b = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return fmaxf(__uint_as_float(b[0]), __uint_as_float(b[1]));
}
__device__ __forceinline__ float sum_rows(float v) {
  auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  v = __uint_as_float(a[0]) + __uint_as_float(a[1]);
  auto b = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float(b[0]) + __uint_as_float(b[1]);
}

// Four E4M3 codes as two words of bf16 pairs (exact).
__device__ __forceinline__ u32x2 codes_bf16(uint32_t w) {
  return u32x2{__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.f, false)),
               __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.f, true))};
}

// The page that holds a key: key / page_size by a product with ceil(2^62 / page_size), exact for
// keys and page sizes below 2^31 (the product's error, key * (page_size - 1) at most, is below
// 2^62).
struct PageOf {
  uint64_t reciprocal;
  int page_size;
  __host__ explicit PageOf(int size)
      : reciprocal(((uint64_t{1} << 62) + (uint64_t)size - 1) / (uint64_t)size), page_size(size) {}
  PageOf() = default;
  __device__ __forceinline__ int operator()(int key) const {
    return (int)__umul64hi((uint64_t)(uint32_t)key << 2, reciprocal);
  }
};

// The largest i <= n with at(i) <= x, at not decreasing (0 if there is none); x the same in all
// lanes. 64 samples a step.
template <typename F>
__device__ __forceinline__ int last_not_past(int n, int x, int lane, F at) {
  int lo = 0, hi = n;
  while (hi > lo) {
    const int step = (hi - lo + 63) >> 6;
    const int i = lo + (lane + 1) * step;
    lo += __popcll(__ballot(i <= hi && at(i) <= x)) * step;
    hi = min(hi, lo + step - 1);
  }
  return __builtin_amdgcn_readfirstlane(lo);
}

}  // namespace fp8rl
