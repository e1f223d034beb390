// Host-side launchers and shared device helpers of the operators between the linears (arguments
// are validated in block_abi.hip before these are called).
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "device_common.hpp"
#include "fp8rl_block.h"

namespace fp8rl {

// ---- norm.hip
struct NormArgs {
  const uint16_t* x;
  const uint16_t* res;  // or null
  const uint16_t* weight;
  uint16_t* h;   // or null; may be x or res
  uint16_t* y;   // or null
  uint8_t* xq;   // or null, with sa
  float* sa;
  int64_t ld_x, ld_res, ld_h, ld_y, ld_xq;
  int64_t M;
  int nc;  // 16-byte chunks of a row: K / 8
  float eps;
  int pow2;
};
hipError_t launch_add_rmsnorm_quant(const NormArgs& a, hipStream_t stream);

struct NormBwdArgs {
  const uint16_t* dy;
  const uint16_t* h;
  const uint16_t* weight;
  const uint16_t* dh;  // or null
  uint16_t* dx;        // may be dy or dh
  float* part;         // [groups][K] partial sums of dw, or null
  int64_t ld_dy, ld_h, ld_dh, ld_dx;
  int64_t M;
  int nc;
  float eps;
};
// Workgroups (= rows of partial sums of dw) that the backward pass of M rows of K runs with.
int64_t norm_bwd_groups(int64_t M, int64_t K);
hipError_t launch_add_rmsnorm_bwd(const NormBwdArgs& a, float* dw, hipStream_t stream);

// ---- moe.hip
// Workgroups of the counting sort of n choices (1: one kernel, no workspace).
int64_t sort_blocks(int64_t n);
hipError_t launch_moe_sort(const void* ids, bool wide, int64_t n, int top_k, int E,
                           int32_t* offsets, int32_t* row_ids, int32_t* pos, int32_t* counts,
                           hipStream_t stream);
struct MoeArgs {
  const void* x;  // dispatch: token rows; combine: grouped rows; combine_bwd: dout
  const void* y;  // combine_bwd: grouped rows, or null
  void* out;      // dispatch, combine_bwd: grouped rows; combine: token rows
  const int32_t* pos;
  const float* weights;  // or null
  float* dweights;       // combine_bwd, or null
  int64_t ld_x, ld_y, ld_out;
  int64_t T, R;
  int top_k;
  int nc;  // chunks of 8 values in a row: N / 8
};
hipError_t launch_moe_dispatch(const MoeArgs& a, hipStream_t stream);
hipError_t launch_moe_combine(const MoeArgs& a, bool y_f32, bool out_f32, hipStream_t stream);
hipError_t launch_moe_combine_bwd(const MoeArgs& a, bool y_f32, hipStream_t stream);

// ---- rope_append.hip
hipError_t launch_rope_kv_append(const fp8rl_rope_kv_args& a, hipStream_t stream);

// ---------------------------------------------------------------------------------------------
// Device helpers
// ---------------------------------------------------------------------------------------------

typedef float f32x4 __attribute__((ext_vector_type(4)));

// The 8 bf16 values of a 16-byte chunk as float32 (exact).
__device__ __forceinline__ void widen8(u32x4 w, float (&f)[8]) {
  f[0] = bf16_lo(w.x), f[1] = bf16_hi(w.x), f[2] = bf16_lo(w.y), f[3] = bf16_hi(w.y);
  f[4] = bf16_lo(w.z), f[5] = bf16_hi(w.z), f[6] = bf16_lo(w.w), f[7] = bf16_hi(w.w);
}

// Two float32 rounded to bf16 (nearest, ties to even; NaN stays NaN), the first in the low half.
__device__ __forceinline__ uint32_t pack2_bf16(float lo, float hi) {
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
  typedef float f32x2 __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2{lo, hi}), bf16x2));
}

__device__ __forceinline__ u32x4 round8(const float (&f)[8]) {
  return u32x4{pack2_bf16(f[0], f[1]), pack2_bf16(f[2], f[3]), pack2_bf16(f[4], f[5]),
               pack2_bf16(f[6], f[7])};
}

// E4M3 codes of 8 float32 values, saturating; a NaN gives a NaN code. The clamp is one median of
// three; it loses a NaN, so values among which there is one (four unordered comparisons tell) go
// through a select instead.
__device__ __forceinline__ u32x2 encode8(float (&t)[8]) {
  const bool nan = __builtin_isunordered(t[0], t[1]) | __builtin_isunordered(t[2], t[3]) |
                   __builtin_isunordered(t[4], t[5]) | __builtin_isunordered(t[6], t[7]);
  if (nan) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      t[i] = __builtin_fabsf(t[i]) > kE4M3Max ? __builtin_copysignf(kE4M3Max, t[i]) : t[i];
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) t[i] = clamp_e4m3(t[i]);
  }
  return u32x2{pack4_e4m3(t[0], t[1], t[2], t[3]), pack4_e4m3(t[4], t[5], t[6], t[7])};
}

// The E4M3 codes of f * r, the product formed in float64 and rounded through float32.
__device__ __forceinline__ u32x2 codes8(const float (&f)[8], double r) {
  float t[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) t[i] = (float)((double)f[i] * r);
  return encode8(t);
}

// Sum over the 64 lanes of a wave, the same bits in every lane.
__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o, 64);
  return v;
}

}  // namespace fp8rl
