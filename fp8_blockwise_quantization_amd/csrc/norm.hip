// The residual stream's root-mean-square norm with an E4M3 output, and its backward pass.
//
//   h = bf16(x + residual),  y = h w r,  r = 1 / sqrt(mean h^2 + eps),
//   group of 128:  S = fp32(max|y| / 448),  code = E4M3(y / S).
//
// p = h w is exact in float32 (8 + 8 significant bits) and the row's r cancels out of y / S:
//   y / S = 448 p / max|p|,   S = r max|p| / 448,
// so the codes wait for no reduction over the row and are those of the exact quotient: with A =
// max|p| the float64 product p * RN64(448 / A) is within 2^-52 of it, a nonzero distance of the
// quotient from an E4M3 midpoint m = M 2^c (M < 2^5) is at least 1 / (M A) > 2^-21 of it (448 p and
// M A are integers in a common unit), and an exact tie comes back from the rounding to float32 as
// the tie that it is. With power-of-two scales S needs r first and the codes are those of
// p * (r / S).
#include "block_ops.hpp"

namespace fp8rl {

namespace {

// fp32(a / 448) for float32 a: 448 m has more significant bits than a for any rounding midpoint m
// of float32, so the float64 product lies on the right side of every midpoint.
__device__ __forceinline__ float div448(double a) { return (float)(a * (1.0 / 448.0)); }

// The least power of two S with 448 S >= a, at least 2^-127 (448 = 0.875 * 2^9: a > 0.875 * 2^E
// takes 2^(E-8), any other a in [2^(E-1), 2^E) takes 2^(E-9)); NaN for an infinite or NaN a.
__device__ __forceinline__ float pow2_scale(float a) {
  const uint32_t u = __float_as_uint(a);
  const int ef = (int)(u >> 23);
  if (ef == 255) return __builtin_nanf("");
  int e = ef - 135 + ((u & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  if (ef == 0 || e < -127) e = -127;
  return e >= -126 ? __uint_as_float((uint32_t)(e + 127) << 23) : __uint_as_float(0x00400000u);
}

// 1 / sqrt(mean + eps) from a row's sum of squares; NaN when that sum is not finite.
__device__ __forceinline__ float row_rstd(float ss, float inv_k, float eps) {
  const float r = rsqrtf(ss * inv_k + eps);
  return __builtin_isfinite(ss) ? r : __builtin_nanf("");
}

// Bits of max |f| over 8 values, over the 16 lanes that share a group (NaN above everything).
__device__ __forceinline__ uint32_t amax8_bits(const float (&f)[8]) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t u = __float_as_uint(f[i]) & 0x7FFFFFFFu;
    m = m > u ? m : u;
  }
  return m;
}

// Sum of a row's partial sums over the W waves that share it.
template <int W>
__device__ __forceinline__ float row_sum(float v, float* red) {
  v = wave_sum(v);
  if (W == 1) return v;
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
  __syncthreads();
  v = red[0];
#pragma unroll
  for (int k = 1; k < W; ++k) v += red[k];
  return v;
}

}  // namespace

// W waves share a row (W == 1: a workgroup of 4 waves takes 4 rows), each lane holding CH chunks of
// 8 values in registers: one read of x, residual and w, no second pass over memory. Lane l of the
// row's 64 W takes chunks l, l + 64 W, ...: a group of 128 values is 16 neighbouring lanes.
template <int W, int CH>
__global__ __launch_bounds__(W == 1 ? 256 : 64 * W) void add_rmsnorm_quant_kernel(NormArgs a) {
  __shared__ float red[W];
  const int lane = W == 1 ? (int)(threadIdx.x & 63) : (int)threadIdx.x;
  const int64_t row = W == 1 ? (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6) : (int64_t)blockIdx.x;
  if (W == 1 && row >= a.M) return;  // whole waves; W == 1 has no barrier
  const u32x4* x = reinterpret_cast<const u32x4*>(a.x + row * a.ld_x);
  const u32x4* __restrict__ wt = reinterpret_cast<const u32x4*>(a.weight);

  u32x4 hv[CH];
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    const int c = lane + 64 * W * i;
    hv[i] = u32x4{0u, 0u, 0u, 0u};
    if (c < a.nc) hv[i] = __builtin_nontemporal_load(x + c);
  }
  if (a.res) {
    const u32x4* res = reinterpret_cast<const u32x4*>(a.res + row * a.ld_res);
    u32x4 rv[CH];
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int c = lane + 64 * W * i;
      rv[i] = u32x4{0u, 0u, 0u, 0u};
      if (c < a.nc) rv[i] = __builtin_nontemporal_load(res + c);
    }
    u32x4* h = reinterpret_cast<u32x4*>(a.h + row * a.ld_h);
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int c = lane + 64 * W * i;
      float f[8], g[8];
      widen8(hv[i], f);
      widen8(rv[i], g);
#pragma unroll
      for (int k = 0; k < 8; ++k) f[k] += g[k];
      hv[i] = round8(f);
      if (a.h && c < a.nc) h[c] = hv[i];
    }
  }

  float ss = 0.f;
  float amax[CH];
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    const int c = lane + 64 * W * i;
    float f[8], g[8];
    widen8(hv[i], f);
#pragma unroll
    for (int k = 0; k < 8; ++k) ss = __builtin_fmaf(f[k], f[k], ss);
    if (a.xq) {
      const u32x4 wv = c < a.nc ? wt[c] : u32x4{0u, 0u, 0u, 0u};
      widen8(wv, g);
#pragma unroll
      for (int k = 0; k < 8; ++k) f[k] *= g[k];
      amax[i] = __uint_as_float(row16_max_u32(amax8_bits(f)));
      if (!a.pow2 && c < a.nc) {
        const double r = amax[i] == 0.f ? 1.0 : 448.0 / (double)amax[i];
        u32x2* q = reinterpret_cast<u32x2*>(a.xq + row * a.ld_xq);
        __builtin_nontemporal_store(codes8(f, r), q + c);
      }
    }
  }
  const float r = row_rstd(row_sum<W>(ss, red), 0.125f / (float)a.nc, a.eps);

  if (a.xq) {
    float* sa = a.sa + row * (a.nc >> 4);
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int c = lane + 64 * W * i;
      if (c >= a.nc) continue;
      float S = amax[i] == 0.f ? (r == r ? 1.f : r) : div448((double)amax[i] * (double)r);
      if (a.pow2) {
        if (amax[i] != 0.f) S = pow2_scale(amax[i] * r);
        float f[8], g[8];
        widen8(hv[i], f);
        widen8(wt[c], g);
#pragma unroll
        for (int k = 0; k < 8; ++k) f[k] *= g[k];
        u32x2* q = reinterpret_cast<u32x2*>(a.xq + row * a.ld_xq);
        __builtin_nontemporal_store(codes8(f, (double)r / (double)S), q + c);
      }
      if ((c & 15) == 0) sa[c >> 4] = S;
    }
  }
  if (a.y) {
    u32x4* y = reinterpret_cast<u32x4*>(a.y + row * a.ld_y);
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int c = lane + 64 * W * i;
      if (c >= a.nc) continue;
      float f[8], g[8];
      widen8(hv[i], f);
      widen8(wt[c], g);
#pragma unroll
      for (int k = 0; k < 8; ++k) f[k] = f[k] * g[k] * r;
      y[c] = round8(f);
    }
  }
}

// ---------------------------------------------------------------------------------------------
// Backward. Both sums of a row (h^2 and dy w h) are reduced together, and every thread keeps its
// columns over all the rows it takes, so that its share of dw stays in registers.
// ---------------------------------------------------------------------------------------------
namespace {

// The chunks of one row that a thread holds: dy, h and, where there is one, dh.
template <int CH, int STEP>
struct BwdRow {
  u32x4 g[CH], h[CH], s[CH];
  __device__ __forceinline__ void load(const NormBwdArgs& a, int64_t row, int c0) {
    const u32x4* dy = reinterpret_cast<const u32x4*>(a.dy + row * a.ld_dy);
    const u32x4* hp = reinterpret_cast<const u32x4*>(a.h + row * a.ld_h);
    const u32x4* dh = reinterpret_cast<const u32x4*>(a.dh + row * a.ld_dh);
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int c = c0 + STEP * i;
      g[i] = h[i] = s[i] = u32x4{0u, 0u, 0u, 0u};
      if (c < a.nc) {
        g[i] = __builtin_nontemporal_load(dy + c);
        h[i] = __builtin_nontemporal_load(hp + c);
      }
    }
    if (a.dh) {
#pragma unroll
      for (int i = 0; i < CH; ++i) {
        const int c = c0 + STEP * i;
        if (c < a.nc) s[i] = __builtin_nontemporal_load(dh + c);
      }
    }
  }
  __device__ __forceinline__ void sums(const u32x4 (&wt)[CH], float& ss, float& sd) const {
    ss = sd = 0.f;
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      float f[8], d[8], w[8];
      widen8(h[i], f);
      widen8(g[i], d);
      widen8(wt[i], w);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        ss = __builtin_fmaf(f[k], f[k], ss);
        sd = __builtin_fmaf(d[k] * w[k], f[k], sd);
      }
    }
  }
  __device__ __forceinline__ void finish(const NormBwdArgs& a, int64_t row, int c0,
                                         u32x4 (&wt)[CH], float r, float lean,
                                         float (&acc)[CH][8]) {
    u32x4* dx = reinterpret_cast<u32x4*>(a.dx + row * a.ld_dx);
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      // widened again from the 16-byte chunks: kept from sums(), the float32 values would take
      // twice the registers of what was loaded all through the reduction
      asm volatile("" : "+v"(h[i]), "+v"(g[i]), "+v"(wt[i]));
      const int c = c0 + STEP * i;
      float f[8], d[8], w[8], o[8];
      widen8(h[i], f);
      widen8(g[i], d);
      widen8(wt[i], w);
      widen8(s[i], o);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        acc[i][k] = __builtin_fmaf(d[k], f[k] * r, acc[i][k]);
        o[k] = __builtin_fmaf(r, __builtin_fmaf(-f[k], lean, d[k] * w[k]), o[k]);
      }
      if (c < a.nc) __builtin_nontemporal_store(round8(o), dx + c);
    }
  }
};

template <int CH, int STEP>
__device__ __forceinline__ void load_weights(const NormBwdArgs& a, int c0, u32x4 (&wt)[CH]) {
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    const int c = c0 + STEP * i;
    wt[i] = c < a.nc ? reinterpret_cast<const u32x4*>(a.weight)[c] : u32x4{0u, 0u, 0u, 0u};
  }
}

template <int CH, int STEP>
__device__ __forceinline__ void store_part(const NormBwdArgs& a, int c0, const float (&acc)[CH][8]) {
  float4* part = reinterpret_cast<float4*>(a.part) + (int64_t)blockIdx.x * (2 * a.nc);
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    const int c = c0 + STEP * i;
    if (c >= a.nc) continue;
    part[2 * c] = make_float4(acc[i][0], acc[i][1], acc[i][2], acc[i][3]);
    part[2 * c + 1] = make_float4(acc[i][4], acc[i][5], acc[i][6], acc[i][7]);
  }
}

}  // namespace

// Rows of up to 64 CH chunks: each of a workgroup's RW waves takes whole rows, with no barrier
// between them; the waves' shares of dw are added through LDS at the end, in a fixed order.
template <int RW, int CH>
__global__ __launch_bounds__(64 * RW, 2) void add_rmsnorm_bwd_wave_kernel(NormBwdArgs a) {
  __shared__ float red[RW / 2][CH * 8][64];
  const int lane = (int)(threadIdx.x & 63), wave = (int)(threadIdx.x >> 6);
  const float inv_k = 0.125f / (float)a.nc;
  u32x4 wt[CH];
  load_weights<CH, 64>(a, lane, wt);
  float acc[CH][8];
#pragma unroll
  for (int i = 0; i < CH; ++i)
#pragma unroll
    for (int k = 0; k < 8; ++k) acc[i][k] = 0.f;

  for (int64_t row = (int64_t)blockIdx.x * RW + wave; row < a.M; row += (int64_t)gridDim.x * RW) {
    BwdRow<CH, 64> v;
    v.load(a, row, lane);
    float ss, sd;
    v.sums(wt, ss, sd);
    ss = wave_sum(ss);
    sd = wave_sum(sd);
    const float r = row_rstd(ss, inv_k, a.eps);
    v.finish(a, row, lane, wt, r, r * r * (sd * inv_k), acc);
  }
  if (!a.part) return;
#pragma unroll
  for (int n = RW / 2; n > 0; n >>= 1) {
    if (wave >= n && wave < 2 * n)
#pragma unroll
      for (int i = 0; i < CH; ++i)
#pragma unroll
        for (int k = 0; k < 8; ++k) red[wave - n][8 * i + k][lane] = acc[i][k];
    __syncthreads();
    if (wave < n)
#pragma unroll
      for (int i = 0; i < CH; ++i)
#pragma unroll
        for (int k = 0; k < 8; ++k) acc[i][k] += red[wave][8 * i + k][lane];
    __syncthreads();
  }
  if (wave == 0) store_part<CH, 64>(a, lane, acc);
}

// Wider rows: a workgroup of W waves takes a row, the next row's loads in flight while it reduces.
template <int W, int CH, bool AHEAD>
__global__ __launch_bounds__(64 * W) void add_rmsnorm_bwd_kernel(NormBwdArgs a) {
  __shared__ float red[2][2][W];
  const int t = (int)threadIdx.x;
  const float inv_k = 0.125f / (float)a.nc;
  u32x4 wt[CH];
  load_weights<CH, 64 * W>(a, t, wt);
  float acc[CH][8];
#pragma unroll
  for (int i = 0; i < CH; ++i)
#pragma unroll
    for (int k = 0; k < 8; ++k) acc[i][k] = 0.f;

  int buf = 0;
  BwdRow<CH, 64 * W> v;
  int64_t row = blockIdx.x;
  if (AHEAD && row < a.M) v.load(a, row, t);
  for (; row < a.M; row += gridDim.x, buf ^= 1) {
    // in place of dy or dh: the next row's values are read before this row's are written, and no
    // other workgroup writes them
    BwdRow<CH, 64 * W> next;
    if (!AHEAD) v.load(a, row, t);
    if (AHEAD && row + gridDim.x < a.M) next.load(a, row + gridDim.x, t);
    float ss, sd;
    v.sums(wt, ss, sd);
    ss = wave_sum(ss);
    sd = wave_sum(sd);
    // two buffers: a wave writes row n + 2's sums only after the barrier of row n + 1, which no
    // wave reaches before it has read row n's
    if ((t & 63) == 0) red[buf][0][t >> 6] = ss, red[buf][1][t >> 6] = sd;
    __syncthreads();
    ss = red[buf][0][0], sd = red[buf][1][0];
#pragma unroll
    for (int k = 1; k < W; ++k) ss += red[buf][0][k], sd += red[buf][1][k];
    const float r = row_rstd(ss, inv_k, a.eps);
    v.finish(a, row, t, wt, r, r * r * (sd * inv_k), acc);
    if (AHEAD) v = next;
  }
  if (a.part) store_part<CH, 64 * W>(a, t, acc);
}

// dw[k] = sum over the groups of their partial sums: 8 columns of 4 values per workgroup, 32
// threads down each column, then their sums in order.
__global__ __launch_bounds__(256) void norm_dw_kernel(const float4* __restrict__ part, int groups,
                                                      int nc4, float* __restrict__ dw) {
  __shared__ float4 red[32][8];
  const int col = threadIdx.x & 7, g0 = threadIdx.x >> 3;
  const int c = blockIdx.x * 8 + col;  // K % 128 == 0: every column exists
  float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
  for (int g = g0; g < groups; g += 32) {
    const float4 v = part[(int64_t)g * nc4 + c];
    s.x += v.x, s.y += v.y, s.z += v.z, s.w += v.w;
  }
  red[g0][col] = s;
  __syncthreads();
  if (threadIdx.x < 32) {
    const float* r = reinterpret_cast<const float*>(red) + threadIdx.x;
    float sum = r[0];
#pragma unroll
    for (int k = 1; k < 32; ++k) sum += r[32 * k];
    dw[blockIdx.x * 32 + threadIdx.x] = sum;
  }
}

namespace {

template <int W, int CH>
hipError_t run_norm(const NormArgs& a, hipStream_t stream) {
  const int64_t wgs = W == 1 ? (a.M + 3) / 4 : a.M;
  hipLaunchKernelGGL((add_rmsnorm_quant_kernel<W, CH>), dim3((unsigned)wgs),
                     dim3(W == 1 ? 256 : 64 * W), 0, stream, a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_add_rmsnorm_quant(const NormArgs& a, hipStream_t stream) {
  const int nc = a.nc;
  if (nc <= 256) return run_norm<4, 1>(a, stream);
  if (nc <= 512) return run_norm<4, 2>(a, stream);
  if (nc <= 1024) return run_norm<4, 4>(a, stream);
  if (nc <= 2048) return run_norm<16, 2>(a, stream);
  return run_norm<16, 4>(a, stream);
}

namespace {

// How the backward pass of M rows of nc chunks is cut up: waves per row-taking unit and groups.
struct BwdShape {
  bool wave_rows;  // a wave per row (rows of up to 512 chunks), else a workgroup
  int rw;          // waves of a workgroup that take rows of their own
  int64_t groups;
};
BwdShape bwd_shape(int64_t M, int64_t nc) {
  if (nc <= 512) {
    const int rw = M >= 8 * 256 ? 8 : 4;
    const int64_t most = 256 * (8 / rw), g = (M + rw - 1) / rw;
    return {true, rw, g < most ? g : most};
  }
  return {false, 1, M < 512 ? M : 512};
}

template <int RW, int CH>
void run_bwd_wave(const NormBwdArgs& a, int64_t groups, hipStream_t stream) {
  hipLaunchKernelGGL((add_rmsnorm_bwd_wave_kernel<RW, CH>), dim3((unsigned)groups), dim3(64 * RW),
                     0, stream, a);
}
template <int RW>
void run_bwd_waves(const NormBwdArgs& a, int64_t groups, hipStream_t stream) {
  if (a.nc <= 64) run_bwd_wave<RW, 1>(a, groups, stream);
  else if (a.nc <= 128) run_bwd_wave<RW, 2>(a, groups, stream);
  else if (a.nc <= 256) run_bwd_wave<RW, 4>(a, groups, stream);
  else run_bwd_wave<RW, 8>(a, groups, stream);
}
template <int W, int CH, bool AHEAD>
void run_bwd(const NormBwdArgs& a, int64_t groups, hipStream_t stream) {
  hipLaunchKernelGGL((add_rmsnorm_bwd_kernel<W, CH, AHEAD>), dim3((unsigned)groups), dim3(64 * W), 0,
                     stream, a);
}

}  // namespace

int64_t norm_bwd_groups(int64_t M, int64_t K) { return bwd_shape(M, K / 8).groups; }

hipError_t launch_add_rmsnorm_bwd(const NormBwdArgs& a, float* dw, hipStream_t stream) {
  const BwdShape s = bwd_shape(a.M, a.nc);
  if (s.groups > 0) {
    if (s.wave_rows && s.rw == 8) run_bwd_waves<8>(a, s.groups, stream);
    else if (s.wave_rows) run_bwd_waves<4>(a, s.groups, stream);
    else if (a.nc <= 1024) run_bwd<8, 2, true>(a, s.groups, stream);
    else if (a.nc <= 2048) run_bwd<16, 2, true>(a, s.groups, stream);
    else run_bwd<16, 4, false>(a, s.groups, stream);
    if (hipError_t e = hipGetLastError(); e != hipSuccess) return e;
  }
  if (!dw) return hipSuccess;
  hipLaunchKernelGGL(norm_dw_kernel, dim3((unsigned)(a.nc / 4)), dim3(256), 0, stream,
                     reinterpret_cast<const float4*>(a.part), (int)s.groups, 2 * a.nc, dw);
  return hipGetLastError();
}

}  // namespace fp8rl
