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

// Sum over the lanes that share a row: L of them inside a wave, or (L == 0) the whole workgroup.
template <int L, int W>
__device__ __forceinline__ float row_sum(float v, float* red) {
#pragma unroll
  for (int o = L ? L / 2 : 32; o > 0; o >>= 1) v += __shfl_xor(v, o, 64);
  if (L) return v;
  const int waves = W ? W : (int)(blockDim.x >> 6);
  if (waves == 1) return v;
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
  __syncthreads();
  v = red[0];
  for (int k = 1; k < waves; ++k) v += red[k];
  return v;
}

}  // namespace

// A row is held in registers, CH chunks of 8 values per lane: one read of x, residual and w, no
// second pass over memory. It is shared by L lanes of a wave (L < 64: a wave takes 64 / L rows, a
// workgroup of 256 threads 256 / L), or with L == 0 by a whole workgroup of as many waves as it
// needs. Lane l of a row's n lanes takes chunks l, l + n, ...: a group of 128 values is 16
// neighbouring lanes.
template <int CH, int L, int W>
__global__ __launch_bounds__(L ? 256 : W ? 64 * W : 1024) void add_rmsnorm_quant_kernel(NormArgs a) {
  __shared__ float red[16];
  const int step = L ? L : W ? 64 * W : (int)blockDim.x;
  const int lane = (int)threadIdx.x % step;
  const int64_t row = L ? (int64_t)blockIdx.x * (256 / (L ? L : 1)) + threadIdx.x / step
                        : (int64_t)blockIdx.x;
  if (L && row >= a.M) return;  // all lanes of a row; no barrier follows
  const u32x4* x = reinterpret_cast<const u32x4*>(a.x + row * a.ld_x);
  const u32x4* __restrict__ wt = reinterpret_cast<const u32x4*>(a.weight);

  u32x4 hv[CH];
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    const int c = lane + step * i;
    hv[i] = u32x4{0u, 0u, 0u, 0u};
    if (c < a.nc) hv[i] = __builtin_nontemporal_load(x + c);
  }
  if (a.res) {
    const u32x4* res = reinterpret_cast<const u32x4*>(a.res + row * a.ld_res);
    u32x4 rv[CH];
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int c = lane + step * i;
      rv[i] = u32x4{0u, 0u, 0u, 0u};
      if (c < a.nc) rv[i] = __builtin_nontemporal_load(res + c);
    }
    u32x4* h = reinterpret_cast<u32x4*>(a.h + row * a.ld_h);
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int c = lane + step * i;
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
    const int c = lane + step * i;
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
  const float r = row_rstd(row_sum<L, W>(ss, red), 0.125f / (float)a.nc, a.eps);

  if (a.xq) {
    float* sa = a.sa + row * (a.nc >> 4);
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int c = lane + step * i;
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
      const int c = lane + step * i;
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
template <int CH>
struct BwdRow {
  u32x4 g[CH], h[CH], s[CH];
  __device__ __forceinline__ void load(const NormBwdArgs& a, int64_t row, int c0, int step) {
    const u32x4* dy = reinterpret_cast<const u32x4*>(a.dy + row * a.ld_dy);
    const u32x4* hp = reinterpret_cast<const u32x4*>(a.h + row * a.ld_h);
    const u32x4* dh = reinterpret_cast<const u32x4*>(a.dh + row * a.ld_dh);
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int c = c0 + step * i;
      g[i] = h[i] = s[i] = u32x4{0u, 0u, 0u, 0u};
      if (c < a.nc) {
        g[i] = __builtin_nontemporal_load(dy + c);
        h[i] = __builtin_nontemporal_load(hp + c);
      }
    }
    if (a.dh) {
#pragma unroll
      for (int i = 0; i < CH; ++i) {
        const int c = c0 + step * i;
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
  __device__ __forceinline__ void finish(const NormBwdArgs& a, int64_t row, int c0, int step,
                                         u32x4 (&wt)[CH], float r, float lean,
                                         float (&acc)[CH][8]) {
    u32x4* dx = reinterpret_cast<u32x4*>(a.dx + row * a.ld_dx);
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      // widened again from the 16-byte chunks: kept from sums(), the float32 values would take
      // twice the registers of what was loaded all through the reduction
      asm volatile("" : "+v"(h[i]), "+v"(g[i]), "+v"(wt[i]));
      const int c = c0 + step * i;
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

template <int CH>
__device__ __forceinline__ void load_weights(const NormBwdArgs& a, int c0, int step,
                                             u32x4 (&wt)[CH]) {
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    const int c = c0 + step * i;
    wt[i] = c < a.nc ? reinterpret_cast<const u32x4*>(a.weight)[c] : u32x4{0u, 0u, 0u, 0u};
  }
}

template <int CH>
__device__ __forceinline__ void store_part(const NormBwdArgs& a, int c0, int step,
                                           const float (&acc)[CH][8]) {
  float4* part = reinterpret_cast<float4*>(a.part) + (int64_t)blockIdx.x * (2 * a.nc);
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    const int c = c0 + step * i;
    if (c >= a.nc) continue;
    part[2 * c] = make_float4(acc[i][0], acc[i][1], acc[i][2], acc[i][3]);
    part[2 * c + 1] = make_float4(acc[i][4], acc[i][5], acc[i][6], acc[i][7]);
  }
}

}  // namespace

// Rows of up to 64 CH chunks: L lanes of a wave take a whole row (64 / L rows a wave), with no
// barrier between the RW waves of a workgroup; the rows' shares of dw are added across the wave and
// then through LDS at the end, in a fixed order.
template <int RW, int CH, int L>
__global__ __launch_bounds__(64 * RW, 2) void add_rmsnorm_bwd_wave_kernel(NormBwdArgs a) {
  __shared__ float red[RW / 2][CH * 8][L];
  const int lane = (int)threadIdx.x % L, wave = (int)(threadIdx.x >> 6);
  const float inv_k = 0.125f / (float)a.nc;
  u32x4 wt[CH];
  load_weights<CH>(a, lane, L, wt);
  float acc[CH][8];
#pragma unroll
  for (int i = 0; i < CH; ++i)
#pragma unroll
    for (int k = 0; k < 8; ++k) acc[i][k] = 0.f;

  constexpr int kRows = RW * 64 / L;  // of a workgroup's pass
  for (int64_t row = (int64_t)blockIdx.x * kRows + threadIdx.x / L; row < a.M;
       row += (int64_t)gridDim.x * kRows) {
    BwdRow<CH> v;
    v.load(a, row, lane, L);
    float ss, sd;
    v.sums(wt, ss, sd);
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) {
      ss += __shfl_xor(ss, o, 64);
      sd += __shfl_xor(sd, o, 64);
    }
    const float r = row_rstd(ss, inv_k, a.eps);
    v.finish(a, row, lane, L, wt, r, r * r * (sd * inv_k), acc);
  }
  if (!a.part) return;
#pragma unroll
  for (int o = L; o < 64; o <<= 1)
#pragma unroll
    for (int i = 0; i < CH; ++i)
#pragma unroll
      for (int k = 0; k < 8; ++k) acc[i][k] += __shfl_xor(acc[i][k], o, 64);
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
  if (threadIdx.x < L) store_part<CH>(a, lane, L, acc);
}

// A workgroup of as many waves as a row needs takes a row at a time; AHEAD: the next row's loads
// are in flight while it reduces (rows past K = 16384 would not fit the registers twice). 268 MB at
// 8192 x 4096 in 50 us, 5.4 TB/s: what a copy of this size reaches.
template <int CH, bool AHEAD>
__global__ __launch_bounds__(1024) void add_rmsnorm_bwd_kernel(NormBwdArgs a) {
  __shared__ float red[2][2][16];
  const int t = (int)threadIdx.x, step = (int)blockDim.x, waves = step >> 6;
  const float inv_k = 0.125f / (float)a.nc;
  u32x4 wt[CH];
  load_weights<CH>(a, t, step, wt);
  float acc[CH][8];
#pragma unroll
  for (int i = 0; i < CH; ++i)
#pragma unroll
    for (int k = 0; k < 8; ++k) acc[i][k] = 0.f;

  int buf = 0;
  BwdRow<CH> v;
  int64_t row = blockIdx.x;
  if (AHEAD && row < a.M) v.load(a, row, t, step);
  for (; row < a.M; row += gridDim.x, buf ^= 1) {
    // in place of dy or dh: the next row's values are read before this row's are written, and no
    // other workgroup writes them
    BwdRow<CH> next;
    if (!AHEAD) v.load(a, row, t, step);
    if (AHEAD && row + gridDim.x < a.M) next.load(a, row + gridDim.x, t, step);
    float ss, sd;
    v.sums(wt, ss, sd);
    ss = wave_sum(ss);
    sd = wave_sum(sd);
    // two buffers: a wave writes row n + 2's sums only after the barrier of row n + 1, which no
    // wave reaches before it has read row n's
    if ((t & 63) == 0) red[buf][0][t >> 6] = ss, red[buf][1][t >> 6] = sd;
    __syncthreads();
    ss = red[buf][0][0], sd = red[buf][1][0];
    for (int k = 1; k < waves; ++k) ss += red[buf][0][k], sd += red[buf][1][k];
    const float r = row_rstd(ss, inv_k, a.eps);
    v.finish(a, row, t, step, wt, r, r * r * (sd * inv_k), acc);
    if (AHEAD) v = next;
  }
  if (a.part) store_part<CH>(a, t, step, acc);
}

// dw[k] = sum over the groups of their partial sums, in a fixed order: 8 columns of 4 values per
// workgroup and 64 threads down each column with 8 loads in flight each, so that 512 groups are one
// round of loads.
__global__ __launch_bounds__(512) void norm_dw_kernel(const f32x4* __restrict__ part, int groups,
                                                      int nc4, float* __restrict__ dw) {
  __shared__ float red[8][32];
  const int col = threadIdx.x & 7, g0 = threadIdx.x >> 3;
  const f32x4* p = part + blockIdx.x * 8 + col;  // K % 128 == 0: every column exists
  f32x4 s = {0.f, 0.f, 0.f, 0.f};
  for (int g = g0; g < groups; g += 64 * 8) {
    f32x4 v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      v[i] = f32x4{0.f, 0.f, 0.f, 0.f};
      if (g + 64 * i < groups) v[i] = p[(int64_t)(g + 64 * i) * nc4];
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) s += v[i];
  }
#pragma unroll
  for (int o = 8; o < 64; o <<= 1) {
    s.x += __shfl_xor(s.x, o, 64), s.y += __shfl_xor(s.y, o, 64);
    s.z += __shfl_xor(s.z, o, 64), s.w += __shfl_xor(s.w, o, 64);
  }
  if ((threadIdx.x & 63) < 8) *reinterpret_cast<f32x4*>(&red[threadIdx.x >> 6][4 * col]) = s;
  __syncthreads();
  if (threadIdx.x < 32) {
    float sum = red[0][threadIdx.x];
#pragma unroll
    for (int k = 1; k < 8; ++k) sum += red[k][threadIdx.x];
    dw[blockIdx.x * 32 + threadIdx.x] = sum;
  }
}

namespace {

// L lanes per row, or a workgroup of the waves that nc chunks need at CH a lane.
template <int CH, int L, int W = 0>
void run_norm(const NormArgs& a, hipStream_t stream) {
  const int64_t rows = L ? 256 / (L ? L : 1) : 1;
  const int threads = L ? 256 : 64 * ((a.nc + 64 * CH - 1) / (64 * CH));
  const dim3 grid((unsigned)((a.M + rows - 1) / rows));
  hipLaunchKernelGGL((add_rmsnorm_quant_kernel<CH, L, W>), grid, dim3(threads), 0, stream, a);
}

}  // namespace

// Which lanes share a row. Up to 64 chunks (K <= 512) a wave or a part of one: at K = 128 and
// 262144 rows 47 us against 298 us with a workgroup per row. Up to 256 chunks (K <= 2048) a wave per row
// when there are 8192 rows or more: 42.8 against 46.6 us (K = 1024, 32768 rows) and 45.4 against
// 54.3 us (K = 1152), but 6.4 against 5.2 us at 2048 rows of K = 1024, where a quarter of the waves
// is too few to hide the loads. Wider rows by about four waves, 2 to 4 chunks a lane; up to 512
// rows (two a CU) by one chunk a lane, up to 16 waves: 4.0 against 4.8 us (64 rows, K = 4096), 4.7
// against 6.1 us (K = 8192). Four waves at one or two chunks a lane (K of 1664 to 2048 and 3200 to
// 4096) have a form with their number known (its sums unrolled): 42.2 against 43.8 us at 8192 x
// 4096. Four waves at three or four chunks (4736 to 6144, 6272 to 8192) have none, which would save
// 1 to 3 %: 49.9 against 51.6 us at 8192 x 5120, 42.5 against 43.2 us at 4096 x 8192.
// 8192 x 4096 is 134 MB read and 102 MB written, 5.6 TB/s: more than a copy (5.2 - 5.5 TB/s), less
// than reads or writes alone (6.4 and 6.9 TB/s). With power-of-two scales, whose codes wait for the
// row's sum, 42.9 against 40.6 us.
hipError_t launch_add_rmsnorm_quant(const NormArgs& a, hipStream_t stream) {
  const bool few = a.M <= 512, many = a.M >= 8192;
  if (a.nc <= 16) run_norm<1, 16>(a, stream);
  else if (a.nc <= 32) run_norm<1, 32>(a, stream);
  else if (a.nc <= 64) run_norm<1, 64>(a, stream);
  else if (many && a.nc <= 128) run_norm<2, 64>(a, stream);
  else if (many && a.nc <= 192) run_norm<3, 64>(a, stream);
  else if (many && a.nc <= 256) run_norm<4, 64>(a, stream);
  else if (!few && a.nc > 192 && a.nc <= 256) run_norm<1, 0, 4>(a, stream);
  else if (!few && a.nc > 384 && a.nc <= 512) run_norm<2, 0, 4>(a, stream);
  else if (a.nc <= (few ? 1024 : 256)) run_norm<1, 0>(a, stream);
  else if (a.nc <= (few ? 2048 : 512)) run_norm<2, 0>(a, stream);
  else if (!few && a.nc <= 768) run_norm<3, 0>(a, stream);
  else run_norm<4, 0>(a, stream);
  return hipGetLastError();
}

namespace {

// How the backward pass of M rows of nc chunks is cut up. A wave per row up to 256 chunks
// (K <= 2048) once there are more than 512 rows (27.4 us at 8192 x 2048, 5.1 TB/s; 8.6 us against
// 7.9 us by workgroups at 512 rows, 8.9 against 12.5 us at 1024); wider rows by a workgroup each
// (49.8 against 55.3 us at 8192 x 4096, where a wave would hold 256 registers). Every workgroup
// leaves K partial sums: 512 of them keep all CUs busy twice (56 us at 4096 x 8192, 256: 60 us; 49.8
// us at 8192 x 4096, 1024: 56 us), 256 are enough up to 1024 rows (10.0 against 12.1 us at
// 512 x 4096). A single one's sums are dw, without the second kernel: up to 8 rows by a wave each
// (K = 2048: 4.5 us a call of 4 rows from the host, two kernels 6.0), up to 2 of wider rows one after
// the other (K = 4096: 4.0 against 6.0 us, but 6.4 us for 4).
struct BwdShape {
  int lanes;       // of a wave that share a row; 0: a workgroup takes a row
  int rw;          // lanes > 0: waves of a workgroup
  int ch;          // chunks of a lane
  int64_t groups;  // workgroups
};
BwdShape bwd_shape(int64_t M, int64_t nc) {
  if (nc <= 64 || (nc <= 256 && (M > 512 || M <= 8))) {
    const int lanes = nc <= 16 ? 16 : nc <= 32 ? 32 : 64;
    const int ch = nc <= 64 ? 1 : nc <= 128 ? 2 : 4;
    const int rw = M * lanes >= 8 * 256 * 64 || M <= 8 ? 8 : 4;
    const int64_t most = 256 * (8 / rw), rows = rw * 64 / lanes, g = (M + rows - 1) / rows;
    return {lanes, rw, ch, g < most ? g : most};
  }
  const int ch = M <= 512 && nc <= 1024 ? 1 : nc <= 2048 ? 2 : 4;
  const int64_t most = M <= 2 ? 1 : M > 1024 && nc <= 1024 ? 512 : 256;
  return {0, 0, ch, M < most ? M : most};
}

template <int RW, int CH, int L>
void run_bwd_wave(const NormBwdArgs& a, int64_t groups, hipStream_t stream) {
  hipLaunchKernelGGL((add_rmsnorm_bwd_wave_kernel<RW, CH, L>), dim3((unsigned)groups),
                     dim3(64 * RW), 0, stream, a);
}
template <int RW>
void run_bwd_waves(const NormBwdArgs& a, const BwdShape& s, hipStream_t stream) {
  if (s.lanes == 16) run_bwd_wave<RW, 1, 16>(a, s.groups, stream);
  else if (s.lanes == 32) run_bwd_wave<RW, 1, 32>(a, s.groups, stream);
  else if (s.ch == 1) run_bwd_wave<RW, 1, 64>(a, s.groups, stream);
  else if (s.ch == 2) run_bwd_wave<RW, 2, 64>(a, s.groups, stream);
  else run_bwd_wave<RW, 4, 64>(a, s.groups, stream);
}
template <int CH, bool AHEAD>
void run_bwd(const NormBwdArgs& a, int64_t groups, hipStream_t stream) {
  const int threads = 64 * ((a.nc + 64 * CH - 1) / (64 * CH));
  hipLaunchKernelGGL((add_rmsnorm_bwd_kernel<CH, AHEAD>), dim3((unsigned)groups), dim3(threads), 0,
                     stream, a);
}

}  // namespace

int64_t norm_bwd_groups(int64_t M, int64_t K) { return bwd_shape(M, K / 8).groups; }

hipError_t launch_add_rmsnorm_bwd(const NormBwdArgs& args, float* dw, hipStream_t stream) {
  NormBwdArgs a = args;
  const BwdShape s = bwd_shape(a.M, a.nc);
  // the sums of a single workgroup are dw
  const bool direct = dw && s.groups == 1 && reinterpret_cast<uintptr_t>(dw) % 16 == 0;
  if (direct) a.part = dw;
  if (s.groups > 0) {
    if (s.lanes && s.rw == 8) run_bwd_waves<8>(a, s, stream);
    else if (s.lanes) run_bwd_waves<4>(a, s, stream);
    else if (s.ch == 1) run_bwd<1, true>(a, s.groups, stream);
    else if (s.ch == 2) run_bwd<2, true>(a, s.groups, stream);
    else run_bwd<4, false>(a, s.groups, stream);
    if (hipError_t e = hipGetLastError(); e != hipSuccess) return e;
  }
  if (!dw || direct) return hipSuccess;
  hipLaunchKernelGGL(norm_dw_kernel, dim3((unsigned)(a.nc / 4)), dim3(512), 0, stream,
                     reinterpret_cast<const f32x4*>(a.part), (int)s.groups, 2 * a.nc, dw);
  return hipGetLastError();
}

}  // namespace fp8rl
