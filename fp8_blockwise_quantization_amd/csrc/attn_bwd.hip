// Gradients of attention of packed documents: two passes over the scores, one for dq (a query's sums
// stay in one workgroup) and one for dk and dv (a key's do), so that nothing is added atomically
// and the result has the same bits every time. Seven products instead of the five that one
// pass with atomic sums would need.
//
// dq: as the forward pass, 128 queries a workgroup, queries in the columns. Per tile of 64 keys
//   S^T = K Q^T,  dP^T = V dO^T,  P = exp(S - lse),  dS = P (dP - delta),  dQ^T += K^T dS^T,
// where delta = <dout, out> of a query, formed first and left in the workspace for the second pass.
//
// dk, dv: 128 keys a workgroup, keys in the columns, through the tiles of 64 queries of all heads
// that share the keys:
//   S = Q K^T,  dP = dO V^T,  dV^T += dO^T P,  dK^T += Q^T dS.
#include "attn_tile.hpp"

namespace fp8rl {

namespace {

constexpr int kWaves = 4;
constexpr int kOwn = 128;   // rows of a workgroup
constexpr int kPass = 64;   // rows of a tile that it goes through

}  // namespace

template <int DP, bool PAD, bool MORE>
__global__ __launch_bounds__(256, 2) void attn_dq_kernel(AttnArgs d) {
  constexpr int KS = DP / 16, DT = DP / 32;
  __shared__ __align__(1024) uint8_t s_k[2][kPass * DP * 2];
  __shared__ __align__(1024) uint8_t s_v[2][kPass * DP * 2];
  const fp8rl_attn_args& a = d.a;
  const int lane = (int)(threadIdx.x & 63), h = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const int D = PAD ? a.head_dim : DP;

  const int id = (int)blockIdx.x;  // (the order is the forward pass's)
  const int kv = id % a.kv_heads;
  const int head = kv * d.group + id / a.kv_heads % d.group;
  const DocTile t = find_tile<kOwn, false>(a, d.slots - 1 - id / a.q_heads, lane);
  if (t.doc >= (int)a.docs) return;
  const Mask mask(a, t);
  const int shift = t.lk - t.lq;
  const int row = t.first + 32 * wave + (lane & 31);
  const int p = row + shift;
  const int rows = min(32, t.lq - t.first - 32 * wave);
  const int p0 = t.first + 32 * wave + shift, p1 = p0 + rows - 1;
  const bool in = row < t.lq;
  const int64_t qrow = t.q0 + min(row, t.lq - 1);

  bf16x8 q[KS], g[KS];
  float delta = 0.f;
  {
    const uint16_t* qp = a.q + qrow * a.ld_q + (int64_t)head * D;
    const uint16_t* gp = a.dout + qrow * a.ld_dout + (int64_t)head * D;
    const uint16_t* op = a.out + qrow * a.ld_out + (int64_t)head * D;
#pragma unroll
    for (int s = 0; s < KS; ++s) {
      q[s] = row_operand(qp, s, h, D);
      g[s] = row_operand(gp, s, h, D);
      float x[8], y[8];
      widen8(__builtin_bit_cast(u32x4, g[s]), x);
      widen8(__builtin_bit_cast(u32x4, row_operand(op, s, h, D)), y);
#pragma unroll
      for (int e = 0; e < 8; ++e) delta = __builtin_fmaf(x[e], y[e], delta);
    }
    const auto x = __builtin_amdgcn_permlane32_swap(__float_as_uint(delta), __float_as_uint(delta),
                                                    false, false);
    delta = __uint_as_float(x[0]) + __uint_as_float(x[1]);
    if (in && h == 0) d.delta[head * a.Tq + qrow] = delta;
  }
  // a query that sees nothing: exp(S - inf) = 0 throughout
  float lse2 = a.lse[head * a.Tq + qrow] * kLog2e;
  if (lse2 == -__builtin_inff()) lse2 = __builtin_inff();

  const int first = t.first + shift, last = min(t.first + kOwn, t.lq) - 1 + shift;
  const int in_prefix = (mask.prefix + kPass - 1) / kPass;
  const int begin = max(mask.lo(first) / kPass, in_prefix);
  const int tiles = in_prefix + max(0, (mask.hi(last) + kPass - 1) / kPass - begin);
  auto key_of = [&](int i) { return kPass * (i < in_prefix ? i : i - in_prefix + begin); };

  const RowLoader<DP, kPass, kWaves> load_k(a.ld_k, D, wave, lane), load_v(a.ld_v, D, wave, lane);
  const uint16_t* const k0 = a.k + t.k0 * a.ld_k + (int64_t)kv * D;
  const uint16_t* const v0 = a.v + t.k0 * a.ld_v + (int64_t)kv * D;
  auto load = [&](int i) {
    const int j = key_of(i);
    load_k.load(k0 + j * a.ld_k, t.lk - j, s_k[i & 1], wave);
    load_v.load(v0 + j * a.ld_v, t.lk - j, s_v[i & 1], wave);
  };
  const bool capped = MORE && a.cap > 0.f, sloped = MORE && a.slopes;
  const float slope2 = sloped ? a.slopes[head] * kLog2e : 0.f;

  f32x16 o[DT];
#pragma unroll
  for (int i = 0; i < DT; ++i) o[i] = zeros16();

  if (tiles > 0) load(0);
  for (int i = 0; i < tiles; ++i) {
    landed();
    if (i + 1 < tiles) load(i + 1);
    const int j0 = key_of(i), keys = min(kPass, t.lk - j0);
    if (keys < kPass) {
      clear_rows<DP, kPass, kWaves>(s_k[i & 1], keys);
      __syncthreads();
    }
    if (rows <= 0 || !mask.any(p0, p1, j0, j0 + keys)) continue;
    const bool all = keys == kPass && mask.all(p0, p1, j0, j0 + kPass);
    const int lo = mask.lo(p), hi = mask.hi(p);
    const RowOperand<DP> kop(s_k[i & 1], lane), vop(s_v[i & 1], lane);
    const ColOperand<DP> kt(s_k[i & 1], lane);
#pragma unroll
    for (int r = 0; r < 2; ++r) {  // 32 keys
      f32x16 s = zeros16(), dp = zeros16();
#pragma unroll
      for (int c = 0; c < KS; ++c) {
        if (PAD && 16 * c >= D) break;
        s = __builtin_amdgcn_mfma_f32_32x32x16_bf16(kop(32 * r, c), q[c], s, 0, 0, 0);
        dp = __builtin_amdgcn_mfma_f32_32x32x16_bf16(vop(32 * r, c), g[c], dp, 0, 0, 0);
      }
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        const int j = j0 + 32 * r + 8 * (e >> 2) + 4 * h + (e & 3);
        float x = s[e] * d.scale2, slant = 1.f;
        if (capped) {
          const float th = tanh_cap(x);
          x = d.cap2 * th;
          slant = 1.f - th * th;
        }
        if (sloped) x -= slope2 * fabsf((float)(p - j));
        float ds = exp2_fast(x - lse2) * (dp[e] - delta);
        if (capped) ds *= slant;
        if (!all) ds = j < mask.prefix || (j >= lo && j < hi) ? ds : 0.f;
        s[e] = ds;
      }
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const bf16x8 w = operand_of(s, u);
#pragma unroll
        for (int c = 0; c < DT; ++c) {
          if (PAD && 32 * c >= D) break;
          o[c] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(kt(32 * r + 16 * u, c), w, o[c], 0, 0, 0);
        }
      }
    }
  }
  if (rows <= 0) return;
  uint16_t* const out = a.dq + (t.q0 + row) * a.ld_dq + (int64_t)head * D;
#pragma unroll
  for (int c = 0; c < DT; ++c) store_columns(o[c], a.sm_scale, out, 32 * c, h, D, in);
}

template <int DP, bool PAD, bool MORE>
__global__ __launch_bounds__(256, 1) void attn_dkv_kernel(AttnArgs d) {
  constexpr int KS = DP / 16, DT = DP / 32;
  __shared__ __align__(1024) uint8_t s_q[2][kPass * DP * 2];
  __shared__ __align__(1024) uint8_t s_g[2][kPass * DP * 2];
  __shared__ __align__(1024) float s_row[2][2][kPass];  // lse and delta of the tile's queries
  const fp8rl_attn_args& a = d.a;
  const int lane = (int)(threadIdx.x & 63), h = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const int D = PAD ? a.head_dim : DP;

  const int id = (int)blockIdx.x;
  const int kv = id % a.kv_heads;
  const DocTile t = find_tile<kOwn, true>(a, id / a.kv_heads, lane);
  if (t.doc >= (int)a.docs) return;
  const Mask mask(a, t);
  const int shift = t.lk - t.lq;
  const int key = t.first + 32 * wave + (lane & 31);
  const int keys = min(32, t.lk - t.first - 32 * wave);  // of this wave
  const int j0 = t.first + 32 * wave, j1 = j0 + keys;

  bf16x8 k[KS], v[KS];
  {
    const int64_t krow = t.k0 + min(key, t.lk - 1);
    const uint16_t* kp = a.k + krow * a.ld_k + (int64_t)kv * D;
    const uint16_t* vp = a.v + krow * a.ld_v + (int64_t)kv * D;
#pragma unroll
    for (int s = 0; s < KS; ++s) k[s] = row_operand(kp, s, h, D), v[s] = row_operand(vp, s, h, D);
  }

  // the queries that see any of the workgroup's keys, in whole tiles, for each head of the group
  int begin = 0, end = t.lq;
  if (t.first >= mask.prefix) {
    const int past = min(t.first + kOwn, t.lk);  // behind the last key
    if (mask.causal) begin = max(0, t.first - shift);
    if (mask.window) end = (int)min((int64_t)t.lq, (int64_t)past + mask.window - 1 - shift);
  }
  begin /= kPass;
  const int per = max(0, (end + kPass - 1) / kPass - begin);
  const int tiles = per * d.group;

  const RowLoader<DP, kPass, kWaves> load_q(a.ld_q, D, wave, lane), load_g(a.ld_dout, D, wave, lane);
  auto load = [&](int i) {
    const int in_group = i / per;
    const int head = kv * d.group + in_group, r0 = kPass * (i - in_group * per + begin);
    const int64_t row = t.q0 + r0;
    load_q.load(a.q + row * a.ld_q + (int64_t)head * D, t.lq - r0, s_q[i & 1], wave);
    load_g.load(a.dout + row * a.ld_dout + (int64_t)head * D, t.lq - r0, s_g[i & 1], wave);
    if (wave < 2)
      dma_floats((wave == 0 ? a.lse : d.delta) + head * a.Tq + row,
                 4 * (uint32_t)min(lane, t.lq - r0 - 1), s_row[i & 1][wave]);
  };
  const bool capped = MORE && a.cap > 0.f, sloped = MORE && a.slopes;

  f32x16 dk[DT], dv[DT];
#pragma unroll
  for (int i = 0; i < DT; ++i) dk[i] = zeros16(), dv[i] = zeros16();

  if (tiles > 0) load(0);
  for (int i = 0; i < tiles; ++i) {
    landed();
    if (i + 1 < tiles) load(i + 1);
    const int in_group = i / per;
    const int head = kv * d.group + in_group, r0 = kPass * (i - in_group * per + begin);
    const int rows = min(kPass, t.lq - r0);
    if (rows < kPass) {
      clear_rows<DP, kPass, kWaves>(s_q[i & 1], rows);
      clear_rows<DP, kPass, kWaves>(s_g[i & 1], rows);
      __syncthreads();
    }
    const float slope2 = sloped ? a.slopes[head] * kLog2e : 0.f;
    const RowOperand<DP> qop(s_q[i & 1], lane), gop(s_g[i & 1], lane);
    const ColOperand<DP> qt(s_q[i & 1], lane), gt(s_g[i & 1], lane);
#pragma unroll
    for (int r = 0; r < 2; ++r) {  // 32 queries
      const int n = min(32, rows - 32 * r);
      const int p0 = r0 + 32 * r + shift;
      if (keys <= 0 || n <= 0 || !mask.any(p0, p0 + n - 1, j0, j1)) continue;
      const bool all = n == 32 && keys == 32 && mask.all(p0, p0 + 31, j0, j1);
      f32x16 s = zeros16(), dp = zeros16();
#pragma unroll
      for (int c = 0; c < KS; ++c) {
        if (PAD && 16 * c >= D) break;
        s = __builtin_amdgcn_mfma_f32_32x32x16_bf16(qop(32 * r, c), k[c], s, 0, 0, 0);
        dp = __builtin_amdgcn_mfma_f32_32x32x16_bf16(gop(32 * r, c), v[c], dp, 0, 0, 0);
      }
#pragma unroll
      for (int e4 = 0; e4 < 4; ++e4) {
        const f32x4 lse = *reinterpret_cast<const f32x4*>(&s_row[i & 1][0][32 * r + 8 * e4 + 4 * h]);
        const f32x4 delta =
            *reinterpret_cast<const f32x4*>(&s_row[i & 1][1][32 * r + 8 * e4 + 4 * h]);
#pragma unroll
        for (int f = 0; f < 4; ++f) {
          const int e = 4 * e4 + f;
          const int at = 8 * e4 + 4 * h + f, p = p0 + at;
          float x = s[e] * d.scale2, slant = 1.f;
          if (capped) {
            const float th = tanh_cap(x);
            x = d.cap2 * th;
            slant = 1.f - th * th;
          }
          if (sloped) x -= slope2 * fabsf((float)(p - key));
          float w = exp2_fast(x - lse[f] * kLog2e);
          float ds = w * (dp[e] - delta[f]);
          if (capped) ds *= slant;
          if (!all) {
            const bool seen = at < n && key < t.lk && mask.sees(p, key);
            w = seen ? w : 0.f;
            ds = seen ? ds : 0.f;
          }
          s[e] = w;
          dp[e] = ds;
        }
      }
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const bf16x8 w = operand_of(s, u), ds = operand_of(dp, u);
#pragma unroll
        for (int c = 0; c < DT; ++c) {
          if (PAD && 32 * c >= D) break;
          dv[c] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(gt(32 * r + 16 * u, c), w, dv[c], 0, 0, 0);
          dk[c] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(qt(32 * r + 16 * u, c), ds, dk[c], 0, 0, 0);
        }
      }
    }
  }
  if (keys <= 0) return;
  const bool in = key < t.lk;
  uint16_t* const ok = a.dk + (t.k0 + key) * a.ld_dk + (int64_t)kv * D;
  uint16_t* const ov = a.dv + (t.k0 + key) * a.ld_dv + (int64_t)kv * D;
#pragma unroll
  for (int c = 0; c < DT; ++c) {
    store_columns(dk[c], a.sm_scale, ok, 32 * c, h, D, in);
    store_columns(dv[c], 1.f, ov, 32 * c, h, D, in);
  }
}

hipError_t launch_attn_bwd(const fp8rl_attn_args& a, float* delta, hipStream_t stream) {
  AttnArgs q = attn_args(a, kOwn, a.Tq), k = attn_args(a, kOwn, a.Tk);
  q.delta = k.delta = delta;
  const dim3 grid_q((unsigned)(q.slots * a.q_heads)), grid_k((unsigned)(k.slots * a.kv_heads));
  auto go = [&](auto dq, auto dkv) {
    hipLaunchKernelGGL(dq, grid_q, dim3(64 * kWaves), 0, stream, q);
    hipLaunchKernelGGL(dkv, grid_k, dim3(64 * kWaves), 0, stream, k);
  };
  const bool more = a.cap > 0.f || a.slopes;
  if (a.head_dim == 64)
    more ? go(attn_dq_kernel<64, false, true>, attn_dkv_kernel<64, false, true>)
         : go(attn_dq_kernel<64, false, false>, attn_dkv_kernel<64, false, false>);
  else if (a.head_dim < 64)
    more ? go(attn_dq_kernel<64, true, true>, attn_dkv_kernel<64, true, true>)
         : go(attn_dq_kernel<64, true, false>, attn_dkv_kernel<64, true, false>);
  else if (a.head_dim < 128)
    more ? go(attn_dq_kernel<128, true, true>, attn_dkv_kernel<128, true, true>)
         : go(attn_dq_kernel<128, true, false>, attn_dkv_kernel<128, true, false>);
  else
    more ? go(attn_dq_kernel<128, false, true>, attn_dkv_kernel<128, false, true>)
         : go(attn_dq_kernel<128, false, false>, attn_dkv_kernel<128, false, false>);
  return hipGetLastError();
}

}  // namespace fp8rl
