// Gradients of attention of packed documents: two passes over the scores, one for dq (a query's
// sums stay in one workgroup) and one for dk and dv (a key's do), so that nothing is added
// atomically and the result has the same bits every time. Seven products instead of the five that
// one pass with atomic sums would need.
//
// dq: as the forward pass, 128 queries a workgroup, queries in the columns. Per tile of 64 keys
//   S^T = K Q^T,  dP^T = V dO^T,  P = exp(S - lse),  dS = P (dP - delta),  dQ^T += K^T dS^T,
// where delta = <dout, out> of a query, formed first and left in the workspace (with lse in units
// of ln 2) for the second pass.
//
// dk, dv: 128 keys a workgroup, keys in the columns, through the tiles of 64 queries of all heads
// that share the keys:
//   S = Q K^T,  dP = dO V^T,  dV^T += dO^T P,  dK^T += Q^T dS.
// The sums take 128 of a wave's registers at heads of 128, so K stays there in part only and V in
// LDS, and two waves share 32 keys, each with half of a tile's queries; eight waves and three tiles
// in LDS fill a CU. (Four waves with everything in registers, one to a SIMD: 1635 us where this
// takes 1145; with all 64 queries at once in such a wave, or two workgroups of four waves, more
// than 2300.) Where there are few keys, a key tile's queries are dealt out in parts, whose sums a
// third kernel adds.
//
// P and dS go into their products as one bf16 term, 2^-8 of themselves at most: against 64 bits the
// gradients are off by 0.0024 to 0.0026 of their norm, with float32 terms by 0.0018 to 0.0020. Second
// terms would add three products to the seven.
//
// 8192 causal tokens, 32 query heads on 8 of 128: 770 us for dq, 1.07 PFLOP/s of its three
// products, 1145 us for dk and dv, 0.96 of their four; 1.9 ms in all, 0.72 PFLOP/s of the five that
// the gradients need. Memory: 2.1 GB read by the second pass, 1.9 TB/s.
#include <limits.h>

#include <type_traits>

#include "attn_tile.hpp"

namespace fp8rl {

namespace {

constexpr int kWaves = 4;
constexpr int kOwn = 128;   // rows of a workgroup
constexpr int kPass = 64;   // keys of a tile that the first pass goes through
constexpr int kQueries = 64; // queries of a tile that the second goes through
constexpr int kMostParts = 16;
// Workgroups up to which, and keys of a document (on the average) from which on, two waves share 32
// queries in the first pass: a tile takes less time with all of a CU's waves on it. All three
// kernels, one document of 4096 tokens, 8 heads on 1 of 128: 235 us, else 270; 3000 tokens, 8 on 8:
// 146, 170; 1024, 32 on 8: 86, 92. Documents of 128 on the average, 1024 in all: 68, else 60; one
// of 256: 34.1, 33.2. 576 workgroups, two documents of 2048 in all, 32 on 4: 170, 167.
constexpr int kFewQueries = 512, kLong = 512;

// The tiles of queries that see any of a workgroup's keys, those of the group's heads one after
// another.
struct QueryTiles {
  int begin, per, total;  // of a head: begin .. begin + per - 1
  __device__ __forceinline__ QueryTiles(const Mask& mask, const DocTile& t, int group) {
    const int shift = t.lk - t.lq;
    int first = 0, end = t.lq;
    if (t.first >= mask.prefix) {
      const int past = min(t.first + kOwn, t.lk);  // behind the last key
      if (mask.causal) first = max(0, t.first - shift);
      if (mask.window) end = min(t.lq, past + mask.window - 1 - shift);
    }
    begin = first / kQueries;
    per = max(0, (end + kQueries - 1) / kQueries - begin);
    total = per * group;
  }
  __device__ __forceinline__ int cut(int part, int parts) const {
    return (int)((int64_t)total * part / parts);
  }
};

// Products s into scores in units of ln 2, in their places; with a cap, ds times the capped score's
// slope, 1 - tanh^2.
template <typename Far>
__device__ __forceinline__ void finish_scores(f32x16& s, f32x16& ds, const AttnArgs& d, bool capped,
                                              bool sloped, float slope2, Far far) {
  if (capped) {
    tanh_places<16>(s, d.scale2);
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      ds[e] *= __builtin_fmaf(-s[e], s[e], 1.f);
      s[e] *= d.cap2;
    }
  } else {
#pragma unroll
    for (int e = 0; e < 16; ++e) s[e] *= d.scale2;
  }
  if (sloped) slope_scores(s, 1.f, slope2, far);
}

// Where a wave's lane keeps its part of dk (and behind it dv) of the keys of workgroup `tile`.
template <int DP>
__device__ __forceinline__ f32x4* part_of(const AttnArgs& d, int tile, int part, int wave, int lane) {
  return reinterpret_cast<f32x4*>(d.part) +
         (((int64_t)tile * d.parts + part) * kWaves + wave) * (2 * 32 * DP / 4) + lane;
}

}  // namespace

// KH: waves that share 32 queries, each with its part of a tile's keys; their sums meet in the end.
template <int DP, bool PAD, bool MORE, int KH>
__global__ __launch_bounds__(256 * KH, 2) void attn_dq_kernel(AttnArgs d) {
  constexpr int KS = DP / 16, DT = DP / 32;
  constexpr int kAll = 4 * KH, NR = 2 / KH;  // waves, a wave's 32-key parts of a tile
  constexpr int kTile = kPass * DP * 2;      // bytes
  __shared__ __align__(1024) uint8_t s_mem[4 * kTile];  // k and v of two tiles; then some waves' sums
  const fp8rl_attn_args& a = d.a;
  const int lane = (int)(threadIdx.x & 63), h = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const int block = wave & 3, part = wave >> 2;  // of the queries, of a tile's keys
  const int D = PAD ? a.head_dim : DP;

  const int id = (int)blockIdx.x;  // (the order is the forward pass's)
  const int kv = id % a.kv_heads;
  const int head = kv * d.group + id / a.kv_heads % d.group;
  const DocTile t = find_tile<kOwn, false>(d, id / a.q_heads, lane);
  if (t.doc >= (int)a.docs) return;
  const Mask mask(a, t);
  const int shift = t.lk - t.lq;
  const int row = t.first + 32 * block + (lane & 31);
  const int p = row + shift;
  const int rows = min(32, t.lq - t.first - 32 * block);
  const int p0 = t.first + 32 * block + shift, p1 = p0 + rows - 1;
  const bool in = row < t.lq;
  const int64_t qrow = t.q0 + min(row, t.lq - 1);

  const int first = t.first + shift, last = min(t.first + kOwn, t.lq) - 1 + shift;
  const int in_prefix = (mask.prefix + kPass - 1) / kPass;
  const int begin = max(mask.lo(first) / kPass, in_prefix);
  const int tiles = in_prefix + max(0, (mask.hi(last) + kPass - 1) / kPass - begin);
  auto key_of = [&](int i) { return kPass * (i < in_prefix ? i : i - in_prefix + begin); };

  const RowLoader<DP, kPass, kAll> rows_in(D, wave, lane);
  const uint16_t* const k0 = a.k + t.k0 * a.ld_k + (int64_t)kv * D;
  const uint16_t* const v0 = a.v + t.k0 * a.ld_v + (int64_t)kv * D;
  auto load = [&](int i) {
    const int j = key_of(i);
    rows_in.load(k0 + j * a.ld_k, a.ld_k, t.lk - j, s_mem + 2 * (i & 1) * kTile, wave);
    rows_in.load(v0 + j * a.ld_v, a.ld_v, t.lk - j, s_mem + (2 * (i & 1) + 1) * kTile, wave);
  };
  if (tiles > 0) load(0);

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
  }
  // a query that sees nothing: exp(S - inf) = 0 throughout
  float lse2 = a.lse[head * a.Tq + qrow] * kLog2e;
  if (lse2 == -__builtin_inff()) lse2 = __builtin_inff();
  if (in && h == 0 && part == 0) {
    d.stats[head * a.Tq + qrow] = lse2;
    d.stats[(a.q_heads + head) * a.Tq + qrow] = delta;
  }

  const bool capped = MORE && a.cap > 0.f, sloped = MORE && a.slopes;
  const float slope2 = sloped ? a.slopes[head] * kLog2e : 0.f;

  f32x16 o[DT];
#pragma unroll
  for (int i = 0; i < DT; ++i) o[i] = zeros16();

  for (int i = 0; i < tiles; ++i) {
    landed();
    if (i + 1 < tiles) load(i + 1);
    uint8_t *const s_k = s_mem + 2 * (i & 1) * kTile, *const s_v = s_k + kTile;
    const int tile = key_of(i), in_tile = min(kPass, t.lk - tile);
    if (in_tile < kPass) {
      clear_rows<DP, kPass, kAll>(s_k, in_tile);
      __syncthreads();
    }
    // this wave's keys
    constexpr int kMine = 32 * NR;
    const int j0 = tile + kMine * part, keys = min(kMine, t.lk - j0);
    if (rows <= 0 || keys <= 0 || !mask.any(p0, p1, j0, j0 + keys)) continue;
    const int lo = mask.lo(p), hi = mask.hi(p);
    const RowOperand<DP> kop(s_k + kMine * part * DP * 2, lane), vop(s_v + kMine * part * DP * 2, lane);
    const ColOperand<DP> kt(s_k + kMine * part * DP * 2, lane);
    f32x16 s, dp;
    auto weigh = [&](int r, auto masked) {  // dS in its place
      if (MORE) {
#pragma unroll
        for (int e = 0; e < 16; ++e) dp[e] -= delta;
        const float from = (float)(p - j0 - 32 * r - 4 * h);
        finish_scores(s, dp, d, capped, sloped, slope2,
                      [&](int e) { return from - (float)(8 * (e >> 2) + (e & 3)); });
      }
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        const int j = j0 + 32 * r + 8 * (e >> 2) + 4 * h + (e & 3);
        const float x = MORE ? s[e] - lse2 : __builtin_fmaf(s[e], d.scale2, -lse2);
        const float ds = exp2_fast(x) * (MORE ? dp[e] : dp[e] - delta);
        s[e] = !masked || (j < mask.prefix) | ((j >= lo) & (j < hi)) ? ds : 0.f;
      }
    };
    const bool all = keys == kMine && mask.all(p0, p1, j0, j0 + kMine);
#pragma unroll
    for (int r = 0; r < NR; ++r) {  // 32 keys
      s = zeros16(), dp = zeros16();
#pragma unroll
      for (int c = 0; c < KS; ++c) {
        if (PAD && 16 * c >= D) break;
        s = __builtin_amdgcn_mfma_f32_32x32x16_bf16(kop(32 * r, c), q[c], s, 0, 0, 0);
        dp = __builtin_amdgcn_mfma_f32_32x32x16_bf16(vop(32 * r, c), g[c], dp, 0, 0, 0);
      }
      if (all)
        weigh(r, std::false_type{});
      else
        weigh(r, std::true_type{});
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
  if (KH > 1) {
    landed();
    f32x4* const other = reinterpret_cast<f32x4*>(s_mem) + block * (64 * 4 * DT) + lane;
    if (part == 1) {
#pragma unroll
      for (int c = 0; c < 4 * DT; ++c) {
        const int e = 4 * (c & 3);
        other[64 * c] = f32x4{o[c >> 2][e], o[c >> 2][e + 1], o[c >> 2][e + 2], o[c >> 2][e + 3]};
      }
    }
    __syncthreads();
    if (part == 1) return;
#pragma unroll
    for (int c = 0; c < 4 * DT; ++c) {
      const f32x4 x = other[64 * c];
#pragma unroll
      for (int e = 0; e < 4; ++e) o[c >> 2][4 * (c & 3) + e] += x[e];
    }
  }
  if (rows <= 0) return;
  uint16_t* const out = a.dq + (t.q0 + row) * a.ld_dq + (int64_t)head * D;
#pragma unroll
  for (int c = 0; c < DT; ++c) store_columns(o[c], a.sm_scale, out, 32 * c, h, D, in);
}

template <int DP, bool PAD, bool MORE>
__global__ __launch_bounds__(512, 2) void attn_dkv_kernel(AttnArgs d) {
  constexpr int KS = DP / 16, DT = DP / 32;
  constexpr int kTile = kQueries * DP * 2;  // bytes
  // q and dout of three tiles, and v; in the end the sums of half of the waves
  __shared__ __align__(1024) uint8_t s_mem[6 * kTile + kOwn * DP * 2];
  __shared__ __align__(1024) float s_row[3][2][kQueries];  // lse and delta of the tile's queries
  // the steps of the keys' operand that do not fit the registers beside the sums (spilled, their
  // reloads would wait for the tiles in flight: with MORE at 128 whole columns five registers still
  // are)
  constexpr int kHeld = DP == 64 ? KS : MORE ? KS - 6 : KS - 4;
  __shared__ u32x4 s_k[4][KS - kHeld + 1][64];
  uint8_t* const s_v = s_mem + 6 * kTile;
  const fp8rl_attn_args& a = d.a;
  const int lane = (int)(threadIdx.x & 63), h = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const int block = wave & 3, half = wave >> 2;  // of the keys, of a tile's queries
  const int D = PAD ? a.head_dim : DP;

  const int id = (int)blockIdx.x;
  const int kv = id % a.kv_heads;
  const int part = id / a.kv_heads % d.parts;
  const DocTile t = find_tile<kOwn, true>(d, id / (a.kv_heads * d.parts), lane);
  if (t.doc >= (int)a.docs) return;
  const Mask mask(a, t);
  const int shift = t.lk - t.lq;
  const int j0 = t.first + 32 * block, key = j0 + (lane & 31);
  const int keys = min(32, t.lk - j0), j1 = j0 + keys;  // of this wave

  // the queries that see any of the workgroup's keys, in whole tiles, for each head of the group;
  // of these tiles the workgroup's part
  const QueryTiles all_tiles(mask, t, d.group);
  const int from = all_tiles.cut(part, d.parts), tiles = all_tiles.cut(part + 1, d.parts) - from;
  auto head_of = [&](int i) { return kv * d.group + (from + i) / all_tiles.per; };
  auto row_of = [&](int i) { return kQueries * ((from + i) % all_tiles.per + all_tiles.begin); };

  const RowLoader<DP, kQueries, 8> rows_in(D, wave, lane);
  constexpr int kLoads = 2 * RowLoader<DP, kQueries, 8>::kOps + 1;
  auto load = [&](int i) {
    const int head = head_of(i), r0 = row_of(i), at = i % 3;
    const int64_t row = t.q0 + r0;
    rows_in.load(a.q + row * a.ld_q + (int64_t)head * D, a.ld_q, t.lq - r0, s_mem + 2 * at * kTile,
                 wave);
    rows_in.load(a.dout + row * a.ld_dout + (int64_t)head * D, a.ld_dout, t.lq - r0,
                 s_mem + (2 * at + 1) * kTile, wave);
    // (the even waves all load the same, and so do the odd ones: every wave has as many loads in
    // flight)
    dma_floats(d.stats + ((wave & 1) * a.q_heads + head) * a.Tq + row,
               4 * (uint32_t)min(lane, t.lq - r0 - 1), s_row[at][wave & 1]);
  };

  // the keys stay in registers, their values in LDS
  RowLoader<DP, kOwn, 8>(D, wave, lane)
      .load(a.v + (t.k0 + t.first) * a.ld_v + (int64_t)kv * D, a.ld_v, t.lk - t.first, s_v, wave);
  if (tiles > 0) load(0);
  bf16x8 k[kHeld];
  {
    const uint16_t* kp = a.k + (t.k0 + min(key, t.lk - 1)) * a.ld_k + (int64_t)kv * D;
#pragma unroll
    for (int s = 0; s < kHeld; ++s) k[s] = row_operand(kp, s, h, D);
#pragma unroll
    for (int s = kHeld; s < KS; ++s)
      if (half == 0) s_k[block][s - kHeld][lane] = __builtin_bit_cast(u32x4, row_operand(kp, s, h, D));
  }
  const bool capped = MORE && a.cap > 0.f, sloped = MORE && a.slopes;
  const RowOperand<DP> vop(s_v + 32 * block * DP * 2, lane);

  f32x16 dk[DT], dv[DT];
#pragma unroll
  for (int i = 0; i < DT; ++i) dk[i] = zeros16(), dv[i] = zeros16();

  if (tiles > 1) load(1);
  for (int i = 0; i < tiles; ++i) {
    if (i + 1 < tiles)
      landed<kLoads>();
    else
      landed<0>();
    if (i + 2 < tiles) load(i + 2);
    uint8_t* const s_q = s_mem + 2 * (i % 3) * kTile;
    uint8_t* const s_g = s_q + kTile;
    const int r0 = row_of(i);
    const int in_tile = min(kQueries, t.lq - r0);
    if (in_tile < kQueries) {
      clear_rows<DP, kQueries, 8>(s_q, in_tile);
      clear_rows<DP, kQueries, 8>(s_g, in_tile);
      __syncthreads();
    }
    const int rows = min(32, in_tile - 32 * half);  // of this wave
    const int p0 = r0 + 32 * half + shift;
    if (keys <= 0 || rows <= 0 || !mask.any(p0, p0 + rows - 1, j0, j1)) continue;
    const float slope2 = sloped ? a.slopes[head_of(i)] * kLog2e : 0.f;
    const RowOperand<DP> qop(s_q + 32 * half * DP * 2, lane), gop(s_g + 32 * half * DP * 2, lane);
    const ColOperand<DP> qt(s_q + 32 * half * DP * 2, lane), gt(s_g + 32 * half * DP * 2, lane);

    f32x16 s = zeros16(), dp = zeros16();
#pragma unroll
    for (int c = 0; c < KS; ++c) {
      if (PAD && 16 * c >= D) break;
      const bf16x8 kc =
          c < kHeld ? k[c < kHeld ? c : 0] : __builtin_bit_cast(bf16x8, s_k[block][c - kHeld][lane]);
      s = __builtin_amdgcn_mfma_f32_32x32x16_bf16(qop(0, c), kc, s, 0, 0, 0);
    }
#pragma unroll
    for (int c = 0; c < KS; ++c) {
      if (PAD && 16 * c >= D) break;
      dp = __builtin_amdgcn_mfma_f32_32x32x16_bf16(gop(0, c), vop(0, c), dp, 0, 0, 0);
    }
    auto weigh = [&](auto masked) {  // P and dS in their places
      // the positions that see this lane's key: from <= p < to
      int from = 0, to = 0;
      if (masked) {
        const bool prefixed = key < mask.prefix;
        from = key >= t.lk ? INT_MAX : prefixed || !mask.causal ? INT_MIN : key;
        to = min(p0 + rows, prefixed || !mask.window ? INT_MAX : key + mask.window);
      }
      const float* const lse = &s_row[i % 3][0][32 * half + 4 * h];
      const float* const delta = &s_row[i % 3][1][32 * half + 4 * h];
      auto at = [](int e) { return 8 * (e >> 2) + (e & 3); };  // the query of place e, from 4h on
      if (MORE) {
#pragma unroll
        for (int e = 0; e < 16; ++e) dp[e] -= delta[at(e)];
        const float first = (float)(p0 + 4 * h - key);
        finish_scores(s, dp, d, capped, sloped, slope2,
                      [&](int e) { return first + (float)at(e); });
      }
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        const float x = MORE ? s[e] - lse[at(e)] : __builtin_fmaf(s[e], d.scale2, -lse[at(e)]);
        const int p = p0 + 4 * h + at(e);
        const bool seen = !masked || (p >= from) & (p < to);
        const float w = seen ? exp2_fast(x) : 0.f;
        const float ds = w * (MORE ? dp[e] : dp[e] - delta[at(e)]);
        s[e] = w;
        dp[e] = seen ? ds : 0.f;
      }
    };
    if (rows == 32 && keys == 32 && mask.all(p0, p0 + 31, j0, j1))
      weigh(std::false_type{});
    else
      weigh(std::true_type{});
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const bf16x8 w = operand_of(s, u), ds = operand_of(dp, u);
#pragma unroll
      for (int c = 0; c < DT; ++c) {
        if (PAD && 32 * c >= D) break;
        dv[c] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(gt(16 * u, c), w, dv[c], 0, 0, 0);
        dk[c] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(qt(16 * u, c), ds, dk[c], 0, 0, 0);
      }
    }
  }

  // the sums over the other half of the queries, 16 bytes a lane at a time
  landed<0>();
  static_assert(4 * 64 * 2 * 4 * DT * 16 <= sizeof(s_mem), "sums of four waves");
  f32x4* const other = reinterpret_cast<f32x4*>(s_mem) + block * (64 * 8 * DT) + lane;
  auto four = [](const f32x16 (&g)[DT], int c) {
    const int e = 4 * (c & 3);
    return f32x4{g[c >> 2][e], g[c >> 2][e + 1], g[c >> 2][e + 2], g[c >> 2][e + 3]};
  };
  if (half == 1) {
#pragma unroll
    for (int c = 0; c < 4 * DT; ++c) {
      other[64 * c] = four(dk, c);
      other[64 * (4 * DT + c)] = four(dv, c);
    }
  }
  __syncthreads();
  if (half == 1 || keys <= 0) return;
#pragma unroll
  for (int c = 0; c < 4 * DT; ++c) {
    const f32x4 x = other[64 * c], y = other[64 * (4 * DT + c)];
#pragma unroll
    for (int e = 0; e < 4; ++e) dk[c >> 2][4 * (c & 3) + e] += x[e], dv[c >> 2][4 * (c & 3) + e] += y[e];
  }
  if (d.parts > 1) {
    f32x4* const to = part_of<DP>(d, (id / (a.kv_heads * d.parts)) * a.kv_heads + kv, part, block, lane);
#pragma unroll
    for (int c = 0; c < 4 * DT; ++c) {
      to[64 * c] = four(dk, c);
      to[64 * (4 * DT + c)] = four(dv, c);
    }
    return;
  }
  const bool in = key < t.lk;
  uint16_t* const ok = a.dk + (t.k0 + key) * a.ld_dk + (int64_t)kv * D;
  uint16_t* const ov = a.dv + (t.k0 + key) * a.ld_dv + (int64_t)kv * D;
#pragma unroll
  for (int c = 0; c < DT; ++c) {
    store_columns(dk[c], a.sm_scale, ok, 32 * c, h, D, in);
    store_columns(dv[c], 1.f, ov, 32 * c, h, D, in);
  }
}

// The parts of dk and dv of a workgroup's keys, added in order: a wave per 32 keys and 32 columns
// of either.
template <int DP>
__global__ __launch_bounds__(256) void attn_dkv_join_kernel(AttnArgs d) {
  constexpr int DT = DP / 32;
  const fp8rl_attn_args& a = d.a;
  const int lane = (int)(threadIdx.x & 63);
  const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const int kv = (int)blockIdx.x % a.kv_heads, c = (int)blockIdx.y;
  constexpr int kFlight = 8;  // parts whose loads are under way at a time
  f32x4 x[kFlight][4];
  auto load = [&](int first) {
#pragma unroll
    for (int i = 0; i < kFlight; ++i) {
      if (first + i >= d.parts) break;
      const f32x4* const from = part_of<DP>(d, (int)blockIdx.x, first + i, wave, lane) + 64 * 4 * c;
#pragma unroll
      for (int e = 0; e < 4; ++e) x[i][e] = from[64 * e];
    }
  };
  load(0);
  const DocTile t = find_tile<kOwn, true>(d, (int)blockIdx.x / a.kv_heads, lane);
  const int key = t.first + 32 * wave;
  if (t.doc >= (int)a.docs || key >= t.lk) return;
  f32x16 g = zeros16();
  for (int first = 0; first < d.parts; first += kFlight) {
    if (first > 0) load(first);
#pragma unroll
    for (int i = 0; i < kFlight; ++i) {
      if (first + i >= d.parts) break;
#pragma unroll
      for (int e = 0; e < 16; ++e) g[e] += x[i][e >> 2][e & 3];
    }
  }
  const int64_t row = t.k0 + key + (lane & 31);
  uint16_t* const to = c < DT ? a.dk + row * a.ld_dk : a.dv + row * a.ld_dv;
  store_columns(g, c < DT ? a.sm_scale : 1.f, to + (int64_t)kv * a.head_dim, 32 * (c % DT), lane >> 5,
                a.head_dim, key + (lane & 31) < t.lk);
}

namespace {

// Parts that a key tile's queries are dealt out in: up to eight for two and a half workgroups to a
// CU, and more for two to a CU where eight tiles of queries a part remain. (What splitting costs is
// the parts' way through memory, 8 bytes a value of dk and dv and part, each way. The gradients of
// six documents of 4096 tokens in all, 32 query heads on 4 of 128: 202 us; with 512 workgroups for
// 640 217, with 768 209, with 1024 215. One document, 8 heads on 1, with sixteen and with eight
// parts: 4096 tokens 192 and 235 us, 2048 101 and 128; 8192, nine parts for eight, 603 and 580;
// 512, 32 on 8, two tiles a part, 62 and 49.)
int key_parts(int64_t Tq, int64_t Tk, int64_t docs, int q_heads, int kv_heads) {
  const int64_t tiles = max((int64_t)1, (Tk / kOwn + docs) * kv_heads);
  const int64_t through = Tq / kQueries * (q_heads / kv_heads) / max((int64_t)1, docs);
  const int64_t more = min((int64_t)kMostParts, min(through / 8, 528 / tiles));
  return (int)max(max((int64_t)1, more), min((int64_t)8, 640 / tiles));
}

int padded(int head_dim) { return head_dim <= 64 ? 64 : 128; }

}  // namespace

size_t attn_bwd_workspace(int64_t Tq, int64_t Tk, int64_t docs, int q_heads, int kv_heads,
                          int head_dim) {
  const int64_t parts = key_parts(Tq, Tk, docs, q_heads, kv_heads);
  const int64_t stats = (2 * Tq * q_heads + 3) / 4 * 4;
  const int64_t part = parts > 1 ? (Tk / kOwn + docs) * kv_heads * parts * kOwn * 2 : 0;
  return (size_t)(stats + part * padded(head_dim)) * sizeof(float);
}

hipError_t launch_attn_bwd(const fp8rl_attn_args& a, float* workspace, hipStream_t stream) {
  AttnArgs q = attn_args(a, kOwn, a.Tq), k = attn_args(a, kOwn, a.Tk);
  q.stats = k.stats = workspace;
  k.parts = key_parts(a.Tq, a.Tk, a.docs, a.q_heads, a.kv_heads);
  k.part = workspace + (2 * a.Tq * a.q_heads + 3) / 4 * 4;
  const dim3 block(64 * kWaves);
  const dim3 grid_q((unsigned)(q.slots * a.q_heads)), grid_k((unsigned)(k.slots * a.kv_heads * k.parts)),
      grid_j((unsigned)(k.slots * a.kv_heads), (unsigned)(2 * padded(a.head_dim) / 32));
  const bool few = q.slots * a.q_heads <= kFewQueries && a.Tk >= kLong * a.docs;
  auto go = [&](auto one, auto two, auto dkv) {
    if (few)
      hipLaunchKernelGGL(two, grid_q, dim3(512), 0, stream, q);
    else
      hipLaunchKernelGGL(one, grid_q, block, 0, stream, q);
    hipLaunchKernelGGL(dkv, grid_k, dim3(512), 0, stream, k);
  };
  auto choose = [&](auto width, auto pad) {
    constexpr int DP = decltype(width)::value;
    constexpr bool PAD = decltype(pad)::value;
    a.cap > 0.f || a.slopes
        ? go(attn_dq_kernel<DP, PAD, true, 1>, attn_dq_kernel<DP, PAD, true, 2>,
             attn_dkv_kernel<DP, PAD, true>)
        : go(attn_dq_kernel<DP, PAD, false, 1>, attn_dq_kernel<DP, PAD, false, 2>,
             attn_dkv_kernel<DP, PAD, false>);
  };
  constexpr std::integral_constant<int, 64> k64;
  constexpr std::integral_constant<int, 128> k128;
  if (a.head_dim == 64)
    choose(k64, std::false_type{});
  else if (a.head_dim < 64)
    choose(k64, std::true_type{});
  else if (a.head_dim < 128)
    choose(k128, std::true_type{});
  else
    choose(k128, std::false_type{});
  if (k.parts > 1) {
    if (padded(a.head_dim) == 64)
      hipLaunchKernelGGL(attn_dkv_join_kernel<64>, grid_j, block, 0, stream, k);
    else
      hipLaunchKernelGGL(attn_dkv_join_kernel<128>, grid_j, block, 0, stream, k);
  }
  return hipGetLastError();
}

}  // namespace fp8rl
