// Attention of packed documents.
//
// A workgroup has 128 queries of one head of a document, 32 a wave, and goes through the 64-key
// tiles that any of them sees; keys and values reach LDS two tiles deep by direct loads. Per tile,
// with the queries in the columns of the matrix instruction:
//   S^T = K Q^T,   m = max(m, max S),   P = exp(S - m),   l += sum P,   O^T += V^T P^T,
// so that a query's statistics are in the two lanes that hold its column, and P^T goes from one
// product into the other in its registers (attn_tile.hpp). V^T is read out of V's rows by the LDS's
// transposing read. m is raised, and O scaled, only where a maximum is more than 2^8 above it (P up
// to 2^8 loses nothing in float32 sums and bf16 operands).
//
// Bound by the matrix cores and by what stands between their instructions: two waves on a SIMD, one
// in its products while the other is in its exponentials. 8192 causal tokens, 32 query heads on 8
// of 128: 550 to 575 us a call from card to card (without a profiler), 1.0 PFLOP/s, 48 % of the
// cycles in matrix instructions, no LDS bank conflicts; a library product of 8192^3 reaches 1.29. Heads
// of 64: 0.83 PFLOP/s (half the products per exponential), of 256: 0.87 (eight waves, 17 of their
// registers spilled), of 144 to 240: 0.29 (how many steps of q there are is not known to the compiler,
// which leaves the loop over them as it is, and q in scratch memory: each step waits for its load).
// Four tiles in LDS instead of two, with eight waves, changed nothing: it is not the loads that a tile
// waits for.
#include "attn_tile.hpp"

namespace fp8rl {

namespace {

constexpr int kQ = 128, kK = 64;
constexpr float kRise = 8.f;
// Workgroups up to which two waves share 32 queries. Below two workgroups to a CU that halves the
// time of a tile (1024 tokens of 32/8 heads of 128: 27.4 us, else 29.5; 1536: 37.5, 42.8); above,
// it is the joining that counts (four documents of 2050 in all, 640 workgroups: 38.5 us, else 29.4;
// 4096 tokens: 179, else 160).
constexpr int kFew = 512;

}  // namespace

// DP: head_dim rounded up to 64, 128 or 256; PAD: it is less. MORE: capped scores or slopes. KH: waves
// that share 32 queries, each with its part of a tile's keys; their sums meet in the end.
template <int DP, bool PAD, bool MORE, int KH>
__global__ __launch_bounds__(256 * KH, 2) void attn_fwd_kernel(AttnArgs d) {
  constexpr int KS = DP / 16, DT = DP / 32;
  constexpr int kWaves = 4 * KH, NR = 2 / KH;  // a wave's 32-key parts of a tile
  constexpr int kTile = kK * DP * 2;           // bytes
  __shared__ __align__(1024) uint8_t s_mem[4 * kTile];  // k and v of two tiles; then O of some waves
  __shared__ float s_m[4][32], s_l[4][32];
  const fp8rl_attn_args& a = d.a;
  const int lane = (int)(threadIdx.x & 63), h = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const int block = wave & 3, part = wave >> 2;  // of the queries, of a tile's keys
  const int D = PAD ? a.head_dim : DP;

  // key heads fastest: with 8 of them, one to an XCD and its L2
  const int id = (int)blockIdx.x;
  const int kv = id % a.kv_heads;
  const int head = kv * d.group + id / a.kv_heads % d.group;
  const DocTile t = find_tile<kQ, false>(d, id / a.q_heads, lane);
  if (t.doc >= (int)a.docs) return;
  const Mask mask(a, t);
  const int shift = t.lk - t.lq;
  const int row = t.first + 32 * block + (lane & 31);
  const int p = row + shift;
  const int rows = min(32, t.lq - t.first - 32 * block);  // of this wave
  const int p0 = t.first + 32 * block + shift, p1 = p0 + rows - 1;

  bf16x8 q[KS];
  {
    const uint16_t* at = a.q + (t.q0 + min(row, t.lq - 1)) * a.ld_q + (int64_t)head * D;
#pragma unroll
    for (int s = 0; s < KS; ++s) q[s] = row_operand(at, s, h, D);
  }

  // tiles: those of the prefix, then those from the first query's window to the last one's end
  const int first = t.first + shift, last = min(t.first + kQ, t.lq) - 1 + shift;
  const int in_prefix = (mask.prefix + kK - 1) / kK;
  const int begin = max(mask.lo(first) / kK, in_prefix);
  const int tiles = in_prefix + max(0, (mask.hi(last) + kK - 1) / kK - begin);
  auto key_of = [&](int i) { return kK * (i < in_prefix ? i : i - in_prefix + begin); };

  const RowLoader<DP, kK, kWaves> rows_in(D, wave, lane);
  const uint16_t* const k0 = a.k + t.k0 * a.ld_k + (int64_t)kv * D;
  const uint16_t* const v0 = a.v + t.k0 * a.ld_v + (int64_t)kv * D;
  auto load = [&](int i) {
    const int j = key_of(i);
    rows_in.load(k0 + j * a.ld_k, a.ld_k, t.lk - j, s_mem + 2 * (i & 1) * kTile, wave);
    rows_in.load(v0 + j * a.ld_v, a.ld_v, t.lk - j, s_mem + (2 * (i & 1) + 1) * kTile, wave);
  };

  const bool capped = MORE && a.cap > 0.f, sloped = MORE && a.slopes;
  const float slope2 = sloped ? a.slopes[head] * kLog2e : 0.f;

  f32x16 o[DT];
#pragma unroll
  for (int i = 0; i < DT; ++i) o[i] = zeros16();
  float m = -__builtin_inff(), l = 0.f;

  if (tiles > 0) load(0);
  for (int i = 0; i < tiles; ++i) {
    landed();
    if (i + 1 < tiles) load(i + 1);
    uint8_t *const s_k = s_mem + 2 * (i & 1) * kTile, *const s_v = s_k + kTile;
    const int tile = key_of(i), in_tile = min(kK, t.lk - tile);
    if (in_tile < kK) {
      clear_rows<DP, kK, kWaves>(s_v, in_tile);
      __syncthreads();
    }
    // this wave's keys
    constexpr int kOwn = 32 * NR;
    const int j0 = tile + kOwn * part, keys = min(kOwn, t.lk - j0);
    if (rows <= 0 || keys <= 0 || !mask.any(p0, p1, j0, j0 + keys)) continue;

    const RowOperand<DP> kop(s_k + kOwn * part * DP * 2, lane);
    f32x16 s[NR];
#pragma unroll
    for (int r = 0; r < NR; ++r) s[r] = zeros16();
#pragma unroll
    for (int c = 0; c < KS; ++c) {
      if (PAD && 16 * c >= D) break;
#pragma unroll
      for (int r = 0; r < NR; ++r)
        s[r] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(kop(32 * r, c), q[c], s[r], 0, 0, 0);
    }
    float mul = d.scale2;  // a score in units of ln 2 is mul s
    if (capped) {
#pragma unroll
      for (int r = 0; r < NR; ++r) tanh_places<16>(s[r], d.scale2);
      mul = d.cap2;
    }
    if (sloped) {
#pragma unroll
      for (int r = 0; r < NR; ++r) {
        const float from = (float)(p - j0 - 32 * r - 4 * h);
        slope_scores(s[r], mul, slope2,
                     [&](int e) { return from - (float)(8 * (e >> 2) + (e & 3)); });
      }
      mul = 1.f;
    }
    if (keys < kOwn || !mask.all(p0, p1, j0, j0 + kOwn)) {
      const int lo = mask.lo(p), hi = mask.hi(p);
#pragma unroll
      for (int r = 0; r < NR; ++r)
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const int j = j0 + 32 * r + 8 * (e >> 2) + 4 * h + (e & 3);
          s[r][e] = (j < mask.prefix) | ((j >= lo) & (j < hi)) ? s[r][e] : -__builtin_inff();
        }
    }
    float top = s[0][0];
#pragma unroll
    for (int r = 0; r < NR; ++r)
#pragma unroll
      for (int e = 0; e < 16; ++e) top = fmaxf(top, s[r][e]);
    {
      const auto x = __builtin_amdgcn_permlane32_swap(__float_as_uint(top), __float_as_uint(top),
                                                      false, false);
      top = fmaxf(__uint_as_float(x[0]), __uint_as_float(x[1])) * mul;
    }
    if (__any(top > m + kRise)) {
      const float was = m;
      m = fmaxf(m, top);
      const float f = m == -__builtin_inff() ? 1.f : exp2_fast(was - m);
      l *= f;
#pragma unroll
      for (int c = 0; c < DT; ++c) o[c] *= f;
    }
    const float ref = m == -__builtin_inff() ? 0.f : m;
    float sum = 0.f;
#pragma unroll
    for (int r = 0; r < NR; ++r)
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        s[r][e] = exp2_fast(__builtin_fmaf(s[r][e], mul, -ref));
        sum += s[r][e];
      }
    l += sum;

    const ColOperand<DP> vop(s_v + kOwn * part * DP * 2, lane);
#pragma unroll
    for (int r = 0; r < 2 * NR; ++r) {
      // (one bf16 term of a weight, 2^-8 of itself at most, at any size: against 64 bits out is off
      // by 0.0019 to 0.0023 of its norm, with float32 weights by 0.0015 to 0.0017, the rounding of out
      // itself. A second term would double these products.)
      const bf16x8 w = operand_of(s[r >> 1], r & 1);
#pragma unroll
      for (int c = 0; c < DT; ++c) {
        if (PAD && 32 * c >= D) break;
        o[c] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(vop(16 * r, c), w, o[c], 0, 0, 0);
      }
    }
  }

  {
    const auto x = __builtin_amdgcn_permlane32_swap(__float_as_uint(l), __float_as_uint(l), false,
                                                    false);
    l = __uint_as_float(x[0]) + __uint_as_float(x[1]);
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
      if (h == 0) s_m[block][lane] = m, s_l[block][lane] = l;
    }
    __syncthreads();
    if (part == 1) return;
    const float m1 = s_m[block][lane & 31], l1 = s_l[block][lane & 31], both = fmaxf(m, m1);
    // (a wave that saw no key has zeros; one that saw a NaN is not left out)
    const float f0 = l == 0.f ? 0.f : exp2_fast(m - both), f1 = l1 == 0.f ? 0.f : exp2_fast(m1 - both);
    m = both;
    l = l * f0 + l1 * f1;
#pragma unroll
    for (int c = 0; c < 4 * DT; ++c) {
      const f32x4 x = other[64 * c];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int at = 4 * (c & 3) + e;
        o[c >> 2][at] = o[c >> 2][at] * f0 + x[e] * f1;
      }
    }
  }
  if (rows <= 0) return;
  const bool in = row < t.lq;
  const float f = l == 0.f ? 0.f : 1.f / l;
  uint16_t* const out = a.out + (t.q0 + row) * a.ld_out + (int64_t)head * D;
#pragma unroll
  for (int c = 0; c < DT; ++c) store_columns(o[c], f, out, 32 * c, h, D, in);
  if (a.lse && in && h == 0)
    a.lse[head * a.Tq + t.q0 + row] =
        l == 0.f ? -__builtin_inff() : (m + __builtin_amdgcn_logf(l)) * 0.6931471805599453f;
}

hipError_t launch_attn_fwd(const fp8rl_attn_args& a, hipStream_t stream) {
  const AttnArgs d = attn_args(a, kQ, a.Tq);
  const dim3 grid((unsigned)(d.slots * a.q_heads));
  const bool more = a.cap > 0.f || a.slopes;
  const bool few = d.slots * a.q_heads <= kFew;
  auto go = [&](auto one, auto two) {
    if (few)
      hipLaunchKernelGGL(two, grid, dim3(512), 0, stream, d);
    else
      hipLaunchKernelGGL(one, grid, dim3(256), 0, stream, d);
  };
  if (a.head_dim == 64)
    more ? go(attn_fwd_kernel<64, false, true, 1>, attn_fwd_kernel<64, false, true, 2>)
         : go(attn_fwd_kernel<64, false, false, 1>, attn_fwd_kernel<64, false, false, 2>);
  else if (a.head_dim < 64)
    more ? go(attn_fwd_kernel<64, true, true, 1>, attn_fwd_kernel<64, true, true, 2>)
         : go(attn_fwd_kernel<64, true, false, 1>, attn_fwd_kernel<64, true, false, 2>);
  else if (a.head_dim > 128) {
    // 32 queries of 256 columns and their sums take a wave's registers without a second
    // part of keys
    auto wide = [&](auto kernel) { hipLaunchKernelGGL(kernel, grid, dim3(512), 0, stream, d); };
    if (a.head_dim == 256)
      more ? wide(attn_fwd_kernel<256, false, true, 2>) : wide(attn_fwd_kernel<256, false, false, 2>);
    else
      more ? wide(attn_fwd_kernel<256, true, true, 2>) : wide(attn_fwd_kernel<256, true, false, 2>);
  } else if (a.head_dim < 128)
    more ? go(attn_fwd_kernel<128, true, true, 1>, attn_fwd_kernel<128, true, true, 2>)
         : go(attn_fwd_kernel<128, true, false, 1>, attn_fwd_kernel<128, true, false, 2>);
  else
    more ? go(attn_fwd_kernel<128, false, true, 1>, attn_fwd_kernel<128, false, true, 2>)
         : go(attn_fwd_kernel<128, false, false, 1>, attn_fwd_kernel<128, false, false, 2>);
  return hipGetLastError();
}

}  // namespace fp8rl
