// New tokens' q, k and v: per-head norms, rotation by position, and the store of k and v into a
// paged cache, in one pass.
//
// Inside a head, the D / 8 chunks of 8 values are dealt out in pairs, so that both columns of every
// rotated pair (a, b) are in one lane:
//   w[a] = u[a] cos - u[b] sin,   w[b] = u[b] cos + u[a] sin.
// Lane p of a head holds, with C = rot / 16 rotated chunk pairs,
//   halves:       p < C: chunks p and p + C (columns i and i + rot / 2);
//   interleaved:  p < C: chunks 2p and 2p + 1 (columns 2i and 2i + 1 are in one chunk);
//   the rest:     p >= C: chunks 2p and 2p + 1, not rotated (the second may not exist).
// A head takes G lanes, the least power of two with 2 G chunks; sums over a head stay inside them.
//
// A wave takes U * 64 / G heads of one token: what belongs to the token (its position, slot, page
// and row addresses) is scalar, its cosines and sines are fetched once, and the heads' rows are in
// flight together. Two heads a lane group in large calls (36 us at 8192 tokens of 48 heads of 128
// with E4M3 outputs, 155 MB, one: 43 us, three: 36 us but 39 against 37 us with bf16 outputs), one
// where that leaves CUs idle. With bf16 outputs memory bounds it (206 MB in 37.4 us, 5.5 TB/s),
// with E4M3 ones the conversions take about as long as the bytes (16384 tokens: 63 us, 4.9 TB/s).
// Head norms, formed in float64, add to that: with a bf16 q and an E4M3 cache 38.2 against 33.0 us,
// all in E4M3 42.0 against 34.1 us, all in bf16 39.3 against 37.5 us.
#include "block_ops.hpp"

namespace fp8rl {

namespace {

struct RopeArgs {
  fp8rl_rope_kv_args a;
  unsigned waves;  // T * per_token
  unsigned per_token;
  int64_t slots;   // num_pages * page_size
  double inv_dim;  // 1 / head_dim
};

// A float64 on its way through float32 to a type of far fewer bits: cut off, and the last bit set
// where something was (rounding to odd), so that the second rounding sees what the first dropped.
// Less than 16 float64 units past a float32 value are taken for that value: an exact tie between
// two codes (a token at position 0, whose rotation is the identity, can have one) arrives here at
// most 5 units too far out, never short of it, since the reciprocal of the scale is raised (up()).
__device__ __forceinline__ float narrow(double d) {
  const uint64_t u = __builtin_bit_cast(uint64_t, d);
  const uint32_t lo = (uint32_t)u;
  const uint32_t rest = (lo & 0x1FFFFFFFu) + 0x1FFFFFF0u;  // bit 29: 16 units or more
  const uint64_t odd = (u & 0xFFFFFFFF00000000u) | ((lo | rest) & 0xE0000000u);
  return (float)__builtin_bit_cast(double, odd);
}
__device__ __forceinline__ float narrow(float f) { return f; }

// A correctly rounded reciprocal of S, raised by one or two units, so that it is not below 1 / S
// and a product with it not below the quotient. Quotients that go through float32 to the nearest
// keep their bits: x * up(1 / S) is within 2^-50.6 of x / S, whose distance from a float32
// midpoint is more than 2^-49 (div_by_scale).
__device__ __forceinline__ double up(double r) { return r * (1.0 + 0x1p-52); }

// (x, y) -> f (x cos - y sin, y cos + x sin), in the type of f.
template <typename F>
__device__ __forceinline__ void turn(float& x, float& y, float c, float s, F f) {
  const F u = (F)x, v = (F)y;
  x = narrow(__builtin_elementwise_fma(u, (F)c, -(v * (F)s)) * f);
  y = narrow(__builtin_elementwise_fma(v, (F)c, u * (F)s) * f);
}

// A lane's two chunks rotated where they are, and scaled by f. In float32 on the way to bf16. On the
// way to E4M3 in float64, whose products here are exact: a code is a step of up to 1/8 of the value,
// and float32's errors before it would put one value in a million on the wrong side of a step.
// Unrotated columns and v go through float32 to the nearest, as the plain store's do.
template <typename F>
__device__ __forceinline__ void finish(float (&ua)[8], float (&ub)[8], const float (&c)[8],
                                       const float (&s)[8], bool turned, bool halves, F f) {
  if (!turned) {
#pragma unroll
    for (int k = 0; k < 8; ++k) ua[k] = (float)((F)ua[k] * f), ub[k] = (float)((F)ub[k] * f);
  } else if (halves) {
#pragma unroll
    for (int k = 0; k < 8; ++k) turn(ua[k], ub[k], c[k], s[k], f);
  } else {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      turn(ua[2 * k], ua[2 * k + 1], c[k], s[k], f);
      turn(ub[2 * k], ub[2 * k + 1], c[4 + k], s[4 + k], f);
    }
  }
}

}  // namespace

template <int G, int U>
__global__ __launch_bounds__(256) void rope_kv_append_kernel(RopeArgs args) {
  __shared__ double recip[3];  // of the scales of q, k and v, raised
  const fp8rl_rope_kv_args& a = args.a;
  if (threadIdx.x < 3) {
    const float* sp = threadIdx.x == 0 ? a.q_scale : threadIdx.x == 1 ? a.k_scale : a.v_scale;
    if (sp) recip[threadIdx.x] = up(recip_f64(*sp));
  }
  const unsigned wave =
      (unsigned)__builtin_amdgcn_readfirstlane((int)(blockIdx.x * 4 + (threadIdx.x >> 6)));
  const int lane = (int)(threadIdx.x & 63);
  const int p = lane % G;
  const unsigned t = wave / args.per_token;
  const int h0 = (int)(wave - t * args.per_token) * (U * 64 / G) + lane / G;
  const bool in = wave < args.waves;
  const int heads = in ? a.q_heads + 2 * a.kv_heads : 0;

  const int chunks = a.head_dim >> 3, C = a.rot_dim >> 4;
  const bool halves = !a.interleaved && p < C;
  const int ca = halves ? p : 2 * p;
  const int cb = halves ? p + C : 2 * p + 1;
  const bool has_a = ca < chunks, has_b = cb < chunks;

  int64_t at = 0, slot = -1;
  if (in && a.rot_dim > 0) at = a.positions[t];
  if (in) slot = a.slot_mapping[t];
  u32x4 va[U], vb[U];
#pragma unroll
  for (int i = 0; i < U; ++i) {
    const int head = h0 + i * (64 / G);
    va[i] = vb[i] = u32x4{0u, 0u, 0u, 0u};
    if (head >= heads) continue;
    const uint16_t* src = head < a.q_heads ? a.q + (int64_t)t * a.ld_q
                          : head < a.q_heads + a.kv_heads ? a.k + (int64_t)t * a.ld_k
                                                          : a.v + (int64_t)t * a.ld_v;
    const int at_head = head < a.q_heads ? head
                        : head < a.q_heads + a.kv_heads ? head - a.q_heads
                                                        : head - a.q_heads - a.kv_heads;
    const u32x4* row = reinterpret_cast<const u32x4*>(src) + at_head * chunks;
    if (has_a) va[i] = __builtin_nontemporal_load(row + ca);
    if (has_b) vb[i] = __builtin_nontemporal_load(row + cb);
  }
  const bool known = a.rot_dim == 0 || (at >= 0 && at < a.max_pos);  // the token is not skipped

  float c[8], s[8];
  if (known && p < C) {
    const float* cs = a.cos_sin + at * a.rot_dim + 8 * p;
    const float* sn = cs + a.rot_dim / 2;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float4 x = reinterpret_cast<const float4*>(cs)[i];
      const float4 y = reinterpret_cast<const float4*>(sn)[i];
      c[4 * i] = x.x, c[4 * i + 1] = x.y, c[4 * i + 2] = x.z, c[4 * i + 3] = x.w;
      s[4 * i] = y.x, s[4 * i + 1] = y.y, s[4 * i + 2] = y.z, s[4 * i + 3] = y.w;
    }
  }
  __syncthreads();  // the reciprocals
  if (!known) return;
  const bool stored = slot >= 0 && slot < args.slots;
  int64_t cache_row = 0;
  if (stored) {
    const int64_t page = slot >> 32 ? slot / a.page_size
                                    : (int64_t)((uint32_t)slot / (uint32_t)a.page_size);
    cache_row = page * a.page_stride + (slot - page * a.page_size) * a.slot_stride;
  }

#pragma unroll
  for (int i = 0; i < U; ++i) {
    int head = h0 + i * (64 / G);
    if (head >= heads) continue;
    const int kind = head < a.q_heads ? 0 : head < a.q_heads + a.kv_heads ? 1 : 2;  // q, k, v
    if (kind > 0 && !stored) continue;
    head -= kind == 0 ? 0 : kind == 1 ? a.q_heads : a.q_heads + a.kv_heads;
    float ua[8], ub[8];
    widen8(va[i], ua);
    widen8(vb[i], ub);
    double r = 1.0;
    if (kind < 2 && a.q_weight) {
      const u32x4* w = reinterpret_cast<const u32x4*>(kind == 0 ? a.q_weight : a.k_weight);
      float wa[8], wb[8];
      widen8(has_a ? w[ca] : u32x4{0u, 0u, 0u, 0u}, wa);
      widen8(has_b ? w[cb] : u32x4{0u, 0u, 0u, 0u}, wb);
      // widened before they are squared: float32's squares end at |x| = 2^64, bf16 does not
      double ss = 0.0;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const double x = (double)ua[k], y = (double)ub[k];
        ss = __builtin_elementwise_fma(x, x, __builtin_elementwise_fma(y, y, ss));
      }
#pragma unroll
      for (int o = 1; o < G; o <<= 1) ss += __shfl_xor(ss, o, 64);
      r = rsqrt(ss * args.inv_dim + (double)a.eps);
      // a head with an infinity or a NaN has no norm: NaN throughout, not r = 0 and zeros
      if (!(ss < __builtin_inf())) r = __builtin_nan("");
      if (ss > 0x1p100) {  // so far out x w and its rotation could leave float32
#pragma unroll
        for (int k = 0; k < 8; ++k) ua[k] *= 0x1p-64f, ub[k] *= 0x1p-64f;
        r *= 0x1p64;
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) ua[k] *= wa[k], ub[k] *= wb[k];  // exact: 8 + 8 bits
    }
    void* out = kind == 0 ? a.q_out : kind == 1 ? a.k_cache : a.v_cache;
    const int64_t dst = kind == 0 ? (int64_t)t * a.ld_qo + head * a.head_dim
                                  : cache_row + head * a.head_stride;
    const bool turned = kind < 2 && p < C;
    if (kind == 0 ? a.q_scale : a.k_scale) {
      finish(ua, ub, c, s, turned, halves, r * recip[kind]);
      u32x2* o = reinterpret_cast<u32x2*>(static_cast<uint8_t*>(out) + dst);
      if (has_a) o[ca] = encode8(ua);
      if (has_b) o[cb] = encode8(ub);
    } else {
      finish(ua, ub, c, s, turned, halves, (float)r);
      u32x4* o = reinterpret_cast<u32x4*>(static_cast<uint16_t*>(out) + dst);
      if (has_a) o[ca] = round8(ua);
      if (has_b) o[cb] = round8(ub);
    }
  }
}

namespace {

constexpr int kHeads = 2;  // heads of a lane group in large calls

template <int G>
void run_rope(const RopeArgs& r, int u, hipStream_t stream) {
  const dim3 grid((r.waves + 3) / 4);
  if (u == 1)
    hipLaunchKernelGGL((rope_kv_append_kernel<G, 1>), grid, dim3(256), 0, stream, r);
  else
    hipLaunchKernelGGL((rope_kv_append_kernel<G, kHeads>), grid, dim3(256), 0, stream, r);
}

}  // namespace

hipError_t launch_rope_kv_append(const fp8rl_rope_kv_args& a, hipStream_t stream) {
  RopeArgs r;
  r.a = a;
  r.slots = a.num_pages * (int64_t)a.page_size;
  r.inv_dim = 1.0 / a.head_dim;
  const int heads = a.q_heads + 2 * a.kv_heads;
  const int chunks = a.head_dim / 8;
  int g = 1;
  while (2 * g < chunks) g <<= 1;
  const int u = a.T * heads * g >= 64 * 4096 ? kHeads : 1;
  const int per_wave = u * 64 / g;
  r.per_token = (unsigned)((heads + per_wave - 1) / per_wave);
  r.waves = (unsigned)(a.T * r.per_token);
  switch (g) {
    case 1: run_rope<1>(r, u, stream); break;
    case 2: run_rope<2>(r, u, stream); break;
    case 4: run_rope<4>(r, u, stream); break;
    case 8: run_rope<8>(r, u, stream); break;
    case 16: run_rope<16>(r, u, stream); break;
    case 32: run_rope<32>(r, u, stream); break;
  }
  return hipGetLastError();
}

}  // namespace fp8rl
