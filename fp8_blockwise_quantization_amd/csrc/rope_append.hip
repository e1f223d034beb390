// New tokens' q, k and v: per-head norms, rotation by position, and the store of k and v into a
// paged cache, in one pass.
//
// One head of one token is a unit. Its D / 8 chunks of 8 values are dealt out in pairs, so that both
// columns of every rotated pair (a, b) are in one lane:
//   w[a] = u[a] cos - u[b] sin,   w[b] = u[b] cos + u[a] sin.
// Lane p of a unit holds, with C = rot / 16 rotated chunk pairs,
//   halves:       p < C: chunks p and p + C (columns i and i + rot / 2);
//   interleaved:  p < C: chunks 2p and 2p + 1 (columns 2i and 2i + 1 are in one chunk);
//   the rest:     p >= C: chunks 2p and 2p + 1, not rotated (the second may not exist).
// A unit takes G lanes, the least power of two with 2 G chunks; sums over a head stay inside them.
#include "block_ops.hpp"

namespace fp8rl {

namespace {

struct RopeArgs {
  fp8rl_rope_kv_args a;
  unsigned units;        // T * heads
  int64_t slots;         // num_pages * page_size
};

// Stores 8 values as bf16 or as codes of value / scale.
__device__ __forceinline__ void put8(void* base, int64_t at, const float (&f)[8], const float* s,
                                     double r) {
  if (s)
    *reinterpret_cast<u32x2*>(static_cast<uint8_t*>(base) + at) = codes8(f, r);
  else
    *reinterpret_cast<u32x4*>(static_cast<uint16_t*>(base) + at) = round8(f);
}

}  // namespace

template <int G>
__global__ __launch_bounds__(256) void rope_kv_append_kernel(RopeArgs args) {
  const fp8rl_rope_kv_args& a = args.a;
  const unsigned unit = blockIdx.x * (256u / G) + threadIdx.x / G;
  const int p = threadIdx.x % G;
  if (unit >= args.units) return;  // a whole unit's lanes: the others' sums do not reach across
  const unsigned heads = (unsigned)(a.q_heads + 2 * a.kv_heads);
  const unsigned t = unit / heads;
  int head = (int)(unit - t * heads);
  const int kind = head < a.q_heads ? 0 : head < a.q_heads + a.kv_heads ? 1 : 2;  // q, k, v
  head -= kind == 0 ? 0 : kind == 1 ? a.q_heads : a.q_heads + a.kv_heads;

  const int chunks = a.head_dim >> 3, C = a.rot_dim >> 4;
  const bool turned = kind < 2 && p < C;
  const bool halves = !a.interleaved && p < C;
  const int ca = halves ? p : 2 * p;
  const int cb = halves ? p + C : 2 * p + 1;
  const bool has_a = ca < chunks, has_b = cb < chunks;

  const int64_t at = a.rot_dim > 0 ? a.positions[t] : 0;
  if (a.rot_dim > 0 && (at < 0 || at >= a.max_pos)) return;  // a whole unit's lanes
  int64_t dst = 0;
  if (kind > 0) {
    const int64_t slot = a.slot_mapping[t];
    if (slot < 0 || slot >= args.slots) return;
    int64_t page;
    if (slot >> 32)
      page = slot / a.page_size;
    else
      page = (uint32_t)slot / (uint32_t)a.page_size;
    dst = page * a.page_stride + (slot - page * a.page_size) * a.slot_stride + head * a.head_stride;
  } else {
    dst = (int64_t)t * a.ld_qo + head * a.head_dim;
  }

  const uint16_t* src = kind == 0 ? a.q + (int64_t)t * a.ld_q
                                  : kind == 1 ? a.k + (int64_t)t * a.ld_k : a.v + (int64_t)t * a.ld_v;
  src += head * a.head_dim;
  u32x4 va = u32x4{0u, 0u, 0u, 0u}, vb = va;
  if (has_a) va = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(src) + ca);
  if (has_b) vb = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(src) + cb);
  float ua[8], ub[8];
  widen8(va, ua);
  widen8(vb, ub);

  const uint16_t* weight = kind == 0 ? a.q_weight : kind == 1 ? a.k_weight : nullptr;
  if (weight) {
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i)
      ss = __builtin_fmaf(ub[i], ub[i], __builtin_fmaf(ua[i], ua[i], ss));
#pragma unroll
    for (int o = 1; o < G; o <<= 1) ss += __shfl_xor(ss, o, 64);
    const float r = rsqrtf(ss / (float)a.head_dim + a.eps);
    float wa[8], wb[8];
    const u32x4* w = reinterpret_cast<const u32x4*>(weight);
    widen8(has_a ? w[ca] : u32x4{0u, 0u, 0u, 0u}, wa);
    widen8(has_b ? w[cb] : u32x4{0u, 0u, 0u, 0u}, wb);
#pragma unroll
    for (int i = 0; i < 8; ++i) ua[i] = ua[i] * wa[i] * r, ub[i] = ub[i] * wb[i] * r;
  }

  if (turned) {
    const float* cs = a.cos_sin + at * a.rot_dim + 8 * p;
    const float* sn = cs + a.rot_dim / 2;
    float c[8], s[8];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float4 x = reinterpret_cast<const float4*>(cs)[i];
      const float4 y = reinterpret_cast<const float4*>(sn)[i];
      c[4 * i] = x.x, c[4 * i + 1] = x.y, c[4 * i + 2] = x.z, c[4 * i + 3] = x.w;
      s[4 * i] = y.x, s[4 * i + 1] = y.y, s[4 * i + 2] = y.z, s[4 * i + 3] = y.w;
    }
    if (halves) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float x = ua[i], y = ub[i];
        ua[i] = __builtin_fmaf(x, c[i], -(y * s[i]));
        ub[i] = __builtin_fmaf(y, c[i], x * s[i]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float x = ua[2 * i], y = ua[2 * i + 1];
        ua[2 * i] = __builtin_fmaf(x, c[i], -(y * s[i]));
        ua[2 * i + 1] = __builtin_fmaf(y, c[i], x * s[i]);
        const float z = ub[2 * i], w = ub[2 * i + 1];
        ub[2 * i] = __builtin_fmaf(z, c[4 + i], -(w * s[4 + i]));
        ub[2 * i + 1] = __builtin_fmaf(w, c[4 + i], z * s[4 + i]);
      }
    }
  }

  void* out = kind == 0 ? a.q_out : kind == 1 ? a.k_cache : a.v_cache;
  const float* scale = kind == 0 ? a.q_scale : kind == 1 ? a.k_scale : a.v_scale;
  const double r = scale ? recip_f64(*scale) : 0.0;
  if (has_a) put8(out, dst + 8 * ca, ua, scale, r);
  if (has_b) put8(out, dst + 8 * cb, ub, scale, r);
}

hipError_t launch_rope_kv_append(const fp8rl_rope_kv_args& a, hipStream_t stream) {
  RopeArgs r;
  r.a = a;
  r.units = (unsigned)(a.T * (a.q_heads + 2 * a.kv_heads));
  r.slots = a.num_pages * (int64_t)a.page_size;
  const int chunks = a.head_dim / 8;
  int g = 1;
  while (2 * g < chunks) g <<= 1;
  const dim3 grid((unsigned)((r.units + 256 / g - 1) / (256 / g)));
#define FP8RL_ROPE(G) \
  case G: hipLaunchKernelGGL(rope_kv_append_kernel<G>, grid, dim3(256), 0, stream, r); break;
  switch (g) {
    FP8RL_ROPE(1)
    FP8RL_ROPE(2)
    FP8RL_ROPE(4)
    FP8RL_ROPE(8)
    FP8RL_ROPE(16)
    FP8RL_ROPE(32)
  }
#undef FP8RL_ROPE
  return hipGetLastError();
}

}  // namespace fp8rl
