// Attention of one query per sequence over a paged cache, split over the cache's length and joined.
//
// With the running maximum m of a head's scores, its sum l = sum exp(a - m) and o = sum exp(a - m) v,
// a tile of keys updates the three; parts of a sequence meet as
//   M = max m_i,  l = sum l_i 2^(m_i - M),  o = sum o_i 2^(m_i - M)      (scores in units of ln 2).
//
// A wave takes 32 keys at a time, for up to 16 query heads that share them:
//   S^T = K Q^T   matrix instruction 16x16x32, rows = keys, columns = heads, twice;
//   O^T += V^T P^T  the same, rows = columns of v, contracted over the 32 keys.
// Row r of the first (second) product is key 8 (r / 4) + r % 4 (+ 4), so that the four rows a lane
// gets of either are the eight keys 8g .. 8g + 7 of its lane group g: the weights go from one
// product into the next without leaving the lane, and a statistic belongs to a lane's column in
// both. Keys come straight from memory in the layout of the matrix instruction (16 bytes of a row a
// lane), values as 8 rows x VW columns a lane, transposed in registers by byte permutes: no
// LDS on either way. All of it takes a tenth of the time the bytes take.
//
// The cache's rows are found through the page table: lane i resolves key i of the next tile while
// the present one is worked on, and hands the 64-bit offset out through LDS.
#include "attn_ops.hpp"

namespace fp8rl {

namespace {

constexpr int kUnit = 128;    // keys of a workgroup's step: four waves of 32
constexpr int kLeast = 4;     // units that are not split further
constexpr int kGroups = 1024; // workgroups a large call is split into, a sequence's rest not counted

struct DecodeArgs {
  fp8rl_attn_decode_args a;
  float* part;  // [slot][heads of a tile][head_dim], behind them [slot][heads of a tile][m, l]
  PageOf page_of;
  int group;   // query heads of a key head
  int tiles;   // of 16 query heads of a key head
  int heads;   // kv_heads * tiles: workgroups that share a piece of a sequence
  int slots;   // workgroups
};

struct Keys {
  int first, last;  // seen: first <= key < last
  int unit, units;  // the units these lie in
};

__device__ __forceinline__ Keys keys_of(const DecodeArgs& d, int b) {
  Keys k{0, 0, 0, 0};
  if (b < d.a.B && d.a.num_pages > 0) k.last = max(0, min(d.a.lengths[b],
                                                          d.a.table_width * d.a.page_size));
  k.first = d.a.window ? max(0, k.last - d.a.window) : 0;
  k.unit = k.first / kUnit;
  k.units = (k.last + kUnit - 1) / kUnit - k.unit;
  return k;
}

// The piece of a sequence that workgroups x * heads .. take: sequences in order, each in as many
// pieces as its units fill at `per` units, at least one.
struct Piece {
  int b;       // B: none
  int piece, pieces;
  int before;  // pieces of the sequences before
  Keys keys;
};

__device__ __forceinline__ int units_of_a_piece(const DecodeArgs& d, int lane) {
  int64_t total = 0;
  for (int c = 0; c < (int)d.a.B; c += 64) total += keys_of(d, c + lane).units;
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) total += __shfl_xor(total, o, 64);
  const int64_t per = (total * d.heads + kGroups - 1) / kGroups;
  return __builtin_amdgcn_readfirstlane((int)max((int64_t)kLeast, per));
}

// Of piece x (by_piece) or of sequence x.
__device__ __forceinline__ Piece find_piece(const DecodeArgs& d, int x, bool by_piece, int lane) {
  const int per = units_of_a_piece(d, lane);
  int base = 0;
  for (int c = 0; c < (int)d.a.B; c += 64) {
    const Keys k = keys_of(d, c + lane);
    const int pieces = c + lane < d.a.B ? max(1, (k.units + per - 1) / per) : 0;
    int upto = pieces;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const int t = __shfl_up(upto, o, 64);
      if (lane >= o) upto += t;
    }
    const uint64_t past = __ballot(by_piece ? base + upto > x : c + lane == x);
    if (past) {
      const int at = __builtin_ctzll(past);
      Piece p;
      p.b = c + at;
      p.pieces = __builtin_amdgcn_readlane(pieces, at);
      p.before = base + __builtin_amdgcn_readlane(upto, at) - p.pieces;
      p.piece = x - p.before;
      p.keys.first = __builtin_amdgcn_readlane(k.first, at);
      p.keys.last = __builtin_amdgcn_readlane(k.last, at);
      p.keys.unit = __builtin_amdgcn_readlane(k.unit, at);
      p.keys.units = __builtin_amdgcn_readlane(k.units, at);
      return p;
    }
    base += __builtin_amdgcn_readlane(upto, 63);
  }
  return Piece{(int)d.a.B, 0, 0, 0, {0, 0, 0, 0}};
}

// N 32-bit words at p, which is aligned to 8 bytes (4 for one word).
template <int N>
__device__ __forceinline__ void load_words(uint32_t (&w)[N], const void* p) {
  typedef u32x4 __attribute__((aligned(8))) u32x4_8;
  if constexpr (N == 1) {
    w[0] = *static_cast<const uint32_t*>(p);
  } else if constexpr (N == 2) {
    const u32x2 t = *static_cast<const u32x2*>(p);
    w[0] = t.x, w[1] = t.y;
  } else {
#pragma unroll
    for (int i = 0; i < N / 4; ++i) {
      const u32x4 t = static_cast<const u32x4_8*>(p)[i];
      w[4 * i] = t.x, w[4 * i + 1] = t.y, w[4 * i + 2] = t.z, w[4 * i + 3] = t.w;
    }
  }
}

// The same 16-bit half of two words, the first's in the low half.
__device__ __forceinline__ uint32_t halves(uint32_t a, uint32_t b, bool high) {
  return __builtin_amdgcn_perm(b, a, high ? 0x07060302u : 0x05040100u);
}

}  // namespace

// DP: head_dim rounded up to 64, 128 or 256. CODES: an E4M3 cache.
template <int DP, bool CODES>
__global__ __launch_bounds__(256) void attn_decode_kernel(DecodeArgs d) {
  constexpr int VW = DP / 16;                   // columns of v a lane holds
  constexpr int VN = CODES ? DP / 64 : DP / 32; // words of them
  constexpr int KN = CODES ? DP / 64 : DP / 32; // 16-byte loads of a key's row
  constexpr int EL = CODES ? 1 : 2;             // bytes of an element
  constexpr int OS = DP + 4;
  __shared__ int64_t s_at[4][2][32];
  __shared__ float s_o[4][16][OS];
  __shared__ float s_m[4][16], s_l[4][16];
  const fp8rl_attn_decode_args& a = d.a;
  const int lane = (int)(threadIdx.x & 63);
  const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const int g = lane >> 4, col = lane & 15;
  const int D = a.head_dim;

  const int head = (int)blockIdx.x % d.heads;
  const Piece w = find_piece(d, (int)blockIdx.x / d.heads, true, lane);
  if (w.b >= (int)a.B) return;
  const int kv = head / d.tiles, tile = head % d.tiles;
  const int count = min(16, d.group - 16 * tile);  // query heads of this tile
  const int head0 = kv * d.group + 16 * tile;

  // the piece's units, spread evenly over the sequence's pieces
  const int u0 = w.keys.unit + (int)((int64_t)w.keys.units * w.piece / w.pieces);
  const int u1 = w.keys.unit + (int)((int64_t)w.keys.units * (w.piece + 1) / w.pieces);
  const int end = min(w.keys.last, u1 * kUnit);

  // q, a head a column, its columns of the head in the order in which the keys' come
  bf16x8 qf[DP / 32];
  {
    const int64_t row = (int64_t)w.b * a.ld_q + (int64_t)(head0 + col) * D;
#pragma unroll
    for (int i = 0; i < DP / 32; ++i) {
      const int at = CODES ? 64 * (i / 2) + 16 * g + 8 * (i & 1) : 32 * i + 8 * g;
      u32x4 t{0u, 0u, 0u, 0u};
      if (col < count && at < D) {
        if (a.q_scale) {
          uint32_t c[2];
          load_words(c, static_cast<const uint8_t*>(a.q) + row + at);
          const u32x2 lo = codes_bf16(c[0]), hi = codes_bf16(c[1]);
          t = u32x4{lo.x, lo.y, hi.x, hi.y};
        } else {
          t = *reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(a.q) + row + at);
        }
      }
      qf[i] = __builtin_bit_cast(bf16x8, t);
    }
  }
  const bool capped = a.cap > 0.f, sloped = a.slopes != nullptr;
  // a score in units of ln 2, or of the cap
  float unit = a.sm_scale * (a.q_scale ? *a.q_scale : 1.f) * (CODES ? *a.k_scale : 1.f);
  unit *= capped ? 1.f / a.cap : kLog2e;
  const float cap2 = a.cap * kLog2e;
  const float slope2 = sloped && col < count ? a.slopes[head0 + col] * kLog2e : 0.f;

  const char* const kbase = static_cast<const char*>(a.k_cache) + kv * a.head_stride * EL;
  const char* const vbase = static_cast<const char*>(a.v_cache) + kv * a.head_stride * EL;
  const int32_t* const table = a.page_table + (int64_t)w.b * a.ld_table;
  const int krow = 8 * (col >> 2) + (col & 3);  // the key of this lane's row, less 4 in the second
  // columns past head_dim are read from column 0 and cleared in K (q has zeros there, but 0 * NaN)
  int kcol[KN];
  uint32_t kkeep[KN];
#pragma unroll
  for (int i = 0; i < KN; ++i) {
    const int at = i * (CODES ? 64 : 32) + g * (CODES ? 16 : 8);
    kcol[i] = at < D ? at * EL : 0;
    kkeep[i] = at < D ? ~0u : 0u;
  }
  const bool ragged = D != DP;
  const int vcol = col * VW < D ? col * VW * EL : 0;

  // the key that this lane resolves of the tile at `base`: its page's number, then its row
  auto entry = [&](int base) {
    const int key = base + (lane & 31);
    return key >= w.keys.first && key < end ? table[d.page_of(key)] : -1;
  };
  uint64_t seen = 0, seen_next = 0;  // bit i: key i of the tile is seen
  auto resolve = [&](int base, int page, int slot) {
    const bool ok = page >= 0 && page < a.num_pages;
    const int key = base + (lane & 31);
    const int place = key - d.page_of(key) * a.page_size;
    const int64_t at = ok ? page * a.page_stride + place * a.slot_stride : 0;
    s_at[wave][slot][lane & 31] = at * EL;
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    return __ballot(ok) & 0xFFFFFFFFull;
  };

  uint32_t kf[2][KN][4], vf[8][VN];
  auto load_k = [&](int slot) {
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const char* row = kbase + s_at[wave][slot][krow + 4 * r];
#pragma unroll
      for (int i = 0; i < KN; ++i) load_words(kf[r][i], row + kcol[i]);
    }
  };

  f32x4 o[VW];
#pragma unroll
  for (int t = 0; t < VW; ++t) o[t] = f32x4{0.f, 0.f, 0.f, 0.f};
  float m = -__builtin_inff(), l = 0.f;

  int base = u0 * kUnit + 32 * wave;
  int slot = 0;
  if (base < end) {
    seen = resolve(base, entry(base), 0);
    load_k(0);
  }
  int next_page = entry(base + kUnit);
  for (; base < end; base += kUnit, slot ^= 1) {
#pragma unroll
    for (int e = 0; e < 8; ++e) load_words(vf[e], vbase + s_at[wave][slot][8 * g + e] + vcol);
    seen_next = resolve(base + kUnit, next_page, slot ^ 1);
    next_page = entry(base + 2 * kUnit);

    f32x4 s[2];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      f32x4 acc{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int i = 0; i < KN; ++i) {
        uint32_t* f = kf[r][i];
        if (ragged) {
#pragma unroll
          for (int j = 0; j < 4; ++j) f[j] &= kkeep[i];
        }
        if constexpr (CODES) {
          const u32x2 c0 = codes_bf16(f[0]), c1 = codes_bf16(f[1]), c2 = codes_bf16(f[2]),
                      c3 = codes_bf16(f[3]);
          acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
              __builtin_bit_cast(bf16x8, (u32x4{c0.x, c0.y, c1.x, c1.y})), qf[2 * i], acc, 0, 0, 0);
          acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
              __builtin_bit_cast(bf16x8, (u32x4{c2.x, c2.y, c3.x, c3.y})), qf[2 * i + 1], acc, 0, 0,
              0);
        } else {
          acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
              __builtin_bit_cast(bf16x8, (u32x4{f[0], f[1], f[2], f[3]})), qf[i], acc, 0, 0, 0);
        }
      }
      s[r] = acc;
    }
    if (base + kUnit < end) load_k(slot ^ 1);

    float x[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = s[e >> 2][e & 3] * unit;
    if (capped) {
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = cap2 * tanh_cap(x[e]);
    }
    if (sloped) {
      const float far = (float)(w.keys.last - 1 - base - 8 * g);
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] -= slope2 * (far - (float)e);
    }
    if (seen != 0xFFFFFFFFull) {
      const uint32_t mine = (uint32_t)(seen >> (8 * g));
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const bool in = (mine >> e) & 1;
        x[e] = in ? x[e] : -__builtin_inff();
#pragma unroll
        for (int i = 0; i < VN; ++i) vf[e][i] = in ? vf[e][i] : 0u;
      }
    }
    float top = fmaxf(fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])),
                      fmaxf(fmaxf(x[4], x[5]), fmaxf(x[6], x[7])));
    if (__any(top > m)) {
      const float was = m;
      m = fmaxf(m, max_rows(top));
      const float f = m == -__builtin_inff() ? 1.f : exp2_fast(was - m);
      l *= f;
#pragma unroll
      for (int t = 0; t < VW; ++t) o[t] *= f;
    }
    const float ref = m == -__builtin_inff() ? 0.f : m;
    float p[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) p[e] = exp2_fast(x[e] - ref);
    l += ((p[0] + p[1]) + (p[2] + p[3])) + ((p[4] + p[5]) + (p[6] + p[7]));

    if constexpr (CODES) {
      f16x8 pf;
#pragma unroll
      for (int e = 0; e < 8; ++e) pf[e] = (_Float16)p[e];
#pragma unroll
      for (int i = 0; i < VN; ++i) {  // four columns
        u32x2 c[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) c[e] = codes_f16(vf[e][i]);
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          const bool high = t & 1;
          const u32x4 f{halves(c[0][t >> 1], c[1][t >> 1], high),
                        halves(c[2][t >> 1], c[3][t >> 1], high),
                        halves(c[4][t >> 1], c[5][t >> 1], high),
                        halves(c[6][t >> 1], c[7][t >> 1], high)};
          o[4 * i + t] = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, f), pf,
                                                                o[4 * i + t], 0, 0, 0);
        }
      }
    } else {
      bf16x8 hi, lo;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        hi[e] = (__bf16)p[e];
        lo[e] = (__bf16)(p[e] - (float)hi[e]);
      }
#pragma unroll
      for (int t = 0; t < VW; ++t) {
        const bool high = t & 1;
        const u32x4 f{halves(vf[0][t >> 1], vf[1][t >> 1], high),
                      halves(vf[2][t >> 1], vf[3][t >> 1], high),
                      halves(vf[4][t >> 1], vf[5][t >> 1], high),
                      halves(vf[6][t >> 1], vf[7][t >> 1], high)};
        o[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, f), hi, o[t], 0, 0,
                                                       0);
        o[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, f), lo, o[t], 0, 0,
                                                       0);
      }
    }
    seen = seen_next;
  }

  // the four waves' parts meet
  l = sum_rows(l);
  if (g == 0) s_m[wave][col] = m, s_l[wave][col] = l;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
#pragma unroll
    for (int t = 0; t < VW; ++t) s_o[wave][col][(4 * g + i) * VW + t] = o[t][i];
  }
  __syncthreads();
  const int chunks = D / 8;
  for (int c = (int)threadIdx.x; c < count * chunks; c += 256) {
    const int h = c / chunks, at = 8 * (c - h * chunks);
    const float top = fmaxf(fmaxf(s_m[0][h], s_m[1][h]), fmaxf(s_m[2][h], s_m[3][h]));
    float sum = 0.f, r[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (s_l[i][h] == 0.f) continue;  // saw no key (a NaN is not left out)
      const float f = exp2_fast(s_m[i][h] - top);
      sum += s_l[i][h] * f;
#pragma unroll
      for (int k = 0; k < 8; ++k) r[k] += s_o[i][h][at + k] * f;
    }
    if (w.pieces == 1) {
      const float f = sum == 0.f ? 0.f : (CODES ? *a.v_scale : 1.f) / sum;
#pragma unroll
      for (int k = 0; k < 8; ++k) r[k] *= f;
      *reinterpret_cast<u32x4*>(a.out + (int64_t)w.b * a.ld_out + (int64_t)(head0 + h) * D + at) =
          round8(r);
    } else {
      const int most = min(16, d.group);
      const int64_t row = (int64_t)blockIdx.x * most + h;
      float* part = d.part + row * D + at;
      reinterpret_cast<f32x4*>(part)[0] = f32x4{r[0], r[1], r[2], r[3]};
      reinterpret_cast<f32x4*>(part)[1] = f32x4{r[4], r[5], r[6], r[7]};
      if (at == 0) {
        float* ml = d.part + (int64_t)d.slots * most * D + 2 * row;
        ml[0] = top, ml[1] = sum;
      }
    }
  }
}

// A wave per sequence and query head: the parts of those sequences that were split.
__global__ __launch_bounds__(256) void attn_decode_join_kernel(DecodeArgs d) {
  const fp8rl_attn_decode_args& a = d.a;
  const int lane = (int)(threadIdx.x & 63);
  const int x = __builtin_amdgcn_readfirstlane((int)(blockIdx.x * 4 + (threadIdx.x >> 6)));
  const int b = x / a.q_heads, hq = x - b * a.q_heads;
  if (b >= (int)a.B) return;
  const Piece w = find_piece(d, b, false, lane);
  if (w.pieces == 1) return;
  const int kv = hq / d.group, in = hq - kv * d.group;
  const int most = min(16, d.group);
  // row of the parts that the first piece of this head has, and from one piece to the next
  const int64_t row0 = ((int64_t)w.before * d.heads + kv * d.tiles + in / 16) * most + in % 16;
  const int64_t step = (int64_t)d.heads * most;
  const float* const ml = d.part + (int64_t)d.slots * most * a.head_dim;

  float top = -__builtin_inff();
  for (int c = lane; c < w.pieces; c += 64) top = fmaxf(top, ml[2 * (row0 + c * step)]);
#pragma unroll
  for (int s = 32; s > 0; s >>= 1) top = fmaxf(top, __shfl_xor(top, s, 64));

  const bool has = 4 * lane < a.head_dim;
  f32x4 o{0.f, 0.f, 0.f, 0.f};
  float sum = 0.f;
  for (int c = 0; c < w.pieces; c += 64) {
    float f = 0.f;
    if (c + lane < w.pieces) {
      const float* at = ml + 2 * (row0 + (c + lane) * step);
      f = at[1] == 0.f ? 0.f : exp2_fast(at[0] - top);
      sum += at[1] * f;
    }
    const int n = min(64, w.pieces - c);
    for (int i = 0; i < n; i += 8) {  // eight parts in flight
      f32x4 t[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        t[j] = f32x4{0.f, 0.f, 0.f, 0.f};
        if (has && i + j < n)
          t[j] = reinterpret_cast<const f32x4*>(d.part +
                                                (row0 + (c + i + j) * step) * a.head_dim)[lane];
      }
#pragma unroll
      for (int j = 0; j < 8; ++j)
        o += t[j] * __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(f), i + j));
    }
  }
  sum = wave_sum(sum);
  const float f = sum == 0.f ? 0.f : (a.v_scale ? *a.v_scale : 1.f) / sum;
  if (has) {
    u32x2* out = reinterpret_cast<u32x2*>(a.out + (int64_t)b * a.ld_out + (int64_t)hq * a.head_dim);
    out[lane] = u32x2{pack2_bf16(o[0] * f, o[1] * f), pack2_bf16(o[2] * f, o[3] * f)};
  }
}

namespace {

// Workgroups for sequences of up to max_keys keys: kGroups and what each sequence's last piece adds,
// or every piece that the smallest division gives, if that is less.
struct Grid {
  int64_t slots;
  bool split;  // some sequence may be
};
Grid decode_grid(int64_t B, int64_t heads, int64_t max_keys, int window) {
  int64_t units = (max_keys + kUnit - 1) / kUnit;
  if (window) units = min(units, ((int64_t)window + kUnit - 2) / kUnit + 1);
  const int64_t pieces = max((int64_t)1, (units + kLeast - 1) / kLeast);
  const int64_t items = B * heads;
  return {min(items * pieces, items + kGroups), pieces > 1};
}

template <bool CODES>
void run_decode(const DecodeArgs& d, hipStream_t stream) {
  const dim3 grid((unsigned)d.slots), block(256);
  if (d.a.head_dim <= 64)
    hipLaunchKernelGGL((attn_decode_kernel<64, CODES>), grid, block, 0, stream, d);
  else if (d.a.head_dim <= 128)
    hipLaunchKernelGGL((attn_decode_kernel<128, CODES>), grid, block, 0, stream, d);
  else
    hipLaunchKernelGGL((attn_decode_kernel<256, CODES>), grid, block, 0, stream, d);
}

int head_tiles(int q_heads, int kv_heads) { return (q_heads / kv_heads + 15) / 16; }

}  // namespace

size_t attn_decode_workspace(int64_t B, int q_heads, int kv_heads, int head_dim, int64_t max_keys,
                             int window) {
  const Grid g = decode_grid(B, (int64_t)kv_heads * head_tiles(q_heads, kv_heads), max_keys, window);
  if (!g.split) return 0;
  return (size_t)g.slots * (size_t)min(16, q_heads / kv_heads) * (size_t)(head_dim + 2) *
         sizeof(float);
}

hipError_t launch_attn_decode(const fp8rl_attn_decode_args& a, void* workspace, hipStream_t stream) {
  DecodeArgs d;
  d.a = a;
  d.part = static_cast<float*>(workspace);
  d.page_of = PageOf(a.page_size);
  d.group = a.q_heads / a.kv_heads;
  d.tiles = head_tiles(a.q_heads, a.kv_heads);
  d.heads = a.kv_heads * d.tiles;
  const Grid g = decode_grid(a.B, d.heads, (int64_t)a.table_width * a.page_size, a.window);
  d.slots = (int)g.slots;
  if (a.k_scale)
    run_decode<true>(d, stream);
  else
    run_decode<false>(d, stream);
  if (g.split)
    hipLaunchKernelGGL(attn_decode_join_kernel, dim3((unsigned)((a.B * a.q_heads + 3) / 4)),
                       dim3(256), 0, stream, d);
  return hipGetLastError();
}

}  // namespace fp8rl
