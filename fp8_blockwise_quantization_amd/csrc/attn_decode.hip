// Attention of one query per sequence over a paged cache, split over the cache's length and joined.
//
// With the running maximum m of a head's scores, its sum l = sum exp(a - m) and o = sum exp(a - m)
// v, a tile of keys updates the three; parts of a sequence meet as
//   M = max m_i,  l = sum l_i 2^(m_i - M),  o = sum o_i 2^(m_i - M)      (scores in units of ln 2).
//
// A wave, one of eight, takes 32 keys at a time, for up to 16 query heads that share them:
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
//
// Bound by memory; every key and value is read once. Values go past the caches (nontemporal loads:
// 64 uneven sequences of up to 4096 keys of 8 heads of 128 in E4M3, 58.1 us without, 53.8 with; an
// instruction takes their lines whole), keys do not (their rows are read 64 bytes at a time, and the
// other half of a line was gone by the next step: 35 us instead of 32 for a window of 1024 keys of
// 256). Those 64 sequences are 246 MB: 48 us for this kernel, 5.1 TB/s, and 6 for the join; 529 MB,
// eight uneven sequences of up to 32768 keys of 4 heads of 128 in bf16: 88 us, 6.0 TB/s, and 6. What
// lies beside the bytes is the launch and the chain of lengths, table and first keys, about 4 us. bf16
// heads of 144 to 256 columns spill 23 to 48 registers. Two tiles of keys under way in
// a wave (59.9 against 57.4 us: 16 waves' registers become 8's) and sixteen waves a CU with half a
// piece each (69) were slower.
#include "attn_ops.hpp"

namespace fp8rl {

namespace {

constexpr int kWaves = 8;   // of a workgroup, and what a CU runs at once
constexpr int kUnit = 32;   // keys of a wave's step
// Keys, and their bytes in a head, up to which a sequence is not split: one limit for heads of all
// widths, below the crossing of narrow ones and above that of wide ones. Uneven sequences of 32 query
// heads on 8 of 128 in E4M3, up to 1020 keys each, not split and split: one 9.7 and 12.1 us, 64 of
// them 21.1 and 26.2; up to 1500 12.7 and 12.5, 28.8 and 30.5; up to 2040 17.1 and 12.7, both 37. 1024
// keys each of 8 heads of 256, one sequence and 100: in E4M3 15.6 and 15.3, 88.9 and 82.8; in bf16
// (twice these bytes, and so split) 33.2 and 26.4, 212 and 165.
constexpr int kWhole = 1024;
constexpr int kWholeBytes = 256 << 10;
constexpr int kLeast = 2;   // units of a piece

// Who does what.
//   Where all sequences are short (kWhole), a workgroup takes a sequence and head tile, its waves
//   the sequence's units in turn; their parts meet in LDS, and that is all.
//   Else a wave takes a head tile and a piece of all sequences' units in a row. As many waves as
//   run at once all take the same number of units, however the lengths differ; a wave may so end
//   one sequence, take others whole and begin a last one. What it has of a sequence that was cut
//   goes to memory, and a second kernel joins it, told by the wave that began it where it lies
//   (counted anew for each head, 4096 sequences of 160 keys took 286 us instead of 145). The waves
//   of a workgroup have neighbouring heads of the same keys, which a cache laid out by tokens has
//   side by side.
struct DecodeArgs {
  fp8rl_attn_decode_args a;
  float* part;  // [wave][ended, begun][heads of a tile][head_dim], behind them their [m, l]
  int* cut;     // behind those [B]: units in front of a sequence, -1 if it is whole; [1]: of a lot
  PageOf page_of;
  int group;   // query heads of a key head
  int tiles;   // of 16 query heads of a key head
  int heads;   // kv_heads * tiles
  int lots;    // pieces that all units are cut into; 0: a sequence each
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

// A sequence's place among all sequences' units, and what a wave takes of these.
struct Place {
  int b, before;  // sequence and the units in front of it
  int per;
};

// Of the sequence that holds unit per * lot (b = B: none does).
__device__ __forceinline__ Place find_place(const DecodeArgs& d, int lot, int lane) {
  const int B = (int)d.a.B;
  const int front = sum_upto(keys_of(d, lane).units);  // most calls' only sequences
  int total = __builtin_amdgcn_readlane(front, 63);
  for (int c = 64; c < B; c += 64)
    total += __builtin_amdgcn_readlane(sum_upto(keys_of(d, c + lane).units), 63);
  const int per = max(kLeast, (int)((uint32_t)(total + d.lots - 1) / (uint32_t)d.lots));
  int base = 0;
  for (int c = 0; c < B; c += 64) {
    const int upto = base + (c == 0 ? front : sum_upto(keys_of(d, c + lane).units));
    const uint64_t here = __ballot(c + lane < B && upto > lot * per);
    if (here) {
      const int at = __builtin_ctzll(here);
      return {c + at, at ? __builtin_amdgcn_readlane(upto, at - 1) : base, per};
    }
    base = __builtin_amdgcn_readlane(upto, 63);
  }
  return {B, base, per};
}

// N 32-bit words at p, which is aligned to 8 bytes (4 for one word). ONCE: not kept in the caches.
template <bool ONCE, int N>
__device__ __forceinline__ void load_words(uint32_t (&w)[N], const void* p) {
  typedef u32x4 __attribute__((aligned(8))) u32x4_8;
  auto get = [](auto* at) { return ONCE ? __builtin_nontemporal_load(at) : *at; };
  if constexpr (N == 1) {
    w[0] = get(static_cast<const uint32_t*>(p));
  } else if constexpr (N == 2) {
    const u32x2 t = get(static_cast<const u32x2*>(p));
    w[0] = t.x, w[1] = t.y;
  } else {
#pragma unroll
    for (int i = 0; i < N / 4; ++i) {
      const u32x4 t = get(static_cast<const u32x4_8*>(p) + i);
      w[4 * i] = t.x, w[4 * i + 1] = t.y, w[4 * i + 2] = t.z, w[4 * i + 3] = t.w;
    }
  }
}

// The same 16-bit half of two words, the first's in the low half.
__device__ __forceinline__ uint32_t halves(uint32_t a, uint32_t b, bool high) {
  return __builtin_amdgcn_perm(b, a, high ? 0x07060302u : 0x05040100u);
}

}  // namespace

// DP: head_dim rounded up to 64, 128 or 256; PAD: it is less. CODES: an E4M3 cache. SPLIT: pieces
// to waves.
template <int DP, bool PAD, bool CODES, bool SPLIT>
__global__ __launch_bounds__(64 * kWaves, 2) void attn_decode_kernel(DecodeArgs d) {
  constexpr int VW = DP / 16;                   // columns of v a lane holds
  constexpr int VN = CODES ? DP / 64 : DP / 32; // words of them
  constexpr int KN = CODES ? DP / 64 : DP / 32; // 16-byte loads of a key's row
  constexpr int EL = CODES ? 1 : 2;             // bytes of an element
  constexpr int OS = DP + 4;
  constexpr int kStep = SPLIT ? kUnit : kUnit * kWaves;
  __shared__ int64_t s_at[kWaves][2][32];
  __shared__ float s_o[kWaves][16][OS];  // (of no use, and so not there, with SPLIT)
  __shared__ float s_m[kWaves][16], s_l[kWaves][16];
  const fp8rl_attn_decode_args& a = d.a;
  const int lane = (int)(threadIdx.x & 63);
  const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const int g = lane >> 4, col = lane & 15;
  const int D = PAD ? a.head_dim : DP;

  const int id = SPLIT ? (int)blockIdx.x * kWaves + wave : (int)blockIdx.x;
  const int lot = id / d.heads, head = id - lot * d.heads;
  if (SPLIT && lot >= d.lots) return;
  const int kv = head / d.tiles, tile = head - kv * d.tiles;
  const int count = min(16, d.group - 16 * tile);  // query heads of this tile
  const int head0 = kv * d.group + 16 * tile;
  const bool capped = a.cap > 0.f, sloped = a.slopes != nullptr;
  // a score in units of ln 2, or of the cap
  float unit = a.sm_scale * (a.q_scale ? *a.q_scale : 1.f) * (CODES ? *a.k_scale : 1.f);
  unit *= capped ? 1.f / a.cap : kLog2e;
  const float v_scale = CODES ? *a.v_scale : 1.f;
  const float cap2 = a.cap * kLog2e;
  const float slope2 = sloped && col < count ? a.slopes[head0 + col] * kLog2e : 0.f;

  const char* const kbase = static_cast<const char*>(a.k_cache) + kv * a.head_stride * EL;
  const char* const vbase = static_cast<const char*>(a.v_cache) + kv * a.head_stride * EL;
  const int krow = 8 * (col >> 2) + (col & 3);  // the key of this lane's row, less 4 in the second
  // columns past head_dim are read from column 0 and cleared in K (q has zeros there, but 0 * NaN)
  auto column = [&](int i) { return i * (CODES ? 64 : 32) + g * (CODES ? 16 : 8); };
  const int vcol = !PAD || col * VW < D ? col * VW * EL : 0;

  // the piece of a sequence at hand: keys in steps from `base` on to `end`
  int b, taken, stop, before;  // units behind this piece and the wave's last, before sequence b
  bool whole, begun;           // the piece is the whole sequence, its beginning
  Keys keys;
  int base, end;
  const int32_t* table;
  bf16x8 qf[DP / 32];  // q, a head a column, its columns of the head in the order of the keys'

  // the key that this lane resolves of the tile at `base`: its page's number, then its row
  auto entry = [&](int base) {
    const int key = base + (lane & 31);
    return key >= keys.first && key < end ? table[d.page_of(key)] : -1;
  };
  uint64_t seen;  // bit i: key i of the tile is seen
  int next_page;
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
      for (int i = 0; i < KN; ++i)
        load_words<false>(kf[r][i], row + (!PAD || column(i) < D ? column(i) * EL : 0));
    }
  };

  auto next = [&]() {  // the next piece: false if there is none
    if (!SPLIT) {
      keys = keys_of(d, b);
      end = keys.last, base = (keys.unit + wave) * kUnit;
    } else {
      for (;; ++b) {
        if (b >= (int)a.B || taken >= stop) return false;
        keys = keys_of(d, b);
        const int from = taken - before, to = min(keys.units, from + stop - taken);
        before += keys.units;
        if (to == 0) continue;  // (a sequence without keys is left to the join)
        begun = from == 0, whole = begun && to == keys.units;
        if (begun && head == 0 && lane == 0) d.cut[b] = whole ? -1 : taken;
        taken += to - from;
        end = min(keys.last, (keys.unit + to) * kUnit);
        base = (keys.unit + from) * kUnit;
        break;
      }
    }
    table = a.page_table + (int64_t)b * a.ld_table;
    return true;
  };
  auto start = [&]() {  // its first loads
    const int64_t row = (int64_t)b * a.ld_q + (int64_t)(head0 + col) * D;
#pragma unroll
    for (int i = 0; i < DP / 32; ++i) {
      const int at = CODES ? 64 * (i / 2) + 16 * g + 8 * (i & 1) : 32 * i + 8 * g;
      u32x4 t{0u, 0u, 0u, 0u};
      if (col < count && at < D) {
        if (a.q_scale) {
          uint32_t c[2];
          load_words<false>(c, static_cast<const uint8_t*>(a.q) + row + at);
          const u32x2 lo = codes_bf16(c[0]), hi = codes_bf16(c[1]);
          t = u32x4{lo.x, lo.y, hi.x, hi.y};
        } else {
          t = *reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(a.q) + row + at);
        }
      }
      qf[i] = __builtin_bit_cast(bf16x8, t);
    }
    seen = 0;
    if (base < end) {
      seen = resolve(base, entry(base), 0);
      load_k(0);
    }
    next_page = entry(base + kStep);
  };

  b = lot;
  if (SPLIT) {
    const Place p = find_place(d, lot, lane);
    b = p.b, before = p.before, taken = lot * p.per, stop = taken + p.per;
    if (id == 0 && lane == 0) d.cut[a.B] = p.per;
  }
  bool more = next();
  if (more) start();
  while (more) {
    f32x4 o[VW];
#pragma unroll
    for (int t = 0; t < VW; ++t) o[t] = f32x4{0.f, 0.f, 0.f, 0.f};
    float m = -__builtin_inff(), l = 0.f;
    for (int slot = 0; base < end; base += kStep, slot ^= 1) {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        load_words<true>(vf[e], vbase + s_at[wave][slot][8 * g + e] + vcol);
      const uint64_t seen_next = resolve(base + kStep, next_page, slot ^ 1);
      next_page = entry(base + 2 * kStep);

      if (PAD) {
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
          for (int i = 0; i < KN; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) kf[r][i][j] = column(i) < D ? kf[r][i][j] : 0u;
      }
      f32x4 s[2];
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        f32x4 acc{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int i = 0; i < KN; ++i) {
          const uint32_t* f = kf[r][i];
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
      if (base + kStep < end) load_k(slot ^ 1);

      float x[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = s[e >> 2][e & 3];
      if (capped) {
        tanh_places<8>(x, unit);
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] *= cap2;
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] *= unit;
      }
      if (sloped) {
        const float far = (float)(keys.last - 1 - base - 8 * g);
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

      // The weights in two terms, 16 bits at any size: E4M3 values are exact in bf16 as well. (Rounded
      // to fp16, half the products for E4M3, 6.4 for 6.8 us at one sequence of 477 keys and 53.4 for
      // 53.7 at 64 of up to 4096, weights below 2^-14 of the largest lose bits and those below 2^-25
      // vanish: wrong where the largest weight's value is small.)
      bf16x8 hi, lo;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        hi[e] = (__bf16)p[e];
        lo[e] = (__bf16)(p[e] - (float)hi[e]);
      }
      auto add = [&](f32x4& sum, const uint32_t (&w)[8], bool high) {  // a column of each key
        const bf16x8 f = __builtin_bit_cast(
            bf16x8, (u32x4{halves(w[0], w[1], high), halves(w[2], w[3], high),
                           halves(w[4], w[5], high), halves(w[6], w[7], high)}));
        sum = __builtin_amdgcn_mfma_f32_16x16x32_bf16(f, hi, sum, 0, 0, 0);
        sum = __builtin_amdgcn_mfma_f32_16x16x32_bf16(f, lo, sum, 0, 0, 0);
      };
#pragma unroll
      for (int i = 0; i < VN; ++i) {
        constexpr int VC = VW / VN;  // columns of a word
        uint32_t w[VC / 2][8];       // pairs of columns
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          if constexpr (CODES) {
            const u32x2 c = codes_bf16(vf[e][i]);
            w[0][e] = c.x, w[1][e] = c.y;
          } else {
            w[0][e] = vf[e][i];
          }
        }
#pragma unroll
        for (int t = 0; t < VC; ++t) add(o[VC * i + t], w[t >> 1], t & 1);
      }
      seen = seen_next;
    }
    l = sum_rows(l);
    const int most = min(16, d.group);
    if (SPLIT) {
      const int done = b;
      const bool direct = whole;
      const int64_t row = (2 * (int64_t)id + begun) * most + col;
      ++b;
      more = next();
      if (more) start();  // its first loads are under way while this piece is written
      if (col < count) {
        const float f = l == 0.f ? 0.f : v_scale / l;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int at = (4 * g + i) * VW;
          if (at >= D) continue;
          if (direct) {
            uint16_t* const out = a.out + (int64_t)done * a.ld_out + (int64_t)(head0 + col) * D + at;
#pragma unroll
            for (int t = 0; t < VW; t += 4)
              *reinterpret_cast<u32x2*>(out + t) = u32x2{pack2_bf16(o[t][i] * f, o[t + 1][i] * f),
                                                         pack2_bf16(o[t + 2][i] * f, o[t + 3][i] * f)};
          } else {
#pragma unroll
            for (int t = 0; t < VW; t += 4)
              *reinterpret_cast<f32x4*>(d.part + row * D + at + t) =
                  f32x4{o[t][i], o[t + 1][i], o[t + 2][i], o[t + 3][i]};
          }
        }
        if (!direct && g == 0)
          *reinterpret_cast<float2*>(d.part + 2 * (int64_t)d.lots * d.heads * most * D + 2 * row) =
              float2{m, l};
      }
      continue;
    }
    if (g == 0) s_m[wave][col] = m, s_l[wave][col] = l;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
#pragma unroll
      for (int t = 0; t < VW; ++t) s_o[wave][col][(4 * g + i) * VW + t] = o[t][i];
    }
    __syncthreads();
    const int pairs = D / 2;
    for (int c = (int)threadIdx.x; c < count * pairs; c += 64 * kWaves) {
      const int h = (int)((uint32_t)c / (uint32_t)pairs), at = 2 * (c - h * pairs);
      float top = s_m[0][h];
#pragma unroll
      for (int i = 1; i < kWaves; ++i) top = fmaxf(top, s_m[i][h]);
      float sum = 0.f, x = 0.f, y = 0.f;
#pragma unroll
      for (int i = 0; i < kWaves; ++i) {
        // (a wave that saw no key has zeros; one that saw a NaN is not left out)
        const float li = s_l[i][h], f = li == 0.f ? 0.f : exp2_fast(s_m[i][h] - top);
        const float2 v = *reinterpret_cast<const float2*>(&s_o[i][h][at]);
        sum += li * f;
        x += v.x * f;
        y += v.y * f;
      }
      const float f = sum == 0.f ? 0.f : v_scale / sum;
      *reinterpret_cast<uint32_t*>(a.out + (int64_t)b * a.ld_out + (int64_t)(head0 + h) * D + at) =
          pack2_bf16(x * f, y * f);
    }
    more = false;
  }
}

// The parts of a sequence that was cut, for one query head. W waves share the parts, and then their
// sums.
template <int W>
__global__ __launch_bounds__(W > 1 ? 64 * W : 256) void attn_decode_join_kernel(DecodeArgs d) {
  constexpr int kItems = W > 1 ? 1 : 4;  // of a workgroup
  __shared__ float s_sum[W];
  __shared__ f32x4 s_o[W][64];
  const fp8rl_attn_decode_args& a = d.a;
  const int lane = (int)(threadIdx.x & 63);
  const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const int x = (int)blockIdx.x * kItems + wave / W, part = wave % W;
  const int b = x / a.q_heads, hq = x - b * a.q_heads;
  if (b >= (int)a.B) return;
  const Keys keys = keys_of(d, b);
  const bool has = 4 * lane < a.head_dim;
  u32x2* const out =
      reinterpret_cast<u32x2*>(a.out + (int64_t)b * a.ld_out + (int64_t)hq * a.head_dim);
  if (keys.units == 0) {
    if (has && part == 0) out[lane] = u32x2{0u, 0u};
    return;
  }
  const int before = d.cut[b], per = d.cut[a.B];
  if (before < 0) return;
  const int lot = before / per, pieces = (before + keys.units - 1) / per - lot + 1;
  const int kv = hq / d.group, in = hq - kv * d.group;
  const int most = min(16, d.group);
  // the row that piece i left: the first began the sequence, the others end it or go on
  auto row_of = [&](int i) {
    return (2 * ((int64_t)(lot + i) * d.heads + kv * d.tiles + in / 16) + (i == 0)) * most + in % 16;
  };
  const float* const ml = d.part + 2 * (int64_t)d.lots * d.heads * most * a.head_dim;

  float top = -__builtin_inff();
  for (int c = lane; c < pieces; c += 64) top = fmaxf(top, ml[2 * row_of(c)]);
#pragma unroll
  for (int s = 32; s > 0; s >>= 1) top = fmaxf(top, __shfl_xor(top, s, 64));

  f32x4 o{0.f, 0.f, 0.f, 0.f};
  float sum = 0.f;
  for (int c = 16 * part; c < pieces; c += 16 * W) {  // sixteen in flight
    f32x4 t[16];
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      t[j] = f32x4{0.f, 0.f, 0.f, 0.f};
      if (has && c + j < pieces)
        t[j] = reinterpret_cast<const f32x4*>(d.part + row_of(c + j) * a.head_dim)[lane];
    }
    float f = 0.f;
    if (lane < 16 && c + lane < pieces) {
      const float* at = ml + 2 * row_of(c + lane);
      f = at[1] == 0.f ? 0.f : exp2_fast(at[0] - top);
      sum += at[1] * f;
    }
#pragma unroll
    for (int j = 0; j < 16; ++j)
      o += t[j] * __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(f), j));
  }
  sum = wave_sum(sum);
  if (W > 1) {
    if (lane == 0) s_sum[wave] = sum;
    s_o[wave][lane] = o;
    __syncthreads();
    if (part > 0) return;
#pragma unroll
    for (int i = 1; i < W; ++i) sum += s_sum[i], o += s_o[i][lane];
  }
  const float f = sum == 0.f ? 0.f : (a.v_scale ? *a.v_scale : 1.f) / sum;
  if (has) out[lane] = u32x2{pack2_bf16(o[0] * f, o[1] * f), pack2_bf16(o[2] * f, o[3] * f)};
}

namespace {

// Pieces of all sequences' units, 0 where a workgroup takes a sequence.
int decode_lots(int64_t heads, int64_t max_keys, int window, int row_bytes) {
  if (window) max_keys = min(max_keys, (int64_t)window);
  if (max_keys <= min(kWhole, kWholeBytes / row_bytes)) return 0;
  return (int)max((int64_t)1, 256 * kWaves / heads);
}

template <bool CODES, bool SPLIT>
void run_decode(const DecodeArgs& d, hipStream_t stream) {
  const int64_t n = SPLIT ? ((int64_t)d.lots * d.heads + kWaves - 1) / kWaves : d.a.B * d.heads;
  const dim3 grid((unsigned)n), block(64 * kWaves);
  auto go = [&](auto kernel) { hipLaunchKernelGGL(kernel, grid, block, 0, stream, d); };
  const int D = d.a.head_dim;
  if (D <= 64)
    D == 64 ? go(attn_decode_kernel<64, false, CODES, SPLIT>)
            : go(attn_decode_kernel<64, true, CODES, SPLIT>);
  else if (D <= 128)
    D == 128 ? go(attn_decode_kernel<128, false, CODES, SPLIT>)
             : go(attn_decode_kernel<128, true, CODES, SPLIT>);
  else
    D == 256 ? go(attn_decode_kernel<256, false, CODES, SPLIT>)
             : go(attn_decode_kernel<256, true, CODES, SPLIT>);
}

// Of all parts, with their statistics.
int64_t part_floats(int64_t waves, int group, int head_dim) {
  return 2 * waves * min(16, group) * (head_dim + 2);
}

int head_tiles(int q_heads, int kv_heads) { return (q_heads / kv_heads + 15) / 16; }

}  // namespace

size_t attn_decode_workspace(int64_t B, int q_heads, int kv_heads, int head_dim, int64_t max_keys,
                             int window) {
  if (B == 0) return 0;
  const int64_t heads = (int64_t)kv_heads * head_tiles(q_heads, kv_heads);
  const int64_t lots = decode_lots(heads, max_keys, window, 2 * head_dim);
  if (lots == 0) return 0;
  return (size_t)part_floats(heads * lots, q_heads / kv_heads, head_dim) * sizeof(float) +
         (size_t)(B + 1) * sizeof(int);
}

hipError_t launch_attn_decode(const fp8rl_attn_decode_args& a, void* workspace, hipStream_t stream) {
  DecodeArgs d;
  d.a = a;
  d.part = static_cast<float*>(workspace);
  d.page_of = PageOf(a.page_size);
  d.group = a.q_heads / a.kv_heads;
  d.tiles = head_tiles(a.q_heads, a.kv_heads);
  d.heads = a.kv_heads * d.tiles;
  d.lots = decode_lots(d.heads, (int64_t)a.table_width * a.page_size, a.window,
                       a.head_dim * (a.k_scale ? 1 : 2));
  if (d.lots == 0) {
    a.k_scale ? run_decode<true, false>(d, stream) : run_decode<false, false>(d, stream);
    return hipGetLastError();
  }
  d.cut = reinterpret_cast<int*>(d.part + part_floats((int64_t)d.heads * d.lots, d.group, a.head_dim));
  a.k_scale ? run_decode<true, true>(d, stream) : run_decode<false, true>(d, stream);
  // a wave has sixteen of a sequence's parts in flight at a time; where there are more, eight waves
  // share them
  const int64_t items = a.B * a.q_heads;
  if (d.lots <= 16 * a.B)
    hipLaunchKernelGGL(attn_decode_join_kernel<1>, dim3((unsigned)((items + 3) / 4)), dim3(256), 0,
                       stream, d);
  else
    hipLaunchKernelGGL(attn_decode_join_kernel<8>, dim3((unsigned)items), dim3(512), 0, stream, d);
  return hipGetLastError();
}

}  // namespace fp8rl
