// What the kernels over packed documents share: documents and masks, tiles of rows in LDS, and the
// operands of the 32x32x16 matrix instruction.
//
// The instruction's layouts (lane l, h = l / 32): operand A holds row l % 32, operand B column l %
// 32, each at the 8 places 8h .. 8h + 7 of the contraction; the result's column is l % 32, its rows
// are 8 (i / 4) + 4h + i % 4 for i = 0 .. 15. The rows that a lane has of a result, eight by eight,
// serve as the places of the next contraction (16 of them: 16s + {4h .. 4h + 3, 8 + 4h .. 8 + 4h +
// 3}), so a result turns into an operand without leaving the lane, as long as the other operand
// takes its places in the same order: ColOperand does.
#pragma once

#include "attn_ops.hpp"

namespace fp8rl {

// The plain arguments, and what the launch adds.
struct AttnArgs {
  fp8rl_attn_args a;
  float* stats;  // backward: [2][q_heads][Tq], lse in units of ln 2 and <dout, out>
  float* part;   // sums of dk and dv in parts
  int parts;
  int group;     // query heads of a key head
  int slots;     // tiles of rows, every document's last one counted whole
  float scale2;  // sm_scale log2(e); capped: sm_scale / cap
  float cap2;    // cap log2(e)
};

inline AttnArgs attn_args(const fp8rl_attn_args& a, int tile, int64_t T) {
  AttnArgs d{};
  d.a = a;
  d.a.window = min(a.window, 1 << 25);  // past every distance; positions less a window stay in range
  d.group = a.q_heads / a.kv_heads;
  d.slots = (int)(T / tile + a.docs);
  d.parts = 1;
  d.scale2 = a.cap > 0.f ? a.sm_scale / a.cap : a.sm_scale * kLog2e;
  d.cap2 = a.cap * kLog2e;
  return d;
}

// A tile of BM rows of a document: of its queries, or with KEYS of its keys.
struct DocTile {
  int doc;         // docs: none
  int first;       // the tile's first row in the document
  int lq, lk;      // queries and keys of the document
  int64_t q0, k0;  // its first row of q, of k and v
};

// The tile that comes at place `index` of the launch's args.slots.
//
// Up to 64 documents: tiles that take longest first, so that the last ones to run are short. A tile
// of queries goes through the keys in front of it, one of keys through the queries behind it; with
// `weight` the number of these tiles of the other kind less those that the tile's own place adds,
// a document has a tile of each weight + 0 .. weight + tiles - 1 (not causal: all of the same). How
// many tiles there are of at least k is a sum over the documents, one to a lane, and k is found by
// its bits.
//
// (The gradients of six uneven documents of 4096 tokens in all: 202 us, document after document
// 220; the output of four, 2048 queries behind 4096 keys, a window of 1024: 30.7 and 36.5. The
// search takes about a microsecond.)
//
// More documents: from the last (with KEYS the first) document's on. Documents take
//   rows[d + 1] / BM + d + 1 - (rows[d] / BM + d)  >=  ceil(length / BM)
// places each, so that a tile is found from the offsets alone.
template <int BM, bool KEYS>
__device__ __forceinline__ DocTile find_tile(const AttnArgs& args, int index, int lane) {
  const fp8rl_attn_args& a = args.a;
  const int n = (int)a.docs, Tq = (int)a.Tq, Tk = (int)a.Tk;
  auto q_at = [&](int i) { return min(max(a.q_offsets[i], 0), Tq); };
  auto k_at = [&](int i) { return min(max(a.k_offsets[i], 0), Tk); };
  DocTile t;
  t.doc = n;
  if (n <= 64) {
    int q0 = 0, k0 = 0, lq = 0, lk = 0;
    if (lane < n) {
      q0 = q_at(lane), k0 = k_at(lane);
      lq = max(0, q_at(lane + 1) - q0), lk = max(0, k_at(lane + 1) - k0);
    }
    const int own = KEYS ? lk : lq, other = KEYS ? lq : lk;
    const int tiles = (own + BM - 1) / BM;
    const int weight = (a.causal ? max(0, other - own) : other) / BM;
    // tiles of at least k
    auto heavy = [&](int k) {
      return a.causal ? min(max(tiles + weight - k, 0), tiles) : weight >= k ? tiles : 0;
    };
    auto all_heavy = [&](int k) { return __builtin_amdgcn_readlane(sum_upto(heavy(k)), 63); };
    if (index >= all_heavy(0)) return t;
    int bit = 1, k = 0;
    while (__ballot(tiles + weight >= bit)) bit *= 2;
    for (; bit > 0; bit /= 2)
      if (index < all_heavy(k + bit)) k += bit;
    const int rest = index - all_heavy(k + 1);
    const int mine = heavy(k) - heavy(k + 1);
    const int upto = sum_upto(mine);
    const int d = __builtin_ctzll(__ballot(upto > rest));
    const int at = a.causal ? k - weight : rest - (upto - mine);
    t.doc = d;
    t.first = BM * __builtin_amdgcn_readlane(KEYS && a.causal ? tiles - 1 - at : at, d);
    t.q0 = __builtin_amdgcn_readlane(q0, d), t.k0 = __builtin_amdgcn_readlane(k0, d);
    t.lq = __builtin_amdgcn_readlane(lq, d), t.lk = __builtin_amdgcn_readlane(lk, d);
    return t;
  }
  const int slot = KEYS ? index : args.slots - 1 - index;
  const int d =
      last_not_past(n, slot, lane, [&](int i) { return (KEYS ? k_at(i) : q_at(i)) / BM + i; });
  if (d >= n) return t;
  t.q0 = q_at(d), t.k0 = k_at(d);
  t.lq = max(0, q_at(d + 1) - (int)t.q0);
  t.lk = max(0, k_at(d + 1) - (int)t.k0);
  t.first = (slot - ((int)(KEYS ? t.k0 : t.q0) / BM + d)) * BM;
  if (t.first >= 0 && t.first < (KEYS ? t.lk : t.lq)) t.doc = d;
  return t;
}

// Which keys a query at position p sees: lo <= j < hi, or j < prefix.
struct Mask {
  int prefix, lk, window;
  bool causal;
  __device__ __forceinline__ Mask(const fp8rl_attn_args& a, const DocTile& t)
      : prefix(a.prefix ? min(max(a.prefix[t.doc], 0), t.lk) : 0),
        lk(t.lk),
        window(a.window),
        causal(a.causal) {}
  __device__ __forceinline__ int hi(int p) const { return causal ? min(p + 1, lk) : lk; }
  __device__ __forceinline__ int lo(int p) const { return window ? max(0, p - window + 1) : 0; }
  // Whether queries at positions p0 <= .. <= p1 see all (any) of the keys j0 <= .. < j1.
  __device__ __forceinline__ bool all(int p0, int p1, int j0, int j1) const {
    return j1 <= prefix || (j1 <= hi(p0) && j0 >= lo(p1));
  }
  __device__ __forceinline__ bool any(int p0, int p1, int j0, int j1) const {
    return j0 < prefix || (j0 < hi(p1) && j1 > lo(p0));
  }
};

// The scores of values v, mul v, less slope2 times the distances far(e). (Loops of their own, so
// that they stay in one piece under branches that are the same for a call.)
template <typename Far>
__device__ __forceinline__ void slope_scores(f32x16& v, float mul, float slope2, Far far) {
#pragma unroll
  for (int e = 0; e < 16; ++e) v[e] = __builtin_fmaf(-slope2, fabsf(far(e)), v[e] * mul);
}

// ------------------------------------------------------------------------------ rows in LDS

// A tile of rows of DP bf16 values, 16-byte chunks c of row r at place c ^ swizzle(r): reads of one
// chunk of consecutive rows, and of 64 consecutive bytes of four rows, spread over the banks.
template <int DP>
__device__ __forceinline__ int swizzle(int r) {
  return DP == 64 ? ((r & 1) << 2) | ((r >> 1) & 3) : ((r & 3) << 2) | ((r >> 2) & 3);
}

typedef __attribute__((address_space(3))) void* lds_void_t;

__device__ __forceinline__ const void* scalar_ptr(const void* p) {
  const uint64_t v = (uint64_t)(uintptr_t)p;
  const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)v);
  const uint32_t hi = __builtin_amdgcn_readfirstlane((uint32_t)(v >> 32));
  return (const void*)(uintptr_t)(((uint64_t)hi << 32) | lo);
}

// 16 bytes a lane from base + off (base the same in all lanes) to lds + 16 * lane, past the
// registers. In assembly because the compiler would wait for every such load in flight before any
// read of LDS; landed() waits instead. The address may come from v_readfirstlane right before,
// which needs 5 wait states, and M0 needs 1.
__device__ __forceinline__ void dma_rows(const void* base, uint32_t off, const void* lds) {
  const uint32_t m0 = __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)(lds_void_t)lds);
  asm volatile("s_nop 4\n\tglobal_load_lds_dwordx4 %0, %1"
               :: "v"(off), "s"(scalar_ptr(base)), "{m0}"(m0) : "memory");
}

// The same, 4 bytes a lane to lds + 4 * lane.
__device__ __forceinline__ void dma_floats(const void* base, uint32_t off, const void* lds) {
  const uint32_t m0 = __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)(lds_void_t)lds);
  asm volatile("s_nop 4\n\tglobal_load_lds_dword %0, %1"
               :: "v"(off), "s"(scalar_ptr(base)), "{m0}"(m0) : "memory");
}

// This wave's loads but the last N have arrived and its reads of LDS are done, and so with the
// others.
template <int N = 0>
__device__ __forceinline__ void landed() {
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(N) : "memory");
}

// N rows of a matrix (pitch ld) into LDS by W waves, those from `rows` on as copies of the last
// one, columns past the head's as its first ones (what becomes of them is masked or not stored).
template <int DP, int N, int W>
struct RowLoader {
  static constexpr int kChunks = DP / 8;         // of a row
  static constexpr int kRows = 64 / kChunks;     // of an instruction
  static constexpr int kOps = N / kRows / W;     // of a wave
  static_assert(kOps * kRows * W == N, "rows of a tile");
  static_assert(kRows * W % (DP == 64 ? 8 : 16) == 0, "one swizzle for a lane's rows");
  int row;          // of the first load; the others' are W * kRows further each
  uint32_t column;  // bytes

  __device__ __forceinline__ RowLoader(int head_dim, int wave, int lane)
      : row(wave * kRows + lane / kChunks) {
    const int c = (lane % kChunks) ^ swizzle<DP>(row);
    column = 8 * c < head_dim ? 16 * c : 0;
  }
  __device__ __forceinline__ void load(const uint16_t* first, int64_t ld, int rows, uint8_t* lds,
                                       int wave) const {
#pragma unroll
    for (int i = 0; i < kOps; ++i)
      dma_rows(first, (uint32_t)min(row + i * W * kRows, rows - 1) * ((uint32_t)ld * 2) + column,
               lds + (i * W + wave) * 1024);
  }
};

// Rows from `rows` on set to zero.
template <int DP, int N, int W>
__device__ __forceinline__ void clear_rows(uint8_t* lds, int rows) {
  for (int i = rows * (DP / 8) + (int)threadIdx.x; i < N * (DP / 8); i += 64 * W)
    reinterpret_cast<u32x4*>(lds)[i] = u32x4{0u, 0u, 0u, 0u};
}

// Operand A or B of 32 rows of a tile from row r0 (a multiple of 32) on, step s of the contraction
// over the columns: lane l has row l % 32, columns 16s + 8h ...
template <int DP>
struct RowOperand {
  const uint8_t* row;
  int f, h;
  __device__ __forceinline__ RowOperand(const uint8_t* lds, int lane)
      : row(lds + (lane & 31) * DP * 2), f(swizzle<DP>(lane & 31)), h(lane >> 5) {}
  __device__ __forceinline__ bf16x8 operator()(int r0, int s) const {
    return *reinterpret_cast<const bf16x8*>(row + r0 * DP * 2 + (((2 * s + h) ^ f) << 4));
  }
};

// Operand A or B transposed: 32 columns from 32 t on as its rows, step s of the contraction over
// the tile's rows: lane l has column 32 t + l % 32, rows r0 + {4h .. 4h + 3, 8 + 4h .. 8 + 4h + 3}
// (r0 a multiple of 16). ds_read_b64_tr_b16 deals the 16 x 4 values that 16 lanes point to out by
// columns.
template <int DP>
struct ColOperand {
  typedef short s16x4 __attribute__((ext_vector_type(4)));
  const uint8_t* row;
  int window, inner[2], odd;
  __device__ __forceinline__ ColOperand(const uint8_t* lds, int lane) {
    const int h = lane >> 5, i = (lane & 15) >> 2;  // row 4h + i of eight, 8 further in the second
    row = lds + (4 * h + i) * DP * 2;
    odd = (lane & 1) * 8;
    const int c = ((lane >> 4) & 1) * 2 + ((lane & 3) >> 1);
    // the swizzle's two parts: which 64 bytes of the row, which 16 of these
    const int f0 = swizzle<DP>(4 * h + i), f1 = swizzle<DP>(8 + 4 * h + i);
    window = f0 >> 2;  // the same in both
    inner[0] = (c ^ (f0 & 3)) << 4;
    inner[1] = (c ^ (f1 & 3)) << 4;
  }
  __device__ __forceinline__ bf16x8 operator()(int r0, int t) const {
    typedef __attribute__((address_space(3))) s16x4* p_t;
    const uint8_t* at = row + r0 * DP * 2 + ((t * 4) ^ (window << 2)) * 16 + odd;
    const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((p_t)(at + inner[0]));
    const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((p_t)(at + 8 * DP * 2 + inner[1]));
    typedef short s16x8 __attribute__((ext_vector_type(8)));
    return __builtin_bit_cast(
        bf16x8, (s16x8{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]}));
  }
};

// Eight values of a result, i = 8s .. 8s + 7, rounded to the operand of step s.
__device__ __forceinline__ bf16x8 operand_of(const f32x16& v, int s) {
  return __builtin_bit_cast(bf16x8, (u32x4{pack2_bf16(v[8 * s], v[8 * s + 1]),
                                           pack2_bf16(v[8 * s + 2], v[8 * s + 3]),
                                           pack2_bf16(v[8 * s + 4], v[8 * s + 5]),
                                           pack2_bf16(v[8 * s + 6], v[8 * s + 7])}));
}

// Operand B (or A) of 32 rows straight from memory, step s: zeros past the head's columns.
__device__ __forceinline__ bf16x8 row_operand(const uint16_t* row, int s, int h, int head_dim) {
  const int c = 16 * s + 8 * h;
  u32x4 t{0u, 0u, 0u, 0u};
  if (c < head_dim) t = *reinterpret_cast<const u32x4*>(row + c);
  return __builtin_bit_cast(bf16x8, t);
}

// A result with a row of the matrix in each column (lane l: row l % 32, columns c0 + 8 (i / 4) + 4h
// + i % 4), times f, rounded and stored where `in`: 16 bytes a lane after the two halves of the
// wave have exchanged every other four.
__device__ __forceinline__ void store_columns(const f32x16& v, float f, uint16_t* row, int c0, int h,
                                              int head_dim, bool in) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    if (c0 + 16 * i >= head_dim) return;
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
      w[j] = pack2_bf16(v[8 * i + 2 * j] * f, v[8 * i + 2 * j + 1] * f);
    const auto x = __builtin_amdgcn_permlane32_swap(w[0], w[2], false, false);
    const auto y = __builtin_amdgcn_permlane32_swap(w[1], w[3], false, false);
    if (in)
      *reinterpret_cast<u32x4*>(row + c0 + 16 * i + 8 * h) = u32x4{x[0], y[0], x[1], y[1]};
  }
}

__device__ __forceinline__ f32x16 zeros16() {
  f32x16 z;
#pragma unroll
  for (int i = 0; i < 16; ++i) z[i] = 0.f;
  return z;
}

}  // namespace fp8rl
