// Mixture-of-experts rows: the router's choices in expert order, rows moved there, and the experts'
// rows weighted and summed back, with the gradients of that sum.
#include "block_ops.hpp"

namespace fp8rl {

// ---------------------------------------------------------------------------------------------
// Stable counting sort of n choices by expert. The choices are cut into one contiguous piece per
// wave (16 waves per workgroup), and the grouped row of a choice is
//   (choices of lower experts) + (choices of its expert in earlier pieces)
//   + (choices of its expert before it in its piece).
// The first two terms come from per-wave histograms in LDS; the last is kept by one wave walking
// its piece 64 choices at a time, where lanes with the same expert find each other by one ballot
// per bit of the expert's number: a lane's place among them is the number of set bits below it.
// Nothing depends on the order in which waves run. One workgroup sorts up to kSortOne choices, every
// lane keeping its four in registers from the histogram to the placing; more are cut into blocks,
// whose histograms a first kernel leaves in the workspace and every block of the second one sums for
// itself. Latency and the matching's instructions bound it, not its bytes: 3.7 us for 512 choices of
// 128 experts, 6.1 us for 4096 (one workgroup for 8192 takes 10 us, two kernels 7.7), 9.4 us for
// 65536, 14.1 us for 524288. Counting by the matching too, to save LDS additions to one address, was
// slower (12.8 us for 65536).
// ---------------------------------------------------------------------------------------------
constexpr int kSortWaves = 16;
constexpr int kSortLoads = 4;  // choices a lane has in flight and keeps: a wave's tile is 256
constexpr int64_t kSortOne = 64 * kSortLoads * kSortWaves;  // a tile for each wave
constexpr int64_t kSortMostBlocks = 256;

int64_t sort_blocks(int64_t n) {
  if (n <= kSortOne) return 1;
  const int64_t b = (n + kSortOne - 1) / kSortOne;
  return b < kSortMostBlocks ? b : kSortMostBlocks;
}

namespace {

// Choices of one wave of a sort in `blocks` blocks: whole groups of 64.
int64_t sort_piece(int64_t n, int64_t blocks) {
  const int64_t waves = blocks * kSortWaves;
  return ((n + waves - 1) / waves + 63) / 64 * 64;
}

// The experts of a wave's choices i0 + 64 j + lane, E (counted nowhere) for one without an expert
// or past the end.
template <typename ID>
__device__ __forceinline__ void load_tile(const ID* __restrict__ ids, int64_t i0, int64_t end,
                                          int E, int (&e)[kSortLoads]) {
  ID id[kSortLoads];
#pragma unroll
  for (int j = 0; j < kSortLoads; ++j) {
    const int64_t i = i0 + 64 * j + (threadIdx.x & 63);
    id[j] = -1;
    if (i < end) id[j] = ids[i];
  }
#pragma unroll
  for (int j = 0; j < kSortLoads; ++j) e[j] = id[j] >= 0 && id[j] < (ID)E ? (int)id[j] : E;
}

// Integers: the counts are the same in any order of the additions.
__device__ __forceinline__ void count_tile(const int (&e)[kSortLoads], int E, int* cnt) {
#pragma unroll
  for (int j = 0; j < kSortLoads; ++j)
    if (e[j] < E) atomicAdd(&cnt[e[j]], 1);
}

// Lanes of the wave with this lane's expert: for each bit, those whose bit is the same.
__device__ __forceinline__ uint64_t same_expert(int e, int bits) {
  uint32_t lo = ~0u, hi = ~0u;
#pragma unroll
  for (int b = 0; b < 11; ++b) {
    if (b >= bits) break;
    const uint32_t mine = (uint32_t)__builtin_amdgcn_sbfe(e, (unsigned)b, 1u);  // all ones or zeros
    const uint64_t set = __ballot(mine != 0);
    lo &= ~((uint32_t)set ^ mine);
    hi &= ~((uint32_t)(set >> 32) ^ mine);
  }
  return (uint64_t)hi << 32 | lo;
}

}  // namespace

template <typename ID>
__global__ __launch_bounds__(1024) void moe_count_kernel(const ID* __restrict__ ids, int64_t n,
                                                         int64_t piece, int E,
                                                         int32_t* __restrict__ counts) {
  extern __shared__ int cnt[];  // [E]
  const int64_t begin = ((int64_t)blockIdx.x * kSortWaves + (threadIdx.x >> 6)) * piece;
  const int64_t end = begin + piece < n ? begin + piece : n;
  int e[kSortLoads];
  load_tile(ids, begin, end, E, e);
  for (int i = threadIdx.x; i < E; i += 1024) cnt[i] = 0;
  __syncthreads();
  count_tile(e, E, cnt);
  for (int64_t i0 = begin + 64 * kSortLoads; i0 < end; i0 += 64 * kSortLoads) {
    load_tile(ids, i0, end, E, e);
    count_tile(e, E, cnt);
  }
  __syncthreads();
  for (int i = threadIdx.x; i < E; i += 1024) counts[(int64_t)blockIdx.x * E + i] = cnt[i];
}

// counts: [gridDim.x][E] of moe_count_kernel, or null for a single block.
template <typename ID>
__global__ __launch_bounds__(1024) void moe_place_kernel(const ID* __restrict__ ids, int64_t n,
                                                         int64_t piece, int top_k, int E, int bits,
                                                         const int32_t* __restrict__ counts,
                                                         int32_t* __restrict__ offsets,
                                                         int32_t* __restrict__ row_ids,
                                                         int32_t* __restrict__ pos) {
  extern __shared__ int cnt[];  // [kSortWaves][E]
  __shared__ int wave_total[kSortWaves];
  const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
  const int64_t begin = ((int64_t)blockIdx.x * kSortWaves + wave) * piece;
  const int64_t end = begin + piece < n ? begin + piece : n;
  int* mine = cnt + wave * E;
  int e[kSortLoads];
  load_tile(ids, begin, end, E, e);

  // expert t's choices in earlier blocks and in all
  int total = 0, before = 0;
  if (counts && t < E) {
#pragma unroll 8
    for (int b = 0; b < (int)gridDim.x; ++b) {
      const int c = counts[(int64_t)b * E + t];
      total += c;
      before += b < (int)blockIdx.x ? c : 0;
    }
  }
  for (int i = t; i < kSortWaves * E; i += 1024) cnt[i] = 0;
  __syncthreads();
  count_tile(e, E, mine);
  for (int64_t i0 = begin + 64 * kSortLoads; i0 < end; i0 += 64 * kSortLoads) {
    int more[kSortLoads];
    load_tile(ids, i0, end, E, more);
    count_tile(more, E, mine);
  }
  __syncthreads();
  if (!counts && t < E)
    for (int w = 0; w < kSortWaves; ++w) total += cnt[w * E + t];

  // exclusive prefix of the totals over the experts
  int incl = total;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int up = __shfl_up(incl, o, 64);
    if (lane >= o) incl += up;
  }
  if (lane == 63) wave_total[wave] = incl;
  __syncthreads();
  int base = incl - total, all = 0;
#pragma unroll
  for (int w = 0; w < kSortWaves; ++w) {
    base += w < wave ? wave_total[w] : 0;
    all += wave_total[w];
  }
  if (blockIdx.x == 0) {
    if (t < E) offsets[t] = base;
    if (t == 0) offsets[E] = all;
  }
  if (t < E) {
    int next = base + before;
    for (int w = 0; w < kSortWaves; ++w) {
      const int c = cnt[w * E + t];
      cnt[w * E + t] = next;  // the first grouped row of this wave's choices of expert t
      next += c;
    }
  }
  __syncthreads();

  for (int64_t i0 = begin; i0 < end; i0 += 64 * kSortLoads) {
    if (i0 != begin) load_tile(ids, i0, end, E, e);
#pragma unroll
    for (int j = 0; j < kSortLoads; ++j) {
      if (i0 + 64 * j >= end) break;
      const int64_t i = i0 + 64 * j + lane;
      const uint64_t same = same_expert(e[j], bits);
      const int below = __popcll(same & ((1ull << lane) - 1));
      int at = 0;
      if (below == 0 && e[j] < E) at = atomicAdd(&mine[e[j]], (int)__popcll(same));
      at = __shfl(at, __ffsll((unsigned long long)same) - 1, 64) + below;
      if (i < end) {
        pos[i] = e[j] < E ? at : -1;
        // (at < n but for ids that change while the call runs)
        if (e[j] < E && at < n) row_ids[at] = (int)((unsigned)i / (unsigned)top_k);
      }
    }
  }
  // no row behind the last expert's
  for (int64_t i = all + (int64_t)blockIdx.x * 1024 + t; i < n; i += (int64_t)gridDim.x * 1024)
    row_ids[i] = -1;
}

namespace {

template <typename ID>
hipError_t run_sort(const ID* ids, int64_t n, int top_k, int E, int32_t* offsets, int32_t* row_ids,
                    int32_t* pos, int32_t* counts, hipStream_t stream) {
  const int64_t blocks = sort_blocks(n);
  const int64_t piece = sort_piece(n, blocks);
  int bits = 1;
  while ((1 << bits) <= E) ++bits;  // E itself stands for "no expert"
  if (blocks > 1) {
    hipLaunchKernelGGL(moe_count_kernel<ID>, dim3((unsigned)blocks), dim3(1024), E * sizeof(int),
                       stream, ids, n, piece, E, counts);
    if (hipError_t e = hipGetLastError(); e != hipSuccess) return e;
  }
  hipLaunchKernelGGL(moe_place_kernel<ID>, dim3((unsigned)blocks), dim3(1024),
                     (size_t)kSortWaves * E * sizeof(int), stream, ids, n, piece, top_k, E, bits,
                     blocks > 1 ? counts : nullptr, offsets, row_ids, pos);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_moe_sort(const void* ids, bool wide, int64_t n, int top_k, int E,
                           int32_t* offsets, int32_t* row_ids, int32_t* pos, int32_t* counts,
                           hipStream_t stream) {
  return wide ? run_sort(static_cast<const int64_t*>(ids), n, top_k, E, offsets, row_ids, pos,
                         counts, stream)
              : run_sort(static_cast<const int32_t*>(ids), n, top_k, E, offsets, row_ids, pos,
                         counts, stream);
}

// ---------------------------------------------------------------------------------------------
// Rows. A workgroup owns a token; a lane owns chunks of 8 values of the row. A value type Y or O is
// float or uint16_t (bf16).
//
// The choices of a token that have a grouped row are found once per wave: lane j reads pos[t][j], a
// ballot marks the live ones, and their rows (and weights) are read out of the lanes in increasing
// order into scalar registers. Rows are then loaded S at a time without a branch between the loads,
// so that all of them are in flight; places past the last live choice load its row again and are
// taken out of the result by a select, never by a zero weight, which would let a NaN through.
// ---------------------------------------------------------------------------------------------
namespace {

// 8 values as they lie in memory: what a load in flight occupies.
template <typename T>
struct Raw8;
template <>
struct Raw8<uint16_t> {
  u32x4 v;
  __device__ __forceinline__ void load(const uint16_t* p) {
    v = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(p));
  }
  __device__ __forceinline__ void widen(float (&f)[8]) const { widen8(v, f); }
};
template <>
struct Raw8<float> {
  f32x4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = __builtin_nontemporal_load(reinterpret_cast<const f32x4*>(p));
    b = __builtin_nontemporal_load(reinterpret_cast<const f32x4*>(p) + 1);
  }
  __device__ __forceinline__ void widen(float (&f)[8]) const {
    f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w, f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
  }
};

// Stores past the caches (NT) where rows start on 128-byte lines, plain ones elsewhere, whose parts
// of a line meet in the L2: dy of 8 x 2048 values for 4096 tokens 55.6 against 59.4 us; 8 x 1032,
// where every row shares a line with the next, 37.0 against 30.8 us. That is scattered rows; combine
// writes its rows in order and stores past the caches wherever they start: 8192 tokens of 1032
// values 29.6 against 30.8 us from 8 choices, 10.5 against 11.3 us from one, 12.5 against 13.4 us
// where three choices in four are another rank's (37 tokens: 3.0 against 2.7 us).
template <bool NT, typename V>
__device__ __forceinline__ void put(const V& v, V* p) {
  if (NT)
    __builtin_nontemporal_store(v, p);
  else
    *p = v;
}
template <bool NT>
__device__ __forceinline__ void store8(uint16_t* p, const float (&f)[8]) {
  put<NT>(round8(f), reinterpret_cast<u32x4*>(p));
}
template <bool NT>
__device__ __forceinline__ void store8(float* p, const float (&f)[8]) {
  put<NT>(f32x4{f[0], f[1], f[2], f[3]}, reinterpret_cast<f32x4*>(p));
  put<NT>(f32x4{f[4], f[5], f[6], f[7]}, reinterpret_cast<f32x4*>(p) + 1);
}

// A token's live choices, held across the lanes of a wave.
struct Choices {
  int row;         // lane j: grouped row of choice j
  float weight;    // lane j: its weight
  uint64_t live;   // lanes with a row in [0, R)
  __device__ __forceinline__ void read(const MoeArgs& a, int64_t t) {
    const int lane = threadIdx.x & 63;
    row = -1;
    weight = 1.f;
    if (lane < a.top_k) {
      row = a.pos[t * a.top_k + lane];
      if (a.weights) weight = a.weights[t * a.top_k + lane];
    }
    live = __ballot(row >= 0 && row < a.R);
  }
};

// The next S live choices out of `left` (which loses them): lane numbers, the last one repeated.
template <int S>
__device__ __forceinline__ int take(uint64_t& left, int (&lane)[S]) {
  int n = 0, last = 0;
#pragma unroll
  for (int j = 0; j < S; ++j) {
    if (left) last = __ffsll((unsigned long long)left) - 1, ++n;
    left &= left - 1;  // 0 stays 0: 0 & anything
    lane[j] = last;
  }
  return n;
}

template <int S, typename Y>
__device__ __forceinline__ void combine_step(const MoeArgs& a, const Choices& ch, uint64_t& left,
                                             int c, float (&acc)[8]) {
  int lane[S];
  const int n = take<S>(left, lane);
  Raw8<Y> f[S];
#pragma unroll
  for (int j = 0; j < S; ++j) {
    const int64_t p = __builtin_amdgcn_readlane(ch.row, lane[j]);
    f[j].load(static_cast<const Y*>(a.x) + p * a.ld_x + c * 8);
  }
#pragma unroll
  for (int j = 0; j < S; ++j) {
    const float w = __uint_as_float(
        (uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(ch.weight), lane[j]));
    float v[8];
    f[j].widen(v);
#pragma unroll
    for (int k = 0; k < 8; ++k) acc[k] = j < n ? __builtin_fmaf(w, v[k], acc[k]) : acc[k];
  }
}

}  // namespace

// A wave takes a block of 64 CH chunks of one token's row, reads it once and writes it to each of
// the token's grouped rows: 302 MB at 8191 tokens of 8 x 2048 values in 58.5 us, 5.2 TB/s, bound by
// its writes (rows in order instead of scattered: 51 us). By grouped rows instead of tokens, each
// token would be read top_k times: 92 us.
template <int CH, bool NT>
__global__ __launch_bounds__(256) void moe_dispatch_kernel(MoeArgs a, int pieces) {
  const unsigned w = blockIdx.x * 4 + (threadIdx.x >> 6);
  const unsigned t = w / (unsigned)pieces;
  if (t >= a.T) return;
  const int c0 = (int)(w - t * pieces) * (64 * CH) + (int)(threadIdx.x & 63);
  const u32x4* x =
      reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(a.x) + (int64_t)t * a.ld_x);
  u32x4 v[CH];
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    v[i] = u32x4{0u, 0u, 0u, 0u};
    if (c0 + 64 * i < a.nc) v[i] = __builtin_nontemporal_load(x + c0 + 64 * i);
  }
  Choices ch;
  ch.read(a, t);
  for (uint64_t left = ch.live; left; left &= left - 1) {
    const int64_t p = __builtin_amdgcn_readlane(ch.row, __ffsll((unsigned long long)left) - 1);
    u32x4* out = reinterpret_cast<u32x4*>(static_cast<uint16_t*>(a.out) + p * a.ld_out) + c0;
#pragma unroll
    for (int i = 0; i < CH; ++i)
      if (c0 + 64 * i < a.nc) put<NT>(v[i], out + 64 * i);
  }
}

// A workgroup owns a token. 302 MB at 8192 tokens of 8 x 2048 values in 52 us, 5.8 TB/s, bound by
// memory; with a branch around each load, which then waits for its own, 68 us.
template <typename Y, typename O>
__global__ __launch_bounds__(256) void moe_combine_kernel(MoeArgs a) {
  const int64_t t = blockIdx.x;
  Choices ch;
  ch.read(a, t);
  for (int c = threadIdx.x; c < a.nc; c += blockDim.x) {
    float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    for (uint64_t left = ch.live; left;) {
      const int n = __popcll(left);
      if (n > 4)
        combine_step<8, Y>(a, ch, left, c, acc);
      else if (n > 2)
        combine_step<4, Y>(a, ch, left, c, acc);
      else
        combine_step<2, Y>(a, ch, left, c, acc);
    }
    store8<true>(static_cast<O*>(a.out) + t * a.ld_out + c * 8, acc);
  }
}

namespace {

// Sums of S values over the 64 lanes of a wave: each exchange between lanes l and l ^ o halves the
// number of values a lane holds, so S values cost S - 1 + log2(64 / S) exchanges instead of 6 S.
// Returns the sum of value (lane / (64 / S)) in every lane.
template <int S>
__device__ __forceinline__ float wave_sums(float (&v)[S]) {
  const int lane = threadIdx.x & 63;
  int o = 32;
#pragma unroll
  for (int n = S; n > 1; n >>= 1, o >>= 1) {
    const bool up = lane & o;
#pragma unroll
    for (int i = 0; i < n / 2; ++i) {
      const float keep = up ? v[i + n / 2] : v[i], give = up ? v[i] : v[i + n / 2];
      v[i] = keep + __shfl_xor(give, o, 64);
    }
  }
  float s = v[0];
#pragma unroll
  for (; o > 0; o >>= 1) s += __shfl_xor(s, o, 64);
  return s;
}

// S live choices of the token: their rows' products with dout, and their gradients.
template <int S, bool NT, typename Y>
__device__ __forceinline__ void combine_bwd_step(const MoeArgs& a, const Choices& ch,
                                                 uint64_t& left, int64_t t, float (*red)[8]) {
  int lane[S];
  const int n = take<S>(left, lane);
  const uint16_t* dout = static_cast<const uint16_t*>(a.x) + t * a.ld_x;
  float dot[S];
#pragma unroll
  for (int j = 0; j < S; ++j) dot[j] = 0.f;
  for (int c = threadIdx.x; c < a.nc; c += blockDim.x) {
    Raw8<uint16_t> gr;
    gr.load(dout + c * 8);
    Raw8<Y> f[S];
    if (a.y) {
#pragma unroll
      for (int j = 0; j < S; ++j) {
        const int64_t p = __builtin_amdgcn_readlane(ch.row, lane[j]);
        f[j].load(static_cast<const Y*>(a.y) + p * a.ld_y + c * 8);
      }
    }
    float g[8];
    gr.widen(g);
    if (a.y) {
#pragma unroll
      for (int j = 0; j < S; ++j) {
        float v[8];
        f[j].widen(v);
#pragma unroll
        for (int k = 0; k < 8; ++k) dot[j] = __builtin_fmaf(g[k], v[k], dot[j]);
      }
    }
#pragma unroll
    for (int j = 0; j < S; ++j) {
      if (j >= n) break;
      const int64_t p = __builtin_amdgcn_readlane(ch.row, lane[j]);
      const float w = __uint_as_float(
          (uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(ch.weight), lane[j]));
      float d[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) d[k] = w * g[k];
      store8<NT>(static_cast<Y*>(a.out) + p * a.ld_out + c * 8, d);
    }
  }
  if (!a.dweights) return;
  const float s = wave_sums<S>(dot);
  const int l = threadIdx.x & 63;
  __syncthreads();  // the sums of the choices before have been read
  if (l % (64 / S) == 0) red[threadIdx.x >> 6][l / (64 / S)] = s;
  __syncthreads();
  if (threadIdx.x < n) {
    float sum = red[0][threadIdx.x];
    for (int k = 1; k < (int)(blockDim.x >> 6); ++k) sum += red[k][threadIdx.x];
    int j = lane[0];
#pragma unroll
    for (int i = 1; i < S; ++i) j = threadIdx.x == i ? lane[i] : j;
    a.dweights[t * a.top_k + j] = sum;
  }
}

}  // namespace

// A workgroup owns a token: dout is read once for all of its choices. 286 MB at 4096 tokens of
// 8 x 2048 values in 56 us, 5.1 TB/s, bound by memory (a copy of this size: 5.2 - 5.5 TB/s).
// y may be the output: a lane reads the values that it overwrites, and reads them first.
template <bool NT, typename Y>
__global__ __launch_bounds__(256) void moe_combine_bwd_kernel(MoeArgs a) {
  __shared__ float red[4][8];
  const int64_t t = blockIdx.x;
  Choices ch;
  ch.read(a, t);
  if (a.dweights && (int)threadIdx.x < a.top_k && !((ch.live >> threadIdx.x) & 1))
    a.dweights[t * a.top_k + threadIdx.x] = 0.f;
  for (uint64_t left = ch.live; left;) {
    const int n = __popcll(left);
    if (n > 4)
      combine_bwd_step<8, NT, Y>(a, ch, left, t, red);
    else if (n > 2)
      combine_bwd_step<4, NT, Y>(a, ch, left, t, red);
    else
      combine_bwd_step<2, NT, Y>(a, ch, left, t, red);
  }
}

namespace {

// Threads of a workgroup that owns one token: a lane per chunk, up to four waves.
dim3 row_threads(int nc) { return dim3(nc >= 256 ? 256 : nc > 64 ? (nc + 63) / 64 * 64 : 64); }

// Whether rows of `bytes` pitch from p on start on 128-byte lines.
bool on_lines(const void* p, int64_t bytes) {
  return (reinterpret_cast<uintptr_t>(p) | (uintptr_t)bytes) % 128 == 0;
}

template <int CH>
hipError_t run_dispatch(const MoeArgs& a, hipStream_t stream) {
  const int64_t pieces = (a.nc + 64 * CH - 1) / (64 * CH);
  const dim3 grid((unsigned)((a.T * pieces + 3) / 4));
  if (on_lines(a.out, 2 * a.ld_out))
    hipLaunchKernelGGL((moe_dispatch_kernel<CH, true>), grid, dim3(256), 0, stream, a, (int)pieces);
  else
    hipLaunchKernelGGL((moe_dispatch_kernel<CH, false>), grid, dim3(256), 0, stream, a,
                       (int)pieces);
  return hipGetLastError();
}

template <bool NT>
void run_combine_bwd(const MoeArgs& a, bool y_f32, hipStream_t stream) {
  const dim3 g((unsigned)a.T), t = row_threads(a.nc);
  if (y_f32)
    hipLaunchKernelGGL((moe_combine_bwd_kernel<NT, float>), g, t, 0, stream, a);
  else
    hipLaunchKernelGGL((moe_combine_bwd_kernel<NT, uint16_t>), g, t, 0, stream, a);
}

}  // namespace

hipError_t launch_moe_dispatch(const MoeArgs& a, hipStream_t stream) {
  // four chunks a lane (58.5 us at 8191 tokens of 8 x 2048; one: 60.1), one where that would leave
  // CUs without waves
  const int64_t wide = (a.nc + 255) / 256;
  return a.T * wide >= 2048 ? run_dispatch<4>(a, stream) : run_dispatch<1>(a, stream);
}

hipError_t launch_moe_combine(const MoeArgs& a, bool y_f32, bool out_f32, hipStream_t stream) {
  const dim3 g((unsigned)a.T), t = row_threads(a.nc);
  if (y_f32 && out_f32)
    hipLaunchKernelGGL((moe_combine_kernel<float, float>), g, t, 0, stream, a);
  else if (y_f32)
    hipLaunchKernelGGL((moe_combine_kernel<float, uint16_t>), g, t, 0, stream, a);
  else if (out_f32)
    hipLaunchKernelGGL((moe_combine_kernel<uint16_t, float>), g, t, 0, stream, a);
  else
    hipLaunchKernelGGL((moe_combine_kernel<uint16_t, uint16_t>), g, t, 0, stream, a);
  return hipGetLastError();
}

hipError_t launch_moe_combine_bwd(const MoeArgs& a, bool y_f32, hipStream_t stream) {
  if (on_lines(a.out, (y_f32 ? 4 : 2) * a.ld_out))
    run_combine_bwd<true>(a, y_f32, stream);
  else
    run_combine_bwd<false>(a, y_f32, stream);
  return hipGetLastError();
}

}  // namespace fp8rl
