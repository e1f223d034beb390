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
// Nothing depends on the order in which waves run. One workgroup sorts up to kSortOne choices; more
// are cut into blocks, whose histograms a first kernel leaves in the workspace and every block of
// the second one sums for itself.
// ---------------------------------------------------------------------------------------------
constexpr int kSortWaves = 16;
constexpr int64_t kSortOne = 16384;
constexpr int64_t kSortBlock = 8192;
constexpr int64_t kSortMostBlocks = 256;

int64_t sort_blocks(int64_t n) {
  if (n <= kSortOne) return 1;
  const int64_t b = (n + kSortBlock - 1) / kSortBlock;
  return b < kSortMostBlocks ? b : kSortMostBlocks;
}

namespace {

// Choices of one wave of a sort in `blocks` blocks: whole groups of 64.
int64_t sort_piece(int64_t n, int64_t blocks) {
  const int64_t waves = blocks * kSortWaves;
  return ((n + waves - 1) / waves + 63) / 64 * 64;
}

// The expert of choice i, or E (counted nowhere) when it has none.
template <typename ID>
__device__ __forceinline__ int expert_of(const ID* __restrict__ ids, int64_t i, int64_t end, int E) {
  if (i >= end) return E;
  const ID e = ids[i];
  return e >= 0 && e < (ID)E ? (int)e : E;
}

template <typename ID>
__device__ __forceinline__ void count_piece(const ID* __restrict__ ids, int64_t begin, int64_t end,
                                            int E, int* cnt) {
  for (int64_t i = begin + (threadIdx.x & 63); i < end; i += 64) {
    const int e = expert_of(ids, i, end, E);
    if (e < E) atomicAdd(&cnt[e], 1);  // integers: any order gives the same count
  }
}

}  // namespace

template <typename ID>
__global__ __launch_bounds__(1024) void moe_count_kernel(const ID* __restrict__ ids, int64_t n,
                                                         int64_t piece, int E,
                                                         int32_t* __restrict__ counts) {
  extern __shared__ int cnt[];  // [E]
  for (int e = threadIdx.x; e < E; e += 1024) cnt[e] = 0;
  __syncthreads();
  const int64_t begin = ((int64_t)blockIdx.x * kSortWaves + (threadIdx.x >> 6)) * piece;
  const int64_t end = begin + piece < n ? begin + piece : n;
  count_piece(ids, begin, end, E, cnt);
  __syncthreads();
  for (int e = threadIdx.x; e < E; e += 1024) counts[(int64_t)blockIdx.x * E + e] = cnt[e];
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
  for (int i = t; i < kSortWaves * E; i += 1024) cnt[i] = 0;
  __syncthreads();
  const int64_t begin = ((int64_t)blockIdx.x * kSortWaves + wave) * piece;
  const int64_t end = begin + piece < n ? begin + piece : n;
  int* mine = cnt + wave * E;
  count_piece(ids, begin, end, E, mine);
  __syncthreads();

  // thread e: expert e's choices in this block (by wave), in earlier blocks and in all
  int total = 0, before = 0;
  if (t < E) {
    if (counts) {
      for (int b = 0; b < (int)gridDim.x; ++b) {
        const int c = counts[(int64_t)b * E + t];
        total += c;
        before += b < (int)blockIdx.x ? c : 0;
      }
    } else {
      for (int w = 0; w < kSortWaves; ++w) total += cnt[w * E + t];
    }
  }
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

  for (int64_t i0 = begin; i0 < end; i0 += 64) {
    const int64_t i = i0 + lane;
    const int e = expert_of(ids, i, end, E);
    uint64_t same = ~0ull;
    for (int b = 0; b < bits; ++b) {
      const uint64_t set = __ballot((e >> b) & 1);
      same &= (e >> b) & 1 ? set : ~set;
    }
    const int below = __popcll(same & ((1ull << lane) - 1));
    int at = 0;
    if (below == 0 && e < E) at = atomicAdd(&mine[e], (int)__popcll(same));
    at = __shfl(at, __ffsll((unsigned long long)same) - 1, 64) + below;
    if (i < end) {
      pos[i] = e < E ? at : -1;
      if (e < E) row_ids[at] = (int)((unsigned)i / (unsigned)top_k);
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
// Rows. 8 values per lane and chunk. A value type is float or uint16_t (bf16).
// ---------------------------------------------------------------------------------------------
namespace {

__device__ __forceinline__ void load8(const uint16_t* p, float (&f)[8]) {
  widen8(__builtin_nontemporal_load(reinterpret_cast<const u32x4*>(p)), f);
}
__device__ __forceinline__ void load8(const float* p, float (&f)[8]) {
  typedef float f32x4 __attribute__((ext_vector_type(4)));
  const f32x4 a = __builtin_nontemporal_load(reinterpret_cast<const f32x4*>(p));
  const f32x4 b = __builtin_nontemporal_load(reinterpret_cast<const f32x4*>(p) + 1);
  f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w, f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
}
__device__ __forceinline__ void store8(uint16_t* p, const float (&f)[8]) {
  *reinterpret_cast<u32x4*>(p) = round8(f);
}
__device__ __forceinline__ void store8(float* p, const float (&f)[8]) {
  reinterpret_cast<float4*>(p)[0] = make_float4(f[0], f[1], f[2], f[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(f[4], f[5], f[6], f[7]);
}

constexpr int kAtOnce = 8;  // choices whose rows are in flight together

}  // namespace

// One token per workgroup: its row is read once and written to each of its grouped rows.
__global__ __launch_bounds__(256) void moe_dispatch_kernel(MoeArgs a) {
  const int64_t t = blockIdx.x;
  const uint16_t* x = static_cast<const uint16_t*>(a.x) + t * a.ld_x;
  uint16_t* out = static_cast<uint16_t*>(a.out);
  const int32_t* __restrict__ pos = a.pos + t * a.top_k;
  for (int c = threadIdx.x; c < a.nc; c += blockDim.x) {
    const u32x4 v = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(x) + c);
    for (int j = 0; j < a.top_k; ++j) {
      const int64_t p = pos[j];
      if (p >= 0 && p < a.R)
        __builtin_nontemporal_store(v, reinterpret_cast<u32x4*>(out + p * a.ld_out) + c);
    }
  }
}

template <typename Y, typename O>
__global__ __launch_bounds__(256) void moe_combine_kernel(MoeArgs a) {
  const int64_t t = blockIdx.x;
  const Y* y = static_cast<const Y*>(a.x);
  O* out = static_cast<O*>(a.out) + t * a.ld_out;
  const int32_t* __restrict__ pos = a.pos + t * a.top_k;
  const float* __restrict__ w = a.weights ? a.weights + t * a.top_k : nullptr;
  for (int c = threadIdx.x; c < a.nc; c += blockDim.x) {
    float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    for (int j0 = 0; j0 < a.top_k; j0 += kAtOnce) {
      float f[kAtOnce][8];
      float wj[kAtOnce];
#pragma unroll
      for (int j = 0; j < kAtOnce; ++j) {
        const int64_t p = j0 + j < a.top_k ? pos[j0 + j] : -1;
        const bool live = p >= 0 && p < a.R;  // uniform
        wj[j] = live ? (w ? w[j0 + j] : 1.f) : 0.f;
#pragma unroll
        for (int k = 0; k < 8; ++k) f[j][k] = 0.f;
        if (live) load8(y + p * a.ld_x + c * 8, f[j]);
      }
#pragma unroll
      for (int j = 0; j < kAtOnce; ++j)
#pragma unroll
        for (int k = 0; k < 8; ++k) acc[k] = __builtin_fmaf(wj[j], f[j][k], acc[k]);
    }
    store8(out + c * 8, acc);
  }
}

template <typename Y>
__global__ __launch_bounds__(256) void moe_combine_bwd_kernel(MoeArgs a) {
  __shared__ float red[4][kAtOnce];
  const int64_t t = blockIdx.x;
  const uint16_t* dout = static_cast<const uint16_t*>(a.x) + t * a.ld_x;
  const Y* y = static_cast<const Y*>(a.y);  // may be out: each value is read before it is written
  Y* dy = static_cast<Y*>(a.out);
  const int32_t* __restrict__ pos = a.pos + t * a.top_k;
  const float* __restrict__ w = a.weights ? a.weights + t * a.top_k : nullptr;
  const int waves = blockDim.x >> 6;
  for (int j0 = 0; j0 < a.top_k; j0 += kAtOnce) {
    float dot[kAtOnce];
#pragma unroll
    for (int j = 0; j < kAtOnce; ++j) dot[j] = 0.f;
    for (int c = threadIdx.x; c < a.nc; c += blockDim.x) {
      float g[8];
      load8(dout + c * 8, g);
      float f[kAtOnce][8];
      if (y) {
#pragma unroll
        for (int j = 0; j < kAtOnce; ++j) {
          const int64_t p = j0 + j < a.top_k ? pos[j0 + j] : -1;
#pragma unroll
          for (int k = 0; k < 8; ++k) f[j][k] = 0.f;
          if (p >= 0 && p < a.R) load8(y + p * a.ld_y + c * 8, f[j]);
        }
#pragma unroll
        for (int j = 0; j < kAtOnce; ++j)
#pragma unroll
          for (int k = 0; k < 8; ++k) dot[j] = __builtin_fmaf(g[k], f[j][k], dot[j]);
      }
#pragma unroll
      for (int j = 0; j < kAtOnce; ++j) {
        const int64_t p = j0 + j < a.top_k ? pos[j0 + j] : -1;
        if (p < 0 || p >= a.R) continue;
        const float wj = w ? w[j0 + j] : 1.f;
        float d[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) d[k] = wj * g[k];
        store8(dy + p * a.ld_out + c * 8, d);
      }
    }
    if (!a.dweights) continue;
#pragma unroll
    for (int j = 0; j < kAtOnce; ++j) dot[j] = wave_sum(dot[j]);
    __syncthreads();  // the sums of the choices before have been read
    if ((threadIdx.x & 63) == 0)
#pragma unroll
      for (int j = 0; j < kAtOnce; ++j) red[threadIdx.x >> 6][j] = dot[j];
    __syncthreads();
    const int j = threadIdx.x;
    if (j < kAtOnce && j0 + j < a.top_k) {
      float s = red[0][j];
      for (int k = 1; k < waves; ++k) s += red[k][j];
      const int64_t p = pos[j0 + j];
      a.dweights[t * a.top_k + j0 + j] = p >= 0 && p < a.R ? s : 0.f;
    }
  }
}

namespace {

// Threads of a workgroup that owns one token: a lane per chunk, up to four waves.
dim3 row_threads(int nc) { return dim3(nc >= 256 ? 256 : nc > 64 ? (nc + 63) / 64 * 64 : 64); }

}  // namespace

hipError_t launch_moe_dispatch(const MoeArgs& a, hipStream_t stream) {
  hipLaunchKernelGGL(moe_dispatch_kernel, dim3((unsigned)a.T), row_threads(a.nc), 0, stream, a);
  return hipGetLastError();
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
  const dim3 g((unsigned)a.T), t = row_threads(a.nc);
  if (y_f32)
    hipLaunchKernelGGL(moe_combine_bwd_kernel<float>, g, t, 0, stream, a);
  else
    hipLaunchKernelGGL(moe_combine_bwd_kernel<uint16_t>, g, t, 0, stream, a);
  return hipGetLastError();
}

}  // namespace fp8rl
