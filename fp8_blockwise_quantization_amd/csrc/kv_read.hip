// Cached keys and values back as contiguous bf16 rows.
//
// A wave takes kRows rows of the outputs. Lane i finds out where row i comes from (its sequence by
// a search of the offsets, then its page), all rows at once, because these are loads that wait for
// one another; the rows themselves then move with every lane on 8 values at a time.
//
// Bound by memory: 16 sequences, 32768 keys of 8 heads of 128 in E4M3, 67 MB read and 134 written
// in 32 us, 6.2 TB/s (a device copy moves 5.0 to 5.5).
#include "attn_ops.hpp"

namespace fp8rl {

namespace {

constexpr int kRows = 4;

struct ReadArgs {
  fp8rl_kv_read_args a;
  PageOf page_of;
  int chunks;  // of 8 values in a row
  int waves;
};

}  // namespace

template <bool CODES>
__global__ __launch_bounds__(256) void kv_read_kernel(ReadArgs r) {
  const fp8rl_kv_read_args& a = r.a;
  const int lane = (int)(threadIdx.x & 63);
  const int wave = __builtin_amdgcn_readfirstlane((int)(blockIdx.x * 4 + (threadIdx.x >> 6)));
  if (wave >= r.waves) return;
  const int row0 = wave * kRows;

  int64_t from = -1;  // lane i: the cache row that row0 + i is a copy of
  {
    int b = last_not_past((int)a.B, row0, lane, [&](int i) { return a.offsets[i]; });
    const int row = row0 + lane;
    if (lane < kRows && row < a.R) {
      // the row's sequence: as a rule row0's, else past that in doubling steps
      auto past = [&](int i) { return i <= (int)a.B && a.offsets[i] <= row; };
      int step = 1;
      for (; past(b + step); step *= 2) b += step;
      for (; step > 0; step /= 2)
        if (past(b + step)) b += step;
      if (b < (int)a.B && a.offsets[b] <= row) {
        const int64_t key = (int64_t)row - a.offsets[b] + (a.starts ? a.starts[b] : 0);
        if (key >= 0 && key < (int64_t)a.table_width * a.page_size) {
          const int i = r.page_of((int)key);
          const int page = a.page_table[b * a.ld_table + i];
          if (page >= 0 && page < a.num_pages)
            from = page * a.page_stride + ((int)key - i * a.page_size) * a.slot_stride;
        }
      }
    }
  }
  float k_scale = 1.f, v_scale = 1.f;
  if (CODES) k_scale = *a.k_scale, v_scale = *a.v_scale;
  const int per_head = a.head_dim >> 3;

  for (int c = lane; c < r.chunks; c += 64) {
    const int head = c / per_head;
    const int64_t at = head * a.head_stride + 8 * (c - head * per_head);
    u32x4 k[kRows], v[kRows];
    int64_t src[kRows];
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)from, i);
      const uint32_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(from >> 32), i);
      src[i] = (int64_t)((uint64_t)hi << 32 | lo);
      if (src[i] < 0) continue;
      if constexpr (CODES) {
        const u32x2 x = *reinterpret_cast<const u32x2*>(static_cast<const uint8_t*>(a.k_cache) +
                                                        src[i] + at);
        const u32x2 y = *reinterpret_cast<const u32x2*>(static_cast<const uint8_t*>(a.v_cache) +
                                                        src[i] + at);
        k[i].x = x.x, k[i].y = x.y, v[i].x = y.x, v[i].y = y.y;
      } else {
        k[i] = *reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(a.k_cache) + src[i] +
                                               at);
        v[i] = *reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(a.v_cache) + src[i] +
                                               at);
      }
    }
    auto widen = [](u32x4 w, float s) {
      if constexpr (!CODES) return w;
      const u32x2 p = codes_bf16(w.x), q = codes_bf16(w.y);
      float f[8];
      widen8(u32x4{p.x, p.y, q.x, q.y}, f);
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] *= s;
      return round8(f);
    };
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      if (src[i] < 0) continue;
      const int64_t row = row0 + i;
      __builtin_nontemporal_store(widen(k[i], k_scale),
                                  reinterpret_cast<u32x4*>(a.k_out + row * a.ld_k) + c);
      __builtin_nontemporal_store(widen(v[i], v_scale),
                                  reinterpret_cast<u32x4*>(a.v_out + row * a.ld_v) + c);
    }
  }
}

hipError_t launch_kv_read(const fp8rl_kv_read_args& a, hipStream_t stream) {
  ReadArgs r;
  r.a = a;
  r.page_of = PageOf(a.page_size);
  r.chunks = a.kv_heads * (a.head_dim / 8);
  r.waves = (int)((a.R + kRows - 1) / kRows);
  const dim3 grid((unsigned)((r.waves + 3) / 4));
  if (a.k_scale)
    hipLaunchKernelGGL(kv_read_kernel<true>, grid, dim3(256), 0, stream, r);
  else
    hipLaunchKernelGGL(kv_read_kernel<false>, grid, dim3(256), 0, stream, r);
  return hipGetLastError();
}

}  // namespace fp8rl
